"""Operators on the paged KV cache, in their plain form and through the library.

Three groups of operators, each a pass of `run`:
  pages   fork   a batch is laid out anew (forked, reordered, freed, grown): fork_sequences
          copy   blocks are copied between two pools: copy_blocks
          compact  the used blocks move to the low end of the pool: compact_blocks
  shared  a decode step of a batch whose sequences share prefixes in groups: decode_shared
  sparse  score    summaries of the newest blocks, and every block's score: summarize_blocks, score_blocks
          select   the blocks each (sequence, KV head) attends to: select_blocks
          attend   the decode step over the selected blocks: decode_selected

Cache block: [BS slots][Hk heads][K | V][128] elements (bf16 or e4m3), then for e4m3 fp32 scales
[Hk][K, V][BS].  Lengths are a fixed spread of each case's range; the seed shuffles them.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # four beams of a short text: two survive and fork, every row grows by one token
        dict(name="fork_beam4", op="fork", B=4, fan=2, Hk=8, BS=16, MB=16, NB=128, kv="bf16", lo=1, hi=250, grow=1),
        # parallel sampling: every fourth of 64 sequences forks in four (lognormal-like lengths, fp8 pool)
        dict(name="fork_b64_fp8", op="fork", B=64, fan=4, Hk=8, BS=16, MB=1024, NB=16384, kv="fp8", lo=16, hi=16000,
             grow=1),
        # blocks swapped into another pool in one call
        dict(name="copy_2048_blocks", op="copy", n=2048, Hk=4, BS=32, NB=4096, kv="bf16"),
        # a pool that is half empty after a burst of requests is packed
        dict(name="compact_8192", op="compact", B=32, Hk=8, BS=16, MB=256, NB=8192, kv="bf16", lo=300, hi=4000),
        # two short continuations of one short prompt: latency
        dict(name="shared_b2_ctx250", op="shared", B=2, NG=1, Hk=1, QG=8, BS=16, kv="bf16", plo=250, phi=250, lo=1, hi=16),
        # one system prompt for 64 users, fp8 cache
        dict(name="shared_b64_fp8_ctx4001", op="shared", B=64, NG=1, Hk=8, QG=6, BS=16, kv="fp8", plo=4001, phi=4001,
             lo=1, hi=500),
        # four prompts of different lengths, groups of different sizes, some continuations still empty
        dict(name="shared_b32_g4", op="shared", B=32, NG=4, Hk=4, QG=16, BS=32, kv="bf16", plo=2048, phi=8190, lo=0,
             hi=1000),
        # a long document asked about 128 times
        dict(name="shared_b128_ctx32768", op="shared", B=128, NG=1, Hk=8, QG=8, BS=32, kv="bf16", plo=32768, phi=32768,
             lo=1, hi=200),
        # long contexts: the newest block's summary is renewed and every block scored
        dict(name="score_b16_ctx32768", op="score", B=16, Hk=8, QG=8, BS=32, MB=1280, kv="bf16", lo=16001, hi=32768,
             fresh=1),
        # 64 of up to 1024 blocks for each (sequence, KV head)
        dict(name="select_b16_k64", op="select", B=16, Hk=8, BS=32, MB=1280, K=64, first=1, last=2, lo=16001, hi=32768),
        # four long contexts, 64 blocks of 32 tokens each
        dict(name="attend_b4_k64", op="attend", B=4, Hk=8, QG=8, BS=32, NB=5120, K=64, kv="bf16"),
        # a full fp8 batch, 128 blocks of 16 tokens each
        dict(name="attend_b64_k128_fp8", op="attend", B=64, Hk=8, QG=6, BS=16, NB=16384, K=128, kv="fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _smaller(c):
    """Fewer heads where the pool would pass 600 MB."""
    while c["Hk"] > 1 and c["NB"] * _block_bytes(c) > 600e6:
        c["Hk"] //= 2
    return c


def draw(rng):
    op = rng.choice(["fork", "copy", "compact", "shared", "shared", "score", "select", "attend"])
    kv = rng.choice(["bf16", "fp8"])
    BS = rng.choice([16, 32])
    Hk = rng.choice([1, 2, 4, 5, 8])
    QG = rng.choice([6, 8, 16])
    if op == "fork":
        fan = rng.choice([1, 2, 3, 4])
        B = fan * _log(rng, 1, 48 // fan)
        hi = _log(rng, 20, 4000)
        grow = rng.choice([0, 1, 1, 7])
        MB = -(-(hi + grow) // BS) + rng.randint(0, 40)
        NB = B * (-(-hi // BS)) + 2 * B + rng.randint(1, 60)
        return _smaller(dict(op=op, B=B, fan=fan, Hk=Hk, BS=BS, MB=MB, NB=NB, kv=kv, lo=rng.randint(0, hi), hi=hi,
                             grow=grow))
    if op == "copy":
        n = _log(rng, 1, 2048)
        return dict(op=op, n=n, Hk=min(Hk, 4), BS=BS, NB=n + rng.randint(1, 500), kv=kv)
    if op == "compact":
        hi, B = _log(rng, 20, 3000), _log(rng, 1, 32)
        NB = B * -(-hi // BS) * rng.choice([1, 2]) + rng.randint(1, 80)
        return _smaller(dict(op=op, B=B, Hk=Hk, BS=BS, MB=-(-hi // BS) + rng.randint(0, 20), NB=NB, kv=kv,
                             lo=rng.randint(0, hi), hi=hi))
    if op == "shared":
        NG = rng.choice([1, 1, 2, 3, 5])
        B = NG * _log(rng, 1, 64 // NG)
        phi = _log(rng, 60, 20000)
        return dict(op=op, B=B, NG=NG, Hk=Hk, QG=QG, BS=BS, kv=kv, plo=phi if NG == 1 else rng.randint(phi // 3, phi), phi=phi,
                    lo=rng.randint(0, 3), hi=_log(rng, 4, 600))
    hi = _log(rng, 300, 32000)
    MB = -(-hi // BS) + rng.randint(0, 50)
    B = _log(rng, 1, 16)
    if op == "score":
        return dict(op=op, B=B, Hk=Hk, QG=QG, BS=BS, MB=MB, kv=kv, lo=rng.randint(0, hi), hi=hi, fresh=rng.choice([1, 1, BS + 3, hi]))
    K = _log(rng, 4, 128)
    if op == "select":
        return dict(op=op, B=B, Hk=Hk, BS=BS, MB=MB, K=K, first=rng.choice([0, 1, 2]), last=rng.choice([0, 1, 2]), lo=rng.randint(0, hi),
                    hi=hi)
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, Hk=Hk, QG=QG, BS=BS, NB=K + rng.randint(50, 9000), K=K, kv=kv)


# ---------------------------------------------------------------------------- sizes
def _block_bytes(c):
    return c["BS"] * c["Hk"] * (4 * D if c["kv"] == "bf16" else 2 * D + 8)


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm where the range is wide."""
    if n == 1:
        return [hi]
    if hi > 10 * max(lo, 1):
        a, b = math.log(lo + 1), math.log(hi + 1)
        return [int(round(math.exp(a + (b - a) * i / (n - 1)) - 1)) for i in range(n)]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _group_starts(c):
    """Groups of different sizes that cover the batch."""
    B, NG = c["B"], c["NG"]
    return [int(round(B * (g / NG) ** 1.2)) for g in range(NG + 1)]


def work(case):
    c = dict(case)
    op = c["op"]
    if op == "fork":
        B, parents = c["B"], c["B"] // c["fan"]
        copies = B - parents     # each parent's first child keeps the parent's last block
        meta = 2 * 4 * (c["NB"] + B * c["MB"]) + 16 * B
        return {"bytes": 2.0 * copies * _block_bytes(c) + meta, "flops": 0.0}
    if op == "copy":
        return {"bytes": 2.0 * c["n"] * _block_bytes(c) + 8 * c["n"], "flops": 0.0}
    if op == "compact":
        used = sum(-(-x // c["BS"]) for x in _spread(c["B"], c["lo"], c["hi"]))
        moved = used * (c["NB"] - used) / c["NB"]
        return {"bytes": 2.0 * moved * _block_bytes(c) + 4 * (3 * c["NB"] + 2 * c["B"] * c["MB"]), "flops": 0.0}
    if op == "shared":
        starts, plens = _group_starts(c), _spread(c["NG"], c["plo"], c["phi"])
        own_tokens = sum(_spread(c["B"], c["lo"], c["hi"]))
        tok = _block_bytes(c) / c["BS"]
        rows = c["B"] * c["Hk"] * c["QG"]
        dots = sum((starts[g + 1] - starts[g]) * plens[g] for g in range(c["NG"])) + own_tokens
        return {"bytes": (sum(plens) + own_tokens) * tok + rows * D * 4, "flops": 4.0 * D * dots * c["Hk"] * c["QG"]}
    if op == "score":
        lens = _spread(c["B"], c["lo"], c["hi"])
        nb = sum(-(-x // c["BS"]) for x in lens)
        renewed = sum(-(-x // c["BS"]) - max(0, x - c["fresh"]) // c["BS"] for x in lens)
        keys = renewed * _block_bytes(c) / 2
        per = nb * c["Hk"]
        return {"bytes": per * (4 * D + 4) + keys + renewed * c["Hk"] * 4 * D + c["B"] * c["Hk"] * c["QG"] * D * 2,
                "flops": 4.0 * per * c["QG"] * D}
    if op == "select":
        nb = sum(-(-x // c["BS"]) for x in _spread(c["B"], c["lo"], c["hi"]))
        return {"bytes": 4.0 * c["Hk"] * (nb + c["B"] * (2 * c["K"] + 1)), "flops": 0.0}
    tokens = c["B"] * c["Hk"] * c["K"] * c["BS"]
    return {"bytes": tokens * _block_bytes(c) / c["BS"] / c["Hk"] + c["B"] * c["Hk"] * (c["K"] * 4 + c["QG"] * D * 4),
            "flops": 4.0 * D * tokens * c["QG"]}


# ---------------------------------------------------------------------------- inputs
def _make_cache(c, gen, NB, pool=None):
    """A pool of NB blocks with N(0, 1) keys and values (keys of a head share an offset), uint8."""
    BS, Hk = c["BS"], c["Hk"]
    cbb = _block_bytes(c)
    cache = torch.empty(NB, cbb, dtype=torch.uint8, device=DEV)
    bias = torch.randn(Hk, 2, D, generator=gen, device=DEV) * torch.tensor([0.5, 0.0], device=DEV)[:, None]
    step = max(1, (1 << 26) // (BS * Hk * 2 * D))
    for i in range(0, NB, step):
        n = min(step, NB - i)
        x = torch.randn(n, BS, Hk, 2, D, generator=gen, device=DEV) + bias
        if c["kv"] == "bf16":
            cache[i:i + n].view(torch.bfloat16).copy_(x.view(n, -1))
        else:
            scale = x.abs().amax(-1) / 448.0
            codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, -1)
            cache[i:i + n, :codes.shape[1]] = codes
            cache[i:i + n, codes.shape[1]:] = scale.permute(0, 2, 3, 1).contiguous().view(n, -1).view(torch.uint8)
    return cache.view(-1)


def _lens(rs, B, lo, hi):
    x = np.array(_spread(B, lo, hi), np.int32)
    rs.shuffle(x)
    return x


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _tables(rs, lens, BS, MB, ids):
    """Block tables [B][MB] filled from the ids in order; unused entries are -1."""
    t = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for b, n in enumerate(-(-np.asarray(lens) // BS)):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, at


KV = {"bf16": 0, "fp8": 1}


def prepare(case, seed):
    c = dict(case)
    op = c["op"]
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(c=c)
    bf = torch.bfloat16
    if op in ("fork", "compact"):
        lens = _lens(rs, c["B"], c["lo"], c["hi"])
        table, used = _tables(rs, lens, c["BS"], c["MB"], rs.permutation(c["NB"]))
        refs = np.zeros(c["NB"], np.int32)
        refs[table[table >= 0]] = 1
        s.update(cache=_make_cache(c, gen, c["NB"]), table=_i32(table), lens=_i32(lens), refs=_i32(refs),
                 out_table=_i32(table), out_refs=_i32(refs))
        if op == "fork":
            chosen = rs.permutation(c["B"])[:c["B"] // c["fan"]]
            s.update(parents=_i32(rs.permutation(np.repeat(chosen, c["fan"]))), grow=_i32(np.full(c["B"], c["grow"])),
                     out_lens=_i32(lens))
        else:
            s.update(remap=_i32(refs), num_used=_i32([0]))
    elif op == "copy":
        pairs = np.stack([rs.permutation(c["NB"])[:c["n"]], rs.permutation(c["NB"])[:c["n"]]], 1)
        s.update(src=_make_cache(c, gen, c["NB"]), dst=_make_cache(c, gen, c["NB"]), pairs=_i32(pairs))
    elif op == "shared":
        B, NG, BS = c["B"], c["NG"], c["BS"]
        plens, lens = _lens(rs, NG, c["plo"], c["phi"]), _lens(rs, B, c["lo"], c["hi"])
        if NG > 1:      # the spread's order decides the work of each group: only its values move with the seed
            plens = np.array(_spread(NG, c["plo"], c["phi"]), np.int32)
        MP, MB = -(-c["phi"] // BS), max(1, -(-c["hi"] // BS))
        need = int((-(-plens // BS)).sum() + (-(-lens // BS)).sum())
        NB = need + 16
        ids = rs.permutation(NB)
        ptable, at = _tables(rs, plens, BS, MP, ids)
        table, _ = _tables(rs, lens, BS, MB, ids[at:])
        s.update(cache=_make_cache(c, gen, NB), NB=NB, MP=MP, MB=MB, ptable=_i32(ptable), plens=_i32(plens),
                 table=_i32(table), lens=_i32(lens), starts=_i32(_group_starts(c)),
                 q=torch.randn(B, c["Hk"] * c["QG"], D, generator=gen, device=DEV).to(bf),
                 out=torch.zeros(B, c["Hk"] * c["QG"], D, dtype=bf, device=DEV))
    elif op == "score":
        lens = _lens(rs, c["B"], c["lo"], c["hi"])
        NB = int((-(-lens // c["BS"])).sum()) + 16
        table, _ = _tables(rs, lens, c["BS"], c["MB"], rs.permutation(NB))
        s.update(cache=_make_cache(c, gen, NB), NB=NB, table=_i32(table), lens=_i32(lens),
                 since=_i32(np.maximum(0, lens - c["fresh"])),
                 q=torch.randn(c["B"], c["Hk"] * c["QG"], D, generator=gen, device=DEV).to(bf),
                 scores=torch.zeros(c["B"], c["Hk"], c["MB"], device=DEV))
        # summaries of the older blocks, as earlier steps left them
        key = _values(s["cache"], c, torch.arange(NB, device=DEV))[..., 0, :]       # [NB][BS][Hk][D]
        s["summaries"] = torch.stack([_outward(key.amax(1), True), _outward(key.amin(1), False)], 2).contiguous()
    elif op == "select":
        lens = _lens(rs, c["B"], c["lo"], c["hi"])
        need = int((-(-lens // c["BS"])).sum())
        table, _ = _tables(rs, lens, c["BS"], c["MB"], rs.permutation(need + 16))
        # scores of one row share an offset; some are equal, as those of equal blocks are
        x = torch.randn(c["B"], c["Hk"], c["MB"], generator=gen, device=DEV) + 4.0
        x[:, :, ::7] = (x[:, :, ::7] * 4).round() / 4
        s.update(NB=need + 16, table=_i32(table), lens=_i32(lens), scores=x,
                 sel_table=_i32(np.zeros((c["B"], c["Hk"], c["K"]))), sel_blocks=_i32(np.zeros((c["B"], c["Hk"], c["K"]))),
                 sel_lens=_i32(np.zeros((c["B"], c["Hk"]))))
    else:       # attend
        B, Hk, K = c["B"], c["Hk"], c["K"]
        table = np.stack([rs.permutation(c["NB"])[:K] for _ in range(B * Hk)]).reshape(B, Hk, K)
        # the newest block is among the selected ones and ends anywhere
        lens = K * c["BS"] - rs.randint(0, c["BS"], (B, 1)) * np.ones((1, Hk), np.int64)
        s.update(cache=_make_cache(c, gen, c["NB"]), sel_table=_i32(table), sel_lens=_i32(lens),
                 q=torch.randn(B, Hk * c["QG"], D, generator=gen, device=DEV).to(bf),
                 out=torch.zeros(B, Hk * c["QG"], D, dtype=bf, device=DEV))
    if own:
        import paged_kv_gqa_block_gb300 as pda
        kv = KV[c.get("kv", "bf16")]
        qg = c.get("QG", 8)
        s["pda"] = pda
        if op in ("fork", "compact"):
            s["p"] = pda.plan(c["B"], c["Hk"], qg, c["BS"], c["MB"], kv_dtype=kv)
            s["ws"] = pda.page_workspace(s["p"], c["B"], c["NB"], DEV)
        elif op == "copy":
            s["p"] = pda.plan(1, c["Hk"], qg, c["BS"], 1, kv_dtype=kv)
        elif op == "shared":
            s["pp"], s["p"] = pda.shared_plans(c["B"], c["NG"], c["Hk"], qg, c["BS"], s["MP"], s["MB"], kv_dtype=kv)
            s["ws"] = pda.shared_workspace(s["pp"], s["p"], DEV)
        elif op in ("score", "select"):
            s["p"] = pda.plan(c["B"], c["Hk"], qg, c["BS"], c["MB"], kv_dtype=kv)
        else:
            s["p"] = pda.plan(c["B"], c["Hk"], qg, c["BS"], c["K"], kv_dtype=kv)
            s["ws"] = pda.workspace(s["p"], DEV)
    return s


# ---------------------------------------------------------------------------- plain forms
def _values(cache, c, ids):
    """The fp32 values of the blocks `ids` [...]: [...][BS][Hk][2][D]."""
    BS, Hk = c["BS"], c["Hk"]
    blocks = cache.view(-1, _block_bytes(c))[ids]
    if c["kv"] == "bf16":
        return blocks.view(torch.bfloat16).float().unflatten(-1, (BS, Hk, 2, D))
    n = BS * Hk * 2 * D
    x = blocks[..., :n].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (BS, Hk, 2, D))
    scale = blocks[..., n:].contiguous().view(torch.float32).unflatten(-1, (Hk, 2, BS))
    return x * scale.movedim(-1, -3)[..., None]


def _outward(x, up):
    """fp32 to bf16, up or down, so that the rounded value still bounds x."""
    r = x.to(torch.bfloat16)
    short = r.float() < x if up else r.float() > x
    bits = r.view(torch.int16).to(torch.int32) & 0xFFFF
    # one step up is +1 for positive codes and -1 for negative ones (away from -0: the smallest positive code)
    neg = bits >= 0x8000
    away = neg ^ up
    step = torch.where(away, 1, -1)
    nxt = torch.where((bits & 0x7FFF) == 0, torch.full_like(bits, 1 if up else 0x8001), bits + step)
    return torch.where(short, nxt, bits).to(torch.int16).view(torch.bfloat16)


def _fork_plain(s):
    c = s["c"]
    B, BS, MB, NB = c["B"], c["BS"], c["MB"], c["NB"]
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"].long()
    par, grow = s["parents"].long(), s["grow"].long()
    j, rows = torch.arange(MB, device=DEV), torch.arange(B, device=DEV)
    held = (lens + BS - 1) // BS
    counts = refs.clone()
    counts.scatter_add_(0, table.clamp(min=0).flatten(), -(j < held[:, None]).long().flatten())
    valid = (par >= 0) & (par < B)
    pc = par.clamp(0, B - 1)
    L = lens[pc]
    new = L + grow
    valid &= new <= MB * BS
    L, new = torch.where(valid, L, 0), torch.where(valid, new, 0)
    full, h0, h1 = L // BS, (L + BS - 1) // BS, (new + BS - 1) // BS
    first = torch.full((B,), B, device=DEV).scatter_reduce(0, pc, torch.where(valid, rows, B), "amin")[pc] == rows
    tail_id = table[pc].gather(1, full.clamp(max=MB - 1)[:, None])[:, 0]
    tail = full < h0
    copy = tail & ~(first & (refs[tail_id.clamp(min=0)] == 1))
    need = copy.long() + h1 - h0
    off = need.cumsum(0) - need
    is_free = refs == 0
    rank = is_free.long().cumsum(0) - 1
    free = torch.zeros(NB + 1, dtype=torch.long, device=DEV).scatter_(0, torch.where(is_free, rank, NB), torch.arange(NB, device=DEV))
    ok = off + need <= is_free.sum()
    L, new, full, h0, h1 = (torch.where(ok, x, 0) for x in (L, new, full, h0, h1))
    copy, tail = copy & ok, tail & ok
    fresh = free[(off[:, None] + copy[:, None] + j - h0[:, None]).clamp(0, NB)]
    t = torch.where(j < full[:, None], table[pc], -1)
    t = torch.where(tail[:, None] & (j == full[:, None]), torch.where(copy, free[off.clamp(max=NB)], tail_id)[:, None], t)
    t = torch.where((j >= h0[:, None]) & (j < h1[:, None]), fresh, t)
    counts.scatter_add_(0, t.clamp(min=0).flatten(), (t >= 0).long().flatten())
    blocks = s["cache"].view(NB, -1)
    some = copy.nonzero()[:, 0]
    blocks[free[off[some]]] = blocks[tail_id[some]]
    i32 = torch.int32
    return s["cache"].view(torch.bfloat16) if c["kv"] == "bf16" else s["cache"], t.to(i32), new.to(i32), counts.to(i32)


def _compact_plain(s):
    c = s["c"]
    NB, BS = c["NB"], c["BS"]
    table, lens, refs = s["table"].long(), s["lens"].long(), s["refs"]
    ids = torch.arange(NB, device=DEV)
    used = refs > 0
    U = used.sum()
    movers, holes = (used & (ids >= U)).nonzero()[:, 0], (~used & (ids < U)).nonzero()[:, 0]
    remap = torch.where(used, ids, -1)
    remap[movers] = holes
    blocks = s["cache"].view(NB, -1)
    blocks[holes] = blocks[movers]
    counts = torch.where(ids < U, refs, 0)
    counts[holes] = refs[movers]
    held = torch.arange(c["MB"], device=DEV) < ((lens + BS - 1) // BS)[:, None]
    t = torch.where(held, remap[table.clamp(min=0)], -1)
    i32 = torch.int32
    cache = s["cache"].view(torch.bfloat16) if c["kv"] == "bf16" else s["cache"]
    return cache, t.to(i32), counts.to(i32), remap.to(i32), U.to(i32).view(1)


def _parts(logits, v):
    """Running maximum, sum and weighted values of one set of keys: logits [..., r, t], v [..., t, d]."""
    m = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - m.clamp(min=-3e38))
    return m, e.sum(-1, keepdim=True), e @ v


def _shared_plain(s):
    c = s["c"]
    B, NG, Hk, QG, BS = c["B"], c["NG"], c["Hk"], c["QG"], c["BS"]
    scale = D ** -0.5
    q = s["q"].float().view(B, Hk, QG, D)
    starts = s["starts"].long()
    n = max(b - a for a, b in zip(_group_starts(c), _group_starts(c)[1:]))
    pos = torch.arange(n, device=DEV)
    rows = (starts[:-1, None] + pos).clamp(max=B - 1)                               # [NG][n]
    kv = _values(s["cache"], c, s["ptable"].long().clamp(min=0)).flatten(1, 2)      # [NG][T][Hk][2][D]
    k, v = kv[..., 0, :].permute(0, 2, 3, 1), kv[..., 1, :].permute(0, 2, 1, 3)
    qg = q[rows].permute(0, 2, 1, 3, 4).reshape(NG, Hk, n * QG, D)
    dead = torch.arange(k.shape[-1], device=DEV) >= s["plens"].long()[:, None]
    pm, pl, po = _parts((qg @ k * scale).masked_fill_(dead[:, None, None], float("-inf")), v)
    group = (torch.arange(B, device=DEV)[:, None] >= starts[None, 1:]).sum(1)
    at = torch.arange(B, device=DEV) - starts[group]
    pm, pl, po = (x.view(NG, Hk, n, QG, -1)[group, :, at] for x in (pm, pl, po))    # [B][Hk][QG][.]
    kv = _values(s["cache"], c, s["table"].long().clamp(min=0)).flatten(1, 2)
    k, v = kv[..., 0, :].permute(0, 2, 3, 1), kv[..., 1, :].permute(0, 2, 1, 3)
    dead = torch.arange(k.shape[-1], device=DEV) >= s["lens"].long()[:, None]
    sm, sl, so = _parts((q @ k * scale).masked_fill_(dead[:, None, None], float("-inf")), v)
    m = torch.maximum(pm, sm).clamp(min=-3e38)
    wp, ws = torch.exp(pm - m), torch.exp(sm - m)
    total = pl * wp + sl * ws
    out = (po * wp + so * ws) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, Hk * QG, D).to(torch.bfloat16)


def _score_plain(s):
    c = s["c"]
    B, Hk, QG, BS, MB = c["B"], c["Hk"], c["QG"], c["BS"], c["MB"]
    lens, since, table = s["lens"].long(), s["since"].long(), s["table"].long()
    j = torch.arange(MB, device=DEV)
    held = j < ((lens + BS - 1) // BS)[:, None]
    b, blk = (held & (j >= (since // BS)[:, None])).nonzero(as_tuple=True)
    ids = table[b, blk]
    key = _values(s["cache"], c, ids)[..., 0, :]
    dead = (blk[:, None] * BS + torch.arange(BS, device=DEV) >= lens[b][:, None])[..., None, None]
    s["summaries"][ids] = torch.stack([_outward(key.masked_fill(dead, float("-inf")).amax(1), True),
                                       _outward(key.masked_fill(dead, float("inf")).amin(1), False)], 2)
    q = s["q"].float().view(B, Hk, QG, D) * D ** -0.5
    x = s["summaries"][table.clamp(min=0)].float().permute(0, 2, 3, 4, 1)           # [B][Hk][2][D][MB]
    bound = q.clamp(min=0) @ x[:, :, 0] + q.clamp(max=0) @ x[:, :, 1]
    s["scores"] = torch.where(held[:, None], bound.amax(2), s["scores"])
    return s["scores"], s["summaries"]


def _select_plain(s):
    c = s["c"]
    MB, K, BS, B, Hk = c["MB"], c["K"], c["BS"], c["B"], c["Hk"]
    lens, table = s["lens"].long(), s["table"].long()
    j = torch.arange(MB, device=DEV)
    nb = ((lens + BS - 1) // BS)[:, None, None]
    key = torch.where((j < c["first"]) | (j >= nb - c["last"]), float("inf"), s["scores"])
    key = torch.where(j < nb, key, float("-inf"))
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    if MB < K:
        order = torch.cat([order, torch.arange(MB, K, device=DEV).expand(B, Hk, -1)], -1)
    big = MB + K
    blocks = torch.where(order < nb, order, big).sort(-1).values
    some = blocks < big
    phys = table[:, None].expand(-1, Hk, -1).gather(2, torch.where(some, blocks, 0))
    tokens = torch.where(some, (lens[:, None, None] - blocks * BS).clamp(max=BS), 0).sum(-1)
    i32 = torch.int32
    return torch.where(some, phys, -1).to(i32), tokens.to(i32), torch.where(some, blocks, -1).to(i32)


def _attend_plain(s):
    c = s["c"]
    B, Hk, QG, K, BS = c["B"], c["Hk"], c["QG"], c["K"], c["BS"]
    q = s["q"].float().view(B, Hk, QG, D) * D ** -0.5
    cbb, tok = _block_bytes(c), 4 * D if c["kv"] == "bf16" else 2 * D
    blocks = s["cache"].view(-1, cbb)
    heads, t = torch.arange(Hk, device=DEV)[:, None], s["sel_table"].long()
    rows = blocks[:, :BS * Hk * tok].unflatten(1, (BS, Hk, tok)).transpose(1, 2)[t, heads]      # [B][Hk][K][BS][tok]
    if c["kv"] == "bf16":
        kv = rows.contiguous().view(torch.bfloat16).float()
    else:
        scale = blocks[:, BS * Hk * tok:].unflatten(1, (Hk, 2 * BS * 4))[t, heads].contiguous().view(torch.float32)
        kv = rows.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (2, D))
        kv = (kv * scale.unflatten(-1, (2, BS)).transpose(-1, -2)[..., None]).flatten(-2)
    kv = kv.flatten(2, 3).unflatten(-1, (2, D))
    dead = torch.arange(K * BS, device=DEV) >= s["sel_lens"].long()[..., None, None]
    _, total, o = _parts((q @ kv[..., 0, :].transpose(-1, -2)).masked_fill(dead, float("-inf")), kv[..., 1, :])
    return (o / torch.where(total > 0, total, 1.0)).reshape(B, Hk * QG, D).to(torch.bfloat16)


PLAIN = {"fork": _fork_plain, "compact": _compact_plain, "shared": _shared_plain, "score": _score_plain,
         "select": _select_plain, "attend": _attend_plain}


# ---------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        pda, p = s["pda"], s["p"]
        if op == "fork":
            pda.fork_sequences(p, s["cache"], c["NB"], s["table"], s["lens"], s["refs"], s["parents"], s["out_table"],
                               s["out_lens"], s["out_refs"], s["ws"], new_tokens=s["grow"])
            cache = s["cache"].view(torch.bfloat16) if c["kv"] == "bf16" else s["cache"]
            return cache, s["out_table"], s["out_lens"], s["out_refs"]
        if op == "copy":
            pda.copy_blocks(p, s["src"], c["NB"], s["dst"], c["NB"], s["pairs"])
            return s["dst"].view(torch.bfloat16) if c["kv"] == "bf16" else s["dst"]
        if op == "compact":
            pda.compact_blocks(p, s["cache"], c["NB"], s["table"], s["lens"], s["refs"], s["out_table"], s["out_refs"],
                               s["remap"], s["num_used"], s["ws"])
            cache = s["cache"].view(torch.bfloat16) if c["kv"] == "bf16" else s["cache"]
            return cache, s["out_table"], s["out_refs"], s["remap"], s["num_used"]
        if op == "shared":
            return pda.decode_shared(s["pp"], p, s["q"], s["cache"], s["NB"], s["starts"], s["ptable"], s["plens"],
                                     s["table"], s["lens"], s["ws"], s["out"])
        if op == "score":
            pda.summarize_blocks(p, s["cache"], s["NB"], s["table"], s["lens"], s["summaries"], since=s["since"])
            pda.score_blocks(p, s["q"], s["summaries"], s["NB"], s["table"], s["lens"], s["scores"])
            return s["scores"], s["summaries"]
        if op == "select":
            pda.select_blocks(p, s["scores"], s["table"], s["lens"], c["K"], c["first"], c["last"], s["sel_table"],
                              s["sel_lens"], sel_blocks=s["sel_blocks"])
            return s["sel_table"], s["sel_lens"], s["sel_blocks"]
        return pda.decode_selected(p, s["q"], s["cache"], c["NB"], s["sel_table"], s["sel_lens"], ws=s["ws"], out=s["out"])
    if op == "copy":
        pairs = s["pairs"].long()
        s["dst"].view(c["NB"], -1)[pairs[:, 1]] = s["src"].view(c["NB"], -1)[pairs[:, 0]]
        return s["dst"].view(torch.bfloat16) if c["kv"] == "bf16" else s["dst"]
    return PLAIN[op](s)


# ---------------------------------------------------------------------------- exact
def _rows64(cache, c, ids, h):
    """K and V of one head of the blocks `ids` in 64 bits, token by token: [n * BS][D] each."""
    BS, Hk = c["BS"], c["Hk"]
    blocks = cache.view(-1, _block_bytes(c))[ids]
    if c["kv"] == "bf16":
        x = blocks.view(torch.bfloat16).view(len(ids), BS, Hk, 2, D)[:, :, h].double()
    else:
        n = BS * Hk * 2 * D
        x = blocks[:, :n].contiguous().view(torch.float8_e4m3fn).view(len(ids), BS, Hk, 2, D)[:, :, h].double()
        x = x * blocks[:, n:].contiguous().view(torch.float32).view(len(ids), Hk, 2, BS)[:, h].transpose(1, 2)[..., None].double()
    x = x.reshape(-1, 2, D)
    return x[:, 0], x[:, 1]


def exact(case, seed):
    c = dict(case)
    op, BS, Hk = c["op"], c["BS"], c["Hk"]
    s = prepare(case, seed)
    if op == "copy":
        src, dst = s["src"].view(c["NB"], -1), s["dst"].view(c["NB"], -1)
        for a, b in s["pairs"].tolist():
            dst[b] = src[a]
        return s["dst"].view(torch.bfloat16).double() if c["kv"] == "bf16" else None
    if op == "fork":     # block by block, on the host's lists
        if c["kv"] != "bf16":
            return None
        table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
        free, seen = [i for i, r in enumerate(refs) if r == 0], set()
        blocks, at = s["cache"].view(c["NB"], -1), 0
        for p, g in zip(s["parents"].tolist(), s["grow"].tolist()):
            if lens[p] + g > c["MB"] * BS:
                continue
            last = table[p][lens[p] // BS] if lens[p] % BS else None
            moved = last is not None and (p in seen or refs[last] != 1)
            seen.add(p)
            need = int(moved) + -(-(lens[p] + g) // BS) - -(-lens[p] // BS)
            if moved and at + need <= len(free):
                blocks[free[at]] = blocks[last]
            at += need
        return s["cache"].view(torch.bfloat16).double(), None, None, None
    if op == "compact":
        if c["kv"] != "bf16":
            return None
        refs = s["refs"].tolist()
        U = sum(r > 0 for r in refs)
        blocks = s["cache"].view(c["NB"], -1)
        for a, b in zip([i for i in range(U, c["NB"]) if refs[i] > 0], [i for i in range(U) if refs[i] == 0]):
            blocks[b] = blocks[a]
        return s["cache"].view(torch.bfloat16).double(), None, None, None, None
    if op == "select":
        return None      # whole numbers only
    QG, B = c["QG"], c["B"]
    if op == "shared":
        out = torch.zeros(B, Hk, QG, D, dtype=torch.float64, device=DEV)
        starts = _group_starts(c)
        plens, lens = s["plens"].tolist(), s["lens"].tolist()
        for g in range(c["NG"]):
            for h in range(Hk):
                kp, vp = _rows64(s["cache"], c, s["ptable"][g, :-(-plens[g] // BS)].long(), h)
                for b in range(starts[g], starts[g + 1]):
                    ko, vo = _rows64(s["cache"], c, s["table"][b, :-(-lens[b] // BS)].long(), h)
                    k = torch.cat([kp[:plens[g]], ko[:lens[b]]])
                    if len(k):
                        w = torch.softmax(s["q"][b, h * QG:(h + 1) * QG].double() @ k.T / math.sqrt(D), -1)
                        out[b, h] = w @ torch.cat([vp[:plens[g]], vo[:lens[b]]])
        return out.view(B, Hk * QG, D)
    if op == "attend":
        out = torch.zeros(B, Hk, QG, D, dtype=torch.float64, device=DEV)
        lens = s["sel_lens"].tolist()
        for b in range(B):
            for h in range(Hk):
                k, v = _rows64(s["cache"], c, s["sel_table"][b, h].long(), h)
                w = torch.softmax(s["q"][b, h * QG:(h + 1) * QG].double() @ k[:lens[b][h]].T / math.sqrt(D), -1)
                out[b, h] = w @ v[:lens[b][h]]
        return out.view(B, Hk * QG, D)
    # score: summaries renewed by definition, then the bounds; the old summaries stay as they are
    lens, since, table = s["lens"].tolist(), s["since"].tolist(), s["table"].tolist()
    summ = s["summaries"].double()
    scores = torch.zeros(B, Hk, c["MB"], dtype=torch.float64, device=DEV)
    for b in range(B):
        n = -(-lens[b] // BS)
        for j in range(since[b] // BS, n):
            if n - since[b] // BS > 40:
                return None
            for h in range(Hk):
                k, _ = _rows64(s["cache"], c, s["table"][b, j:j + 1].long(), h)
                k = k[:lens[b] - j * BS]
                summ[table[b][j], h, 0] = _outward(k.amax(0).float(), True).double()
                summ[table[b][j], h, 1] = _outward(k.amin(0).float(), False).double()
        if n:
            q = s["q"][b].double().view(Hk, QG, D) / math.sqrt(D)
            x = summ[s["table"][b, :n].long()]
            up = torch.einsum("hqd,nhd->hqn", q.clamp(min=0), x[:, :, 0]) + torch.einsum("hqd,nhd->hqn", q.clamp(max=0), x[:, :, 1])
            scores[b, :, :n] = up.amax(1)
    return scores, summ
