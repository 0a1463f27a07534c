"""Speculative decoding on the paged KV cache, in its plain form and through the library.

Groups of operators, each a pass of `run`:
  write   K and V of many new tokens per sequence are stored in the cache's format: write_kv
  read    tokens of the cache are gathered and dequantised: read_kv
  trip    written in 4 bits and read back: write_kv, read_kv
  tree    a step for a tree (or chain) of drafted tokens per sequence over its cache: decode_tree
  accept  the accepted path of every tree moves to consecutive positions: accept_tokens
  window  a decode step over a sliding window and a few first tokens: decode_window

Cache block: [BS slots][Hk heads][K | V][128] elements, bf16, e4m3 or 4-bit codes (TQ4, two to a byte); then for e4m3
fp32 scales [Hk][K, V][BS], for TQ4 fp16 [Hk][k_norm, v_scale, v_zero][BS].  Lengths are a fixed spread of each case's
range; the seed shuffles them.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
TOKEN_BYTES = {"bf16": 4 * D, "fp8": 2 * D, "tq4": D}     # K and V of one token and head
META_BYTES = {"bf16": 0, "fp8": 8, "tq4": 6}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the drafted tokens of eight sequences enter the cache, as rows of one fused projection: latency
        dict(name="write_b8_drafts_fp8", op="write", B=8, Hk=8, QG=8, BS=16, kv="fp8", lo=100, hi=4000, tlo=1, thi=9),
        # sixteen prompts of all lengths, some behind a cached prefix
        dict(name="write_b16_prompts_fp8", op="write", B=16, Hk=8, QG=6, BS=16, kv="fp8", lo=0, hi=1000, tlo=16, thi=4096),
        # contexts of a batch are read back, to be sent elsewhere
        dict(name="read_b16_ctx8192_fp8", op="read", B=16, Hk=4, BS=32, kv="fp8", lo=0, hi=0, tlo=2048, thi=8192),
        # prompts into a 4-bit cache and back, as a check of the codebook does
        dict(name="trip_b8_tq4", op="trip", B=8, Hk=8, QG=6, BS=16, kv="tq4", lo=0, hi=300, tlo=16, thi=2048),
        # one short text, a chain of four drafted tokens: latency
        dict(name="tree_b1_t4_ctx250", op="tree", B=1, Hk=1, QG=8, BS=16, kv="bf16", lo=250, hi=250, tlo=4, thi=4, tree=False,
             window=0, first=0),
        # a medium batch with trees of up to 33 drafted tokens
        dict(name="tree_b32_t33", op="tree", B=32, Hk=4, QG=16, BS=32, kv="bf16", lo=2048, hi=8192, tlo=9, thi=33, tree=True,
             window=0, first=0),
        # a full fp8 batch, few drafted tokens each, contexts over the whole range, window and sinks
        dict(name="tree_b64_t6_window_fp8", op="tree", B=64, Hk=8, QG=6, BS=16, kv="fp8", lo=16, hi=16384, tlo=1, thi=6, tree=True,
             window=4096, first=4),
        # long contexts, wide trees
        dict(name="tree_b4_t64_ctx32768", op="tree", B=4, Hk=8, QG=8, BS=32, kv="bf16", lo=32768, hi=32768, tlo=64, thi=64,
             tree=True, window=0, first=0),
        # the paths of eight small trees
        dict(name="accept_b8_t9", op="accept", B=8, Hk=8, BS=16, kv="bf16", lo=100, hi=4000, tlo=5, thi=9),
        # the paths of a full fp8 batch of wide trees
        dict(name="accept_b128_t64_fp8", op="accept", B=128, Hk=8, BS=16, kv="fp8", lo=1, hi=2000, tlo=33, thi=64),
        # four long contexts, of which a step sees the last thousand tokens and four sinks
        dict(name="window_b4_w1024", op="window", B=4, Hk=8, QG=8, BS=32, kv="bf16", lo=30001, hi=32768, window=1024, first=4),
        # a full fp8 batch, contexts shorter and longer than the window
        dict(name="window_b64_w4096_fp8", op="window", B=64, Hk=8, QG=6, BS=16, kv="fp8", lo=500, hi=16384, window=4096, first=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "trip", "tree", "tree", "tree", "accept", "window", "window"])
    kv = rng.choice(["bf16", "fp8", "tq4"])
    BS, Hk, QG = rng.choice([16, 32]), rng.choice([1, 2, 4, 5, 8]), rng.choice([6, 8, 16])
    if op in ("write", "read", "trip"):
        if op == "write" and kv == "tq4":
            kv = "fp8"
        if op == "trip":
            kv = "tq4"
        thi = _log(rng, 1, 4096)
        hi = _log(rng, 1, 2000)
        B = _log(rng, 1, max(1, min(32, 40000 // thi)))
        return dict(op=op, B=B, Hk=Hk, QG=QG, BS=BS, kv=kv, lo=rng.randint(0, hi), hi=hi, tlo=rng.randint(0, thi), thi=thi)
    if op == "accept":
        thi = _log(rng, 1, 64)
        hi = _log(rng, 1, 3000)
        return dict(op=op, B=_log(rng, 1, 64), Hk=Hk, BS=BS, kv=kv, lo=rng.randint(0, hi), hi=hi, tlo=rng.randint(1, thi), thi=thi)
    hi = _log(rng, 100, 30000)
    B = _log(rng, 1, max(1, min(48, 120000 // hi)))
    lo = rng.randint(0, hi)
    window, first = _log(rng, 16, 8192), rng.choice([0, 1, 4, 4, 70])
    if op == "window":
        return dict(op=op, B=B, Hk=Hk, QG=QG, BS=BS, kv=kv, lo=lo, hi=hi, window=window, first=first)
    thi = _log(rng, 1, 64)
    if rng.random() < 0.5:
        window = first = 0
    return dict(op=op, B=B, Hk=Hk, QG=QG, BS=BS, kv=kv, lo=lo, hi=hi, tlo=rng.randint(1, thi), thi=thi,
                tree=rng.choice([True, True, False]), window=window, first=first)


# ---------------------------------------------------------------------------- sizes
def _block_bytes(c):
    return c["BS"] * c["Hk"] * (TOKEN_BYTES[c["kv"]] + META_BYTES[c["kv"]])


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm where the range is wide."""
    if n == 1:
        return [hi]
    if hi > 10 * max(lo, 1):
        a, b = math.log(lo + 1), math.log(hi + 1)
        return [int(round(math.exp(a + (b - a) * i / (n - 1)) - 1)) for i in range(n)]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def work(case):
    c = case
    tok = c["Hk"] * (TOKEN_BYTES[c["kv"]] + META_BYTES[c["kv"]])
    plain = c["Hk"] * 4 * D
    lens = _spread(c["B"], c["lo"], c["hi"])
    if c["op"] == "window":
        seen = sum(min(x, c["window"] + c["first"]) for x in lens)
        rows = c["B"] * c["Hk"] * c["QG"]
        return {"bytes": seen * tok + rows * D * 4.0, "flops": 4.0 * D * seen * c["Hk"] * c["QG"]}
    counts = _spread(c["B"], c["tlo"], c["thi"])
    n = sum(counts)
    if c["op"] in ("write", "read"):
        return {"bytes": float(n * (tok + plain)), "flops": 0.0}
    if c["op"] == "trip":
        return {"bytes": float(n * 2 * (tok + plain)), "flops": 0.0}
    if c["op"] == "accept":     # about a path of log2 of the tree's size
        return {"bytes": float(sum(max(1.0, math.log2(x + 1)) for x in counts) * tok * 2), "flops": 0.0}
    seen = [min(x, c["window"] + c["first"]) if c["window"] else x for x in lens]
    seen, mean = sum(seen), sum(seen) / c["B"]
    rows = n * c["Hk"] * c["QG"]
    return {"bytes": (seen + n) * tok + rows * D * 4.0, "flops": 4.0 * D * rows * mean}


# ---------------------------------------------------------------------------- inputs
def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _codebook():
    """16 centroids of N(0, 1/D): its quantiles at (j + 1/2) / 16."""
    p = (torch.arange(16, dtype=torch.float64) + 0.5) / 16.0
    return (torch.special.ndtri(p) / math.sqrt(D)).float().to(DEV)


def _fields(cache, c):
    """Views of the cache: data [NB][BS][Hk][2][bytes] and meta [NB][Hk][fields][BS] (None for bf16)."""
    BS, Hk, n = c["BS"], c["Hk"], c["BS"] * c["Hk"] * TOKEN_BYTES[c["kv"]]
    blocks = cache.view(-1, _block_bytes(c))
    data = blocks[:, :n].unflatten(1, (BS, Hk, 2, TOKEN_BYTES[c["kv"]] // 2))
    if c["kv"] == "bf16":
        return data, None
    if c["kv"] == "fp8":
        return data, blocks[:, n:].view(torch.float32).unflatten(1, (Hk, 2, BS))
    return data, blocks[:, n:].view(torch.float16).unflatten(1, (Hk, 3, BS))


def _make_cache(c, gen, NB):
    """A pool of NB blocks with N(0, 1) keys and values (keys of a head share an offset), uint8."""
    BS, Hk = c["BS"], c["Hk"]
    cache = torch.zeros(NB, _block_bytes(c), dtype=torch.uint8, device=DEV)
    bias = torch.randn(Hk, 2, D, generator=gen, device=DEV) * torch.tensor([0.5, 0.0], device=DEV)[:, None]
    step = max(1, (1 << 26) // (BS * Hk * 2 * D))
    for i in range(0, NB, step):
        n = min(step, NB - i)
        data, meta = _fields(cache[i:i + n].view(-1), c)
        x = torch.randn(n, BS, Hk, 2, D, generator=gen, device=DEV) + bias
        if c["kv"] == "bf16":
            data.view(torch.bfloat16).copy_(x)
        elif c["kv"] == "fp8":
            scale = x.abs().amax(-1) / 448.0
            data.copy_((x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))
            meta.copy_(scale.permute(0, 2, 3, 1))
        else:
            norm, vmin, vmax = x[..., 0, :].norm(dim=-1).half(), x[..., 1, :].amin(-1), x[..., 1, :].amax(-1)
            book = _codebook()
            k = torch.bucketize(x[..., 0, :] / norm.float()[..., None], (book[1:] + book[:-1]) / 2)
            zero, scale = vmin.half(), ((vmax - vmin) / 15).half()
            v = ((x[..., 1, :] - zero.float()[..., None]) / scale.float()[..., None]).round().clamp(0, 15)
            code = torch.stack([k, v.long()], -2).to(torch.uint8)
            data.copy_(code[..., 0::2] | code[..., 1::2] << 4)
            meta.copy_(torch.stack([norm, scale, zero], 2).permute(0, 3, 2, 1))
    return cache.view(-1)


def _shuffled(rs, B, lo, hi):
    x = np.array(_spread(B, lo, hi), np.int64)
    rs.shuffle(x)
    return x


def _drafted(rs, counts, tree):
    """Masks [N][words] of random trees (each token below one of the last few, or below the root) and the longest path of
    each as indices."""
    words = max(1, -(-int(counts.max()) // 64))
    masks, paths = [], []
    for n in counts.tolist():
        seen, depth = [], []
        for j in range(n):
            up = j - 1 if not tree else int(rs.randint(max(-1, j - 1 - n // 3), j)) if j else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << j)
            depth.append(depth[up] + 1 if up >= 0 else 1)
        masks += [[(m >> 64 * w) & (1 << 64) - 1 for w in range(words)] for m in seen]
        end = int(np.argmax(depth)) if n else -1
        paths.append([j for j in range(n) if end >= 0 and seen[end] >> j & 1])
    return np.array(masks, np.uint64).reshape(-1, words), paths


KV = {"bf16": 0, "fp8": 1, "tq4": 2}


def prepare(case, seed):
    c = dict(case)
    op, B, Hk, BS = c["op"], c["B"], c["Hk"], c["BS"]
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    bf = torch.bfloat16
    lens = _shuffled(rs, B, c["lo"], c["hi"])
    counts = np.ones(B, np.int64) if op == "window" else _shuffled(rs, B, c["tlo"], c["thi"])
    total = lens if op == "window" else lens + counts
    blocks = -(-total // BS)
    # the same for every seed: sequences take their blocks from the pool whichever lengths come together
    MB = max(1, -(-int(lens.max() + (0 if op == "window" else counts.max())) // BS))
    NB = int((-(-lens // BS)).sum() + (0 if op == "window" else (-(-counts // BS)).sum())) + 16
    ids, table, at = rs.permutation(NB), np.full((B, MB), -1, np.int64), 0
    for b in range(B):
        table[b, :blocks[b]] = ids[at:at + blocks[b]]
        at += blocks[b]
    starts = np.concatenate([[0], np.cumsum(counts)])
    N = int(starts[-1])
    s = dict(c=c, cache=_make_cache(c, gen, NB), NB=NB, MB=MB, N=N, table=_i32(table), lens=_i32(lens), starts=_i32(starts),
             book=_codebook() if c["kv"] == "tq4" else None)
    if op in ("write", "trip"):     # K and V as they leave a fused projection, behind the query heads
        qkv = torch.randn(N, Hk * (c["QG"] + 2), D, generator=gen, device=DEV).to(bf)
        s.update(k=qkv[:, Hk * c["QG"]:Hk * (c["QG"] + 1)], v=qkv[:, Hk * (c["QG"] + 1):])
    if op in ("read", "trip"):
        s.update(k_out=torch.zeros(N, Hk, D, dtype=bf, device=DEV), v_out=torch.zeros(N, Hk, D, dtype=bf, device=DEV))
    if op == "tree":
        masks, _ = _drafted(rs, counts, c["tree"])
        s["q"] = torch.randn(N, Hk * c["QG"], D, generator=gen, device=DEV).to(bf)
        s["out"] = torch.zeros_like(s["q"])
        s["masks"] = torch.from_numpy(masks.view(np.int64)).to(DEV) if c["tree"] else None
    if op == "accept":
        _, paths = _drafted(rs, counts, True)
        A = max(1, max(len(p) for p in paths))
        s.update(path=_i32([p + [-1] * (A - len(p)) for p in paths]), path_lens=_i32([len(p) for p in paths]),
                 out_lens=_i32(np.zeros(B)), A=A)
    if op == "window":
        s["q"] = torch.randn(B, Hk * c["QG"], D, generator=gen, device=DEV).to(bf)
        s["out"] = torch.zeros_like(s["q"])
    if own:
        import paged_kv_gqa_block_gb300 as pda
        s["pda"] = pda
        s["p"] = pda.plan(B, Hk, c.get("QG", 8), BS, MB, kv_dtype=KV[c["kv"]])
        if op == "tree":
            s["ws"] = pda.tree_workspace(s["p"], N, DEV)
    return s


# ---------------------------------------------------------------------------- plain forms
def _decoded(data, meta, kv, book):
    """fp32 K and V [..., 2, D] of token rows: data [..., 2, bytes], meta [..., fields]."""
    if kv == "bf16":
        return data.contiguous().view(torch.bfloat16).float()
    if kv == "fp8":
        return data.contiguous().view(torch.float8_e4m3fn).float() * meta[..., None]
    code = torch.stack([data & 15, data >> 4], -1).flatten(-2).long()
    m = meta.float()[..., None]
    return torch.stack([book[code[..., 0, :]] * m[..., 0, :], code[..., 1, :] * m[..., 1, :] + m[..., 2, :]], -2)


def _places(s, pos):
    """Block ids and slots of positions [B][n] (those of unused entries: block 0)."""
    BS = s["c"]["BS"]
    blk = s["table"].long().gather(1, (pos // BS).clamp(0, s["MB"] - 1)).clamp(min=0)
    return blk, pos % BS


def _token_places(s):
    """Block and slot of every token of the step: token i of sequence b is at lens[b] + i - starts[b]."""
    i = torch.arange(s["N"], device=DEV)
    starts = s["starts"].long()
    b = (i[:, None] >= starts[None, 1:]).sum(1)
    pos = s["lens"].long()[b] + i - starts[b]
    blk = s["table"].long()[b, pos // s["c"]["BS"]]
    return blk, pos % s["c"]["BS"]


def _written(s):
    """The pool, as its values' types."""
    data, meta = _fields(s["cache"], s["c"])
    return (data.view(torch.bfloat16),) if meta is None else (data.view(torch.float8_e4m3fn), meta)


def _write_plain(s):
    c = s["c"]
    data, meta = _fields(s["cache"], c)
    blk, slot = _token_places(s)
    x = torch.stack([s["k"], s["v"]], 2)                                  # [N][Hk][2][D]
    if c["kv"] == "bf16":
        data.view(torch.bfloat16)[blk, slot] = x
        return
    x = x.float()
    if c["kv"] == "fp8":
        top = x.abs().amax(-1)
        scale = torch.where(top > 0, top / torch.full_like(top, 448.0), 1.0)      # by a number would multiply by its inverse
        data[blk, slot] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        meta[blk, :, :, slot] = scale
        return
    k, v = x[:, :, 0], x[:, :, 1]
    norm = k.double().square().sum(-1).sqrt().to(torch.float16)
    mid = (s["book"][1:] + s["book"][:-1]) / 2
    kc = torch.bucketize(k / torch.where(norm > 0, norm, 1.0).float()[..., None], mid)     # how many midpoints are below
    zero = v.amin(-1).to(torch.float16)
    span = v.amax(-1) - v.amin(-1)
    scale = (span / torch.full_like(span, 15.0)).to(torch.float16)
    vc = ((v - zero.float()[..., None]) / torch.where(scale > 0, scale, 1.0).float()[..., None]).round().clamp(0, 15)
    code = torch.stack([kc, vc.long()], 2).to(torch.uint8)
    data[blk, slot] = code[..., 0::2] | code[..., 1::2] << 4
    meta[blk, :, :, slot] = torch.stack([norm, scale, zero], -1)


def _read_plain(s):
    c = s["c"]
    data, meta = _fields(s["cache"], c)
    blk, slot = _token_places(s)
    x = _decoded(data[blk, slot], None if meta is None else meta[blk, :, :, slot], c["kv"], s["book"])
    return x[:, :, 0].to(torch.bfloat16), x[:, :, 1].to(torch.bfloat16)


def _context(s, n):
    """fp32 K and V [B][Hk][2][n][D] of the first n positions."""
    c = s["c"]
    data, meta = _fields(s["cache"], c)
    blk, slot = _places(s, torch.arange(n, device=DEV).expand(c["B"], n))
    x = _decoded(data[blk, slot], None if meta is None else meta[blk, :, :, slot], c["kv"], s["book"])
    return x.permute(0, 2, 3, 1, 4)


def _attend(q, kv, hidden):
    """Softmax attention of q [B][Hk][rows][D] over kv [B][Hk][2][n][D]; rows that see nothing give 0."""
    logits = (q @ kv[:, :, 0].transpose(-1, -2) * D ** -0.5).masked_fill_(hidden, float("-inf"))
    e = torch.exp(logits - logits.amax(-1, keepdim=True).clamp(min=-3e38))
    total = e.sum(-1, keepdim=True)
    return e @ kv[:, :, 1] / torch.where(total > 0, total, 1.0)


def _tree_plain(s):
    c = s["c"]
    B, Hk, QG, T = c["B"], c["Hk"], c["QG"], c["thi"]
    n = s["MB"] * c["BS"]
    lens, starts = s["lens"].long(), s["starts"].long()
    count = starts[1:] - starts[:-1]
    i, t = torch.arange(T, device=DEV), torch.arange(n, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=s["N"] - 1)                    # [B][T]
    live = i < count[:, None]
    if s["masks"] is None:
        sees = (i[:, None] >= i)[None].expand(B, T, T)
    else:
        bit = torch.arange(64, device=DEV)
        sees = (s["masks"][row][..., None] >> bit & 1).bool().flatten(2)
        sees = torch.cat([sees, torch.zeros(B, T, max(0, T - sees.shape[2]), dtype=torch.bool, device=DEV)], 2)[..., :T]
    sees = sees & live[:, None]
    j = t - lens[:, None]                                                  # [B][n]: index among the drafted
    drafted = (j >= 0) & (j < count[:, None])
    seen = drafted[:, None] & sees.gather(2, j.clamp(0, T - 1)[:, None].expand(B, T, n))
    old = (t < lens[:, None])[:, None].expand(B, T, n)
    if c["window"]:
        others = sees & (i[:, None] != i)
        pos = lens[:, None] + (others.sum(2) if s["masks"] is not None else i)
        old = old & ((t < c["first"]) | (pos[..., None] - t < c["window"]))
        if s["masks"] is None:
            seen = seen & ((t < c["first"]) | (pos[..., None] - t < c["window"]))
    hidden = ~(old | seen) | ~live[..., None]                              # [B][T][n]
    q = s["q"].float().view(-1, Hk, QG, D)[row].permute(0, 2, 1, 3, 4).reshape(B, Hk, T * QG, D)
    o = _attend(q, _context(s, n), hidden.repeat_interleave(QG, 1)[:, None])
    o = o.view(B, Hk, T, QG, D).permute(0, 2, 1, 3, 4)[live]               # in the order of the rows
    return o.reshape(s["N"], Hk * QG, D).to(torch.bfloat16)


def _window_plain(s):
    c = s["c"]
    n = s["MB"] * c["BS"]
    t, lens = torch.arange(n, device=DEV), s["lens"].long()[:, None]
    hidden = (t >= lens) | ((t >= c["first"]) & (lens - 1 - t >= c["window"]))
    q = s["q"].float().view(c["B"], c["Hk"], c["QG"], D)
    return _attend(q, _context(s, n), hidden[:, None, None]).reshape(c["B"], -1, D).to(torch.bfloat16)


def _accept_plain(s):
    c = s["c"]
    data, meta = _fields(s["cache"], c)
    k = torch.arange(s["A"], device=DEV).expand(c["B"], -1)
    keep = k < s["path_lens"][:, None]
    lens = s["lens"].long()[:, None]
    src, dst = _places(s, lens + s["path"].long().clamp(min=0)), _places(s, lens + k)
    (b0, s0), (b1, s1) = [(x[keep], y[keep]) for x, y in (src, dst)]
    data[b1, s1] = data[b0, s0]
    if meta is not None:
        meta[b1, :, :, s1] = meta[b0, :, :, s0]
    return s["lens"] + s["path_lens"]


def _pool(s):
    """The pool as its values' types, 4-bit codes one by one."""
    data, meta = _fields(s["cache"], s["c"])
    if s["c"]["kv"] == "tq4":
        return torch.stack([data & 15, data >> 4], -1), meta
    return _written(s)


# ---------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        pda, p = s["pda"], s["p"]
        if op in ("write", "trip"):
            pda.write_kv(p, s["k"], s["v"], s["cache"], s["NB"], s["table"], s["starts"], s["lens"], centroids=s["book"])
        if op in ("read", "trip"):
            pda.read_kv(p, s["cache"], s["NB"], s["table"], s["starts"], s["lens"], s["k_out"], s["v_out"],
                        centroids=s["book"])
            return s["k_out"], s["v_out"]
        if op == "write":
            return _written(s)
        if op == "tree":
            return pda.decode_tree(p, s["q"], s["cache"], s["NB"], s["table"], s["lens"], s["starts"], tree_masks=s["masks"],
                                   window=c["window"], num_first=c["first"], centroids=s["book"], ws=s["ws"], out=s["out"])
        if op == "accept":
            pda.accept_tokens(p, s["cache"], s["NB"], s["table"], s["lens"], s["path"], s["path_lens"], s["out_lens"])
            return (*_pool(s), s["out_lens"])
        return pda.decode_window(p, s["q"], s["cache"], s["NB"], s["table"], s["lens"], c["window"], num_first=c["first"],
                                 centroids=s["book"], out=s["out"])
    if op in ("write", "trip"):
        _write_plain(s)
    if op in ("read", "trip"):
        return _read_plain(s)
    if op == "write":
        return _written(s)
    if op == "accept":
        lens = _accept_plain(s)
        return (*_pool(s), lens)
    return _tree_plain(s) if op == "tree" else _window_plain(s)


# ---------------------------------------------------------------------------- exact
def _rows64(s, b, h, n):
    """K and V of one head of the first n positions of a sequence, in 64 bits: [n][D] each."""
    c = s["c"]
    BS, Hk, size = c["BS"], c["Hk"], TOKEN_BYTES[c["kv"]]
    ids = s["table"][b, :-(-n // BS)].long()
    blocks = s["cache"].view(s["NB"], -1)[ids]
    raw = blocks[:, :BS * Hk * size].reshape(len(ids), BS, Hk, size)[:, :, h].contiguous()
    rest = blocks[:, BS * Hk * size:].contiguous()
    if c["kv"] == "bf16":
        k, v = raw.view(torch.bfloat16).double().split(D, -1)
    elif c["kv"] == "fp8":
        m = rest.view(torch.float32).view(len(ids), Hk, 2, BS)[:, h].double()
        k, v = raw.view(torch.float8_e4m3fn).double().split(D, -1)
        k, v = k * m[:, 0, :, None], v * m[:, 1, :, None]
    else:
        m = rest.view(torch.float16).view(len(ids), Hk, 3, BS)[:, h].double()
        code = torch.zeros(len(ids), BS, 2 * D, dtype=torch.long, device=DEV)
        code[..., 0::2], code[..., 1::2] = raw.long() % 16, raw.long() // 16
        k = s["book"].double()[code[..., :D]] * m[:, 0, :, None]
        v = code[..., D:].double() * m[:, 1, :, None] + m[:, 2, :, None]
    return k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]


def _pool64(s):
    return tuple(x.double() if x.is_floating_point() else None for x in _pool(s))


def exact(case, seed):
    c = dict(case)
    op, B, Hk, BS = c["op"], c["B"], c["Hk"], c["BS"]
    s = prepare(case, seed)
    lens, starts, table = s["lens"].tolist(), s["starts"].tolist(), s["table"].tolist()
    if op in ("write", "trip"):
        blocks = s["cache"].view(s["NB"], -1)
        size = TOKEN_BYTES[c["kv"]]
        trip = torch.zeros(2, s["N"], Hk, D, dtype=torch.float64, device=DEV)
        pool = None if op == "trip" else [x.double().clone() for x in _written(s)]
        for b in range(B):
            n = starts[b + 1] - starts[b]
            if n == 0:
                continue
            at = torch.arange(lens[b], lens[b] + n, device=DEV)
            ids, slots = s["table"][b].long()[at // BS], at % BS
            for w, x in enumerate((s["k"], s["v"])):
                x = x[starts[b]:starts[b + 1]].double()
                if c["kv"] == "bf16":
                    pool[0][ids, slots, :, w] = x
                elif c["kv"] == "fp8":      # quotients are rounded to 32 bits first: that is the format's definition
                    scale = (x.abs().max(-1).values / 448.0).float().double()
                    scale[scale == 0] = 1.0
                    pool[0][ids, slots, :, w] = (x / scale[..., None]).float().to(torch.float8_e4m3fn).double()
                    pool[1][ids, :, w, slots] = scale
                elif w == 0:
                    norm = x.pow(2).sum(-1).sqrt().half().double()
                    unit = (x / torch.where(norm > 0, norm, torch.ones_like(norm))[..., None]).float()
                    near = torch.zeros_like(unit, dtype=torch.long)
                    for i in range(15):
                        near += ((s["book"][i] + s["book"][i + 1]) / 2 < unit).long()
                    trip[0, starts[b]:starts[b + 1]] = s["book"].double()[near] * norm[..., None]
                else:
                    zero = x.min(-1).values.half().double()
                    step = ((x.max(-1).values - x.min(-1).values).float().double() / 15).float().half().double()
                    code = ((x - zero[..., None]).float().double() / torch.where(step > 0, step, torch.ones_like(step))[..., None])
                    trip[1, starts[b]:starts[b + 1]] = code.float().round().clamp(0, 15).double() * step[..., None] + zero[..., None]
        return (trip[0], trip[1]) if op == "trip" else tuple(pool)
    if op == "read":
        out = torch.zeros(2, s["N"], Hk, D, dtype=torch.float64, device=DEV)
        for b in range(B):
            n = starts[b + 1] - starts[b]
            for h in range(Hk if n else 0):
                k, v = _rows64(s, b, h, lens[b] + n)
                out[0, starts[b]:starts[b + 1], h], out[1, starts[b]:starts[b + 1], h] = k[lens[b]:], v[lens[b]:]
        return out[0], out[1]
    if op == "accept":
        cbb, size = _block_bytes(c), TOKEN_BYTES[c["kv"]] * Hk
        width = {"bf16": 0, "fp8": 4, "tq4": 2}[c["kv"]]
        pool = s["cache"].view(s["NB"], cbb).cpu().numpy()
        meta0 = BS * size
        path, path_lens = s["path"].tolist(), s["path_lens"].tolist()
        for b in range(B):
            for k in range(path_lens[b]):
                p, q = lens[b] + path[b][k], lens[b] + k
                x, y = pool[table[b][p // BS]], pool[table[b][q // BS]]
                y[q % BS * size:(q % BS + 1) * size] = x[p % BS * size:(p % BS + 1) * size]
                if width:
                    x, y = (z[meta0:].reshape(-1, BS, width) for z in (x, y))
                    y[:, q % BS] = x[:, p % BS]
        s["cache"].copy_(torch.from_numpy(pool).view(-1))
        return (*_pool64(s), None)
    QG = c["QG"]
    scale = 1 / math.sqrt(D)
    if op == "window":
        out = torch.zeros(B, Hk, QG, D, dtype=torch.float64, device=DEV)
        for b in range(B):
            keep = [t for t in range(lens[b]) if t < c["first"] or t > lens[b] - 1 - c["window"]]
            for h in range(Hk if keep else 0):
                k, v = _rows64(s, b, h, lens[b])
                w = torch.softmax(s["q"][b, h * QG:(h + 1) * QG].double() @ k[keep].T * scale, -1)
                out[b, h] = w @ v[keep]
        return out.view(B, Hk * QG, D)
    out = torch.zeros(s["N"], Hk, QG, D, dtype=torch.float64, device=DEV)
    masks = None if s["masks"] is None else s["masks"].cpu().numpy().view(np.uint64)
    for b in range(B):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        see = np.zeros((n, lens[b] + n), bool)
        for i in range(n):
            row = range(i + 1) if masks is None else [j for j in range(n) if int(masks[starts[b] + i, j // 64]) >> j % 64 & 1]
            at = lens[b] + (i if masks is None else sum(j != i for j in row))
            lo = at - c["window"] + 1 if c["window"] else 0
            see[i, max(0, lo):lens[b]] = True
            see[i, :min(c["first"], lens[b])] = True
            for j in row:
                if masks is not None or lens[b] + j >= lo or lens[b] + j < c["first"]:
                    see[i, lens[b] + j] = True
        blind = torch.from_numpy(~see).to(DEV).repeat_interleave(QG, 0)
        for h in range(Hk):
            k, v = _rows64(s, b, h, lens[b] + n)
            q = s["q"][starts[b]:starts[b + 1], h * QG:(h + 1) * QG].double().reshape(n * QG, D)
            w = torch.softmax((q @ k.T * scale).masked_fill(blind, float("-inf")), -1)
            out[starts[b]:starts[b + 1], h] = (w @ v).view(n, QG, D)
    return out.view(s["N"], Hk * QG, D)
