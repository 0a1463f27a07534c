"""The decode step over shared prefixes against attention over the concatenated tokens in 64 bits."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp

pytestmark = pytest.mark.gpu

BF16, FP8 = wl.KV_BF16, wl.KV_FP8_E4M3


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


class Case:
    """Groups with prefixes and sequences with tokens of their own, in one pool whose unused slots hold NaN."""

    def __init__(self, kv, Hk, QG, BS, plens, sizes, lens, seed=0, before=0, q_scale=1.0, v_spread=0.0, prefix_blocks=None, k_bias=0.0):
        rng = np.random.default_rng(seed)
        self.kv, self.Hk, self.QG, self.BS, self.plens = kv, Hk, QG, BS, list(plens)
        self.starts = [before]
        for n in sizes:
            self.starts.append(self.starts[-1] + n)
        self.lens = list(lens)
        self.B = len(self.lens)
        assert self.starts[-1] <= self.B
        self.MP = prefix_blocks or max(1, -(-max(plens) // BS))
        self.MB = max(1, -(-max(self.lens) // BS))
        need = [-(-n // BS) for n in self.plens + self.lens]
        self.NB = sum(need) + 3
        self.w = wl.Workload("shared", self.B, Hk, QG, BS, self.MB, self.NB, ("list", tuple(self.lens)), seed=0, kv_dtype=kv)
        self.cache = wl.empty_cache(self.w)
        ids, at, tables = rng.permutation(self.NB).astype(np.int32), 0, []
        for n, blocks in zip(self.plens + self.lens, need):
            row = ids[at:at + blocks]
            at += blocks
            k = rng.standard_normal((n, Hk, 128)) + k_bias
            v = rng.standard_normal((n, Hk, 128)) * np.exp(v_spread * rng.standard_normal((n, Hk, 1)))
            wl.write_tokens(self.w, self.cache, row, k.astype(np.float32), v.astype(np.float32))
            tables.append(row)
        self.ptable = np.full((len(plens), self.MP), -1, np.int32)
        self.table = np.full((self.B, self.MB), -1, np.int32)
        for g in range(len(plens)):
            self.ptable[g, :need[g]] = tables[g]
        for b in range(self.B):
            self.table[b, :need[len(plens) + b]] = tables[len(plens) + b]
        self.q = wl.round_bf16((rng.standard_normal((self.B, Hk * QG, 128)) * q_scale).astype(np.float32))

    def device(self):
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        return dict(query=torch.from_numpy(self.q.view(np.int16)).cuda().view(torch.bfloat16), kv_cache=torch.from_numpy(self.cache).cuda(),
                    num_cache_blocks=self.NB, group_starts=i32(self.starts), prefix_table=i32(self.ptable), prefix_lens=i32(self.plens),
                    block_table=i32(self.table), context_lens=i32(self.lens))

    def plans(self, pda, **kw):
        return pda.shared_plans(self.B, len(self.plens), self.Hk, self.QG, self.BS, self.MP, self.MB, kv_dtype=self.kv, **kw)

    def reference(self, scale=128 ** -0.5):
        """(out, bound) in 64 bits.  The bound: a prefix weight rounded to bf16 is off by at most 2^-8; with fp8 KV the weight, V's
        scale and the scaled V are each rounded to f16, 2^-11 each, 3 * 2^-11 per term; a logit's 128 products are summed in fp32, each addition off by at most a step (2^-23), which moves its
        weight by as much in absolute terms; ex2, the scales and the sums over T tokens each add steps of 2^-23
        per term.  The own part is the library's partition pass (P in 16 bits: 2^-16 bf16, 2^-11 fp8)."""
        K, V = pp.block_values(self.w, self.cache)
        q = wl.bf16_bits_to_f32(self.q).astype(np.float64)
        out, bound = np.zeros((self.B, self.Hk * self.QG, 128)), np.zeros((self.B, self.Hk * self.QG, 128))
        half = 2.0 ** -8 if self.kv == BF16 else 3 * 2.0 ** -11 * (1 + 2.0 ** -10)
        for b in range(self.B):
            for h in range(self.Hk):
                k, v = [], []
                for g in range(len(self.plens)):
                    if self.starts[g] <= b < self.starts[g + 1]:
                        ids, n = self.ptable[g, :-(-self.plens[g] // self.BS)], self.plens[g]
                        k.append(K[ids, :, h].reshape(-1, 128)[:n])
                        v.append(V[ids, :, h].reshape(-1, 128)[:n])
                ids, n = self.table[b, :-(-self.lens[b] // self.BS)], self.lens[b]
                k.append(K[ids, :, h].reshape(-1, 128)[:n])
                v.append(V[ids, :, h].reshape(-1, 128)[:n])
                k, v = np.concatenate(k), np.concatenate(v)
                rows = slice(h * self.QG, (h + 1) * self.QG)
                out[b, rows] = pp.attention(q[b, rows], k, v, scale)
                if len(k):
                    s = scale * q[b, rows] @ k.T
                    p = np.exp(s - s.max(-1, keepdims=True))
                    p /= p.sum(-1, keepdims=True)
                    ds = scale * (np.abs(q[b, rows]) @ np.abs(k).T).max(-1, keepdims=True) * 130 * 2.0 ** -23
                    rel = half + 2 * ds + (len(k) + 64) * 2.0 ** -23
                    # (f16 weights below 2^-14 of the largest lose bits: half a step of 2^-24, 64 times the largest V)
                    low = 0 if self.kv == BF16 else len(k) * 2.0 ** -25 * 64 * np.abs(v).max()
                    bound[b, rows] = rel * (p @ np.abs(v)) + low
        return out, bound


def check(pda, c, out_dtype=torch.float32, plans=None, **kw):
    p2 = plans or c.plans(pda, **kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = c.device()
    guard = 64
    n = pda.lib().pda_shared_workspace_size(*p2)
    ws = torch.full((n + guard,), 0xFF, dtype=torch.uint8, device="cuda")         # NaN everywhere
    out = pda.decode_shared(*p2, **d, ws=ws, out_dtype=out_dtype, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (ws[n:] == 0xFF).all()
    ref, bound = c.reference(p2[1].resolved_softmax_scale)
    got = out.double().cpu().numpy()
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    over = np.abs(got - ref) - bound
    assert np.isfinite(got).all() and over.max() <= 1e-30, (over.max(), np.abs(got - ref).max())
    return out


@pytest.mark.parametrize("kv", [BF16, FP8])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 128, 129, 256, 300, 1000])
def test_prefix_lengths(pda, kv, n):
    check(pda, Case(kv, 1, 8, 16, [n], [3], [5, 1, 40], seed=n))


@pytest.mark.parametrize("kv", [BF16, FP8])
@pytest.mark.parametrize("QG,BS,Hk", [(6, 16, 3), (8, 32, 2), (16, 16, 1), (6, 32, 5)])
def test_head_layouts(pda, kv, QG, BS, Hk):
    check(pda, Case(kv, Hk, QG, BS, [333], [7], [0, 1, BS, BS + 1, 70, 5, 260], seed=QG))


@pytest.mark.parametrize("kv,QG", [(BF16, 8), (FP8, 6), (BF16, 16)])
@pytest.mark.parametrize("B", [1, 15, 16, 17, 32, 33, 47, 64, 100])
def test_batch_sizes(pda, kv, QG, B):
    # row tiles of 128 and 256 rows: full, one row over, one short; QG 6 rows straddle tiles
    rng = np.random.default_rng(B)
    check(pda, Case(kv, 1, QG, 16, [200], [B], rng.integers(0, 50, B).tolist(), seed=B))


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_groups_of_every_kind(pda, kv):
    # sequences before, between and after the groups' range; an empty group, an empty prefix, a group of one
    rng = np.random.default_rng(3)
    c = Case(kv, 2, 8, 16, [700, 30, 0, 129, 1], [20, 0, 3, 1, 40], rng.integers(0, 60, 70).tolist(), before=2, seed=3)
    c.lens[5] = 0
    check(pda, c)
    c = Case(kv, 1, 16, 32, [100, 90, 0], [0, 3, 2], [0, 0, 9, 0, 0, 4], seed=4)
    out = check(pda, c)
    assert (out[3:5] == 0).all()                             # no prefix, no tokens


@pytest.mark.parametrize("kv", [BF16, FP8])
@pytest.mark.parametrize("G", [1, 2, 5, 1000])
def test_pieces(pda, kv, G):
    # the same prefix whole and cut into many pieces
    check(pda, Case(kv, 2, 8, 32, [5000, 777], [40, 2], [3] * 42, seed=G), prefix_tile_groups=G)


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_many_groups(pda, kv):
    rng = np.random.default_rng(6)
    sizes = rng.integers(0, 4, 70).tolist()                  # more groups than one warp's pass
    plens = rng.integers(0, 400, 70).tolist()
    check(pda, Case(kv, 1, 6, 16, plens, sizes, rng.integers(0, 20, sum(sizes)).tolist(), seed=6))


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_large_logits_and_spread_values(pda, kv):
    # peaky softmax (the reference point moves), V scales over many powers of two, keys with an offset
    check(pda, Case(kv, 1, 8, 16, [1500], [20], [30] * 20, seed=7, q_scale=8.0, v_spread=3.0))
    check(pda, Case(kv, 2, 6, 16, [900], [50], [9] * 50, seed=8, q_scale=1e-3, k_bias=3.0))
    check(pda, Case(kv, 1, 8, 16, [400], [4], [9] * 4, seed=9), softmax_scale=0.5)


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_rising_logits_rescale_every_step(pda, kv):
    # keys that grow along the prefix: the maximum rises by more than 2^8 at every step
    c = Case(kv, 1, 8, 16, [1024], [33], [4] * 33, seed=10)
    rng = np.random.default_rng(10)
    ramp = np.linspace(0.2, 40, 1024)[:, None, None]
    k = (rng.standard_normal((1, 1, 128)) * ramp).astype(np.float32)
    v = (rng.standard_normal((1024, 1, 128)) * np.exp(np.linspace(-12, 12, 1024))[:, None, None]).astype(np.float32)
    wl.write_tokens(c.w, c.cache, c.ptable[0], k, v)
    check(pda, c)


def test_v_scales_far_below_their_neighbours(pda):
    """fp8: the tokens that a row attends to have V scales 2^-13 of the largest in their 128 tokens, which itself is 2^-5 of that in
    the 128 tokens before.  A term is off by the three f16 roundings, 3 * 2^-11, and a weight by at most itself or half a step
    of f16's smallest, 2^-25; a V code of few bits by 2^-25 in units of at most half the largest scale."""
    c = Case(FP8, 1, 8, 16, [256], [1], [0], seed=12)
    rng = np.random.default_rng(12)
    k = np.zeros((256, 1, 128), np.float32)
    k[:128, 0, 8] = -10.0
    k[128 + np.arange(8), 0, np.arange(8)] = 3.0
    size = np.where(np.arange(256) < 128, 1.0, 2.0 ** -5)
    size[128:136] = 2.0 ** -18
    v = (rng.standard_normal((256, 1, 128)) * size[:, None, None]).astype(np.float32)
    wl.write_tokens(c.w, c.cache, c.ptable[0], k, v)
    q = np.zeros((1, 8, 128), np.float32)
    q[0, np.arange(8), np.arange(8)] = 100.0
    q[0, :, 8] = 100.0
    c.q = wl.round_bf16(q)
    out = pda.decode_shared(*c.plans(pda), **c.device(), out_dtype=torch.float32).double().cpu().numpy()[0]
    K, V = (x[c.ptable[0], :, 0].reshape(256, 128) for x in pp.block_values(c.w, c.cache))
    s = 128 ** -0.5 * wl.bf16_bits_to_f32(c.q)[0].astype(np.float64) @ K.T
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ds = 128 ** -0.5 * 4 * 1300 * 2.0 ** -23                 # two products, at most 300 and 1000, their sum and scale in fp32
    bound = (3 * 2.0 ** -11 * (1 + 2.0 ** -10) + 2 * ds + 320 * 2.0 ** -23) * (p @ np.abs(V))
    bound += np.minimum(p, 2.0 ** -25) @ np.abs(V) + 2.0 ** -26 * 2.0 ** -5 * 5 / 448
    assert (np.abs(out - p @ V) <= bound).all()


def test_infinite_and_nan_data_stay_in_their_rows(pda):
    for kv in (BF16, FP8):
        c = Case(kv, 1, 8, 16, [300], [20], [3] * 20, seed=11)
        c.q[4, 2] = 0x7FC0                                   # a NaN query row
        p2, d = c.plans(pda), c.device()
        out = pda.decode_shared(*p2, **d, out_dtype=torch.float32).cpu().numpy()
        assert np.isnan(out[4, 2]).all()
        ref, bound = Case.reference(c)
        ok = np.ones(out.shape[:2], bool)
        ok[4, 2] = False
        assert (np.abs(out - ref) <= bound)[ok].all()


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_bf16_output_and_determinism(pda, kv):
    c = Case(kv, 4, 8, 16, [2000, 100], [30, 10], [20] * 40, seed=12)
    p2 = c.plans(pda)
    a = check(pda, c, out_dtype=torch.bfloat16, plans=p2)
    for _ in range(3):
        assert torch.equal(a, check(pda, c, out_dtype=torch.bfloat16, plans=p2))


def test_data_errors(pda):
    for kv in (BF16, FP8):
        c = Case(kv, 1, 8, 16, [100, 64, 50], [2, 2, 2], [5] * 6, seed=13)
        d, p2 = c.device(), c.plans(pda)
        good = pda.decode_shared(*p2, **d, out_dtype=torch.float32)
        def run(**kw):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = pda.decode_shared(*p2, **{**d, **kw}, out_dtype=torch.float32, err_word=err)
            torch.cuda.synchronize()
            return out, int(err.item())
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        out, e = run(prefix_lens=i32(100, c.MP * 16 + 1, 50))
        assert e == pda.ERRW_BAD_CONTEXT_LEN and torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
        alone = pda.decode_step(p2[1], d["query"], d["kv_cache"], c.NB, d["block_table"], d["context_lens"], out_dtype=torch.float32)
        assert (out[2:4] - alone[2:4]).abs().max() <= 1e-6 * alone.abs().max()          # such a group has no prefix
        out, e = run(prefix_lens=i32(-1, 64, 50))
        assert e == pda.ERRW_BAD_CONTEXT_LEN and torch.equal(out[2:], good[2:])
        for starts in ((0, 2, 4, 7), (-1, 2, 4, 6), (0, 2, 1, 6), (0, 9, 4, 6)):
            out, e = run(group_starts=i32(*starts))          # not ascending within the batch: no prefixes
            assert e == pda.ERRW_BAD_GROUP and (out - alone).abs().max() <= 1e-6 * alone.abs().max()
        t = d["prefix_table"].clone()
        t[1, 1], t[1, 2] = -3, c.NB
        out, e = run(prefix_table=t)
        assert e == pda.ERRW_BAD_BLOCK_ID and torch.equal(out[:2], good[:2]) and torch.isfinite(out).all()
        out, e = run(context_lens=i32(5, 5, 5, 5, 5, c.MB * 16 + 1))
        assert e == pda.ERRW_BAD_CONTEXT_LEN and torch.equal(out[:5], good[:5])


def test_wait_timeout_sets_the_error_bit_and_the_next_call_is_correct(pda):
    for kv in (BF16, FP8):
        c = Case(kv, 4, 8, 16, [6000], [64], [20] * 64, seed=14)
        p2 = c.plans(pda, wait_timeout_ns=1)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pda.decode_shared(*p2, **c.device(), err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) & pda.ERRW_PIPELINE_TIMEOUT
        check(pda, c)


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_a_short_wait_limit_is_one_of_single_waits(pda, kv):
    """Hundreds of row tiles of one piece each: a CTA takes several units of some 0.2 ms, far more than the limit of one wait."""
    groups, Hk = 120, 4
    c = Case(kv, Hk, 8, 32, [20000], [groups], [0] * groups, seed=17)
    d = c.device()
    d["group_starts"] = torch.arange(groups + 1, dtype=torch.int32, device="cuda")
    d["prefix_table"] = d["prefix_table"].expand(groups, -1).contiguous()
    d["prefix_lens"] = torch.full((groups,), 20000, dtype=torch.int32, device="cuda")
    outs = []
    for limit in (0, 100000):
        p2 = pda.shared_plans(groups, groups, Hk, 8, 32, c.MP, c.MB, kv_dtype=kv, prefix_tile_groups=79, wait_timeout_ns=limit)
        assert p2[0].num_partitions == 1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs.append(pda.decode_shared(*p2, **d, err_word=err))
        torch.cuda.synchronize()
        assert int(err.item()) == 0
    assert torch.equal(*outs)


def test_pool_past_4_gib_and_pinned_query(pda):
    c = Case(BF16, 2, 8, 16, [300], [5], [20] * 5, seed=15)
    d, p2 = c.device(), c.plans(pda)
    want = pda.decode_shared(*p2, **d, out_dtype=torch.float32)
    cbb = p2[1].cache_block_bytes
    off = ((4 << 30) + (64 << 20)) // cbb
    big = torch.empty((off + c.NB) * cbb, dtype=torch.uint8, device="cuda")
    big[off * cbb:] = d["kv_cache"]
    out = torch.empty((5, 16, 128)).pin_memory()
    pda.decode_shared(*p2, d["query"].cpu().pin_memory(), big, off + c.NB, d["group_starts"], d["prefix_table"] + off, d["prefix_lens"],
                      d["block_table"] + off, d["context_lens"], out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_captured_and_on_another_stream(pda, kv):
    # lengths and groups move in device memory between replays of one captured step; two steps with
    # workspaces of their own run at once
    c = Case(kv, 2, 8, 16, [900, 500], [30, 12], [40] * 42, seed=16)
    p2, d = c.plans(pda), c.device()
    ws, out = pda.shared_workspace(*p2, "cuda"), torch.empty((42, 16, 128), device="cuda")
    pda.decode_shared(*p2, **d, ws=ws, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pda.decode_shared(*p2, **d, ws=ws, out=out)
    for plens, starts, n in (([900, 500], [0, 30, 42], 40), ([1, 499], [0, 1, 40], 0), ([0, 0], [0, 30, 42], 7), ([777, 128], [3, 3, 42], 31)):
        c.plens, c.starts, c.lens = plens, starts, [n] * 42
        d["prefix_lens"].copy_(torch.tensor(plens, dtype=torch.int32))
        d["group_starts"].copy_(torch.tensor(starts, dtype=torch.int32))
        d["context_lens"].fill_(n)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref, bound = c.reference()
        assert (np.abs(out.cpu().numpy() - ref) <= bound + 1e-30).all()
    ws2, out2 = pda.shared_workspace(*p2, "cuda"), torch.empty_like(out)
    for _ in range(20):
        with torch.cuda.stream(s):
            pda.decode_shared(*p2, **d, ws=ws2, out=out2, stream=s)
        pda.decode_shared(*p2, **d, ws=ws, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and (np.abs(out.cpu().numpy() - ref) <= bound + 1e-30).all()


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_steps_without_a_pause_share_a_workspace(pda, kv):
    """Short prefixes run before the own tokens and long ones after: steps of both orders, one behind the other on one stream and
    in one workspace, give what each gives alone."""
    cases = [Case(kv, 4, 8, 16, [900], [40], [3 * b % 60 for b in range(40)], seed=13),          # 32 pieces, beside 160 units
             Case(kv, 1, 8, 16, [250], [3], [5, 0, 17], seed=14),                                # one piece
             Case(kv, 8, 16, 32, [3000, 700], [30, 20], [0] * 10 + [70] * 45, seed=15, before=5),  # every SM
             Case(kv, 8, 8, 16, [256], [100], [b % 9 for b in range(100)], seed=16)]
    plans, dev = [c.plans(pda) for c in cases], [c.device() for c in cases]
    alone = [check(pda, c) for c in cases]
    ws = torch.full((max(pda.lib().pda_shared_workspace_size(*p) for p in plans),), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [[torch.full_like(alone[i], float("nan")) for i in range(len(cases))] for _ in range(6)]
    torch.cuda.synchronize()
    for r in range(6):
        for i in (range(4) if r % 2 else (2, 0, 3, 1)):
            pda.decode_shared(*plans[i], **dev[i], ws=ws, out=outs[r][i])
    torch.cuda.synchronize()
    for r in range(6):
        for i in range(len(cases)):
            assert torch.equal(outs[r][i], alone[i]), (r, i)


@pytest.mark.parametrize("as_int", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(pda, as_int):
    """Calls on a side stream that make their own workspace and output, between allocations of the current stream that are still
    being written: neither writes the other's memory."""
    c = Case(BF16, 2, 8, 16, [1200], [20], [30] * 20, seed=18)
    p2, d = c.plans(pda), c.device()
    want = check(pda, c)
    n = pda.lib().pda_shared_workspace_size(*p2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for size in (n, want.nbytes):                        # freed while the current stream writes them
            x = torch.empty(size, dtype=torch.uint8, device="cuda")
            torch.cuda._sleep(200000)
            x.fill_(0xFF)
            del x
        out = pda.decode_shared(*p2, **d, out_dtype=torch.float32, stream=side.cuda_stream if as_int else side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_fork_then_shared_decode(pda):
    """A prompt's sequence is forked into samples that decode with the prompt as their shared prefix: the same as a decode over
    the forked tables."""
    w = wl.small(num_seqs=1, num_kv_heads=2, ctx=(300,), seed=93, max_blocks_per_seq=24, extra_blocks=60)
    inp = wl.generate(w)
    NB, R = w.num_cache_blocks, 9
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    cache, table, lens = dev(inp.cache), dev(inp.block_table), dev(inp.context_lens)
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    refs[table[0, :19].long()] = 1
    p1, pR = pda.plan(1, 2, 8, 16, 24), pda.plan(R, 2, 8, 16, 24)
    t, l, r = torch.empty((R, 24), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty_like(refs)
    pda.fork_sequences(p1, cache, NB, table, lens, refs, torch.zeros(R, dtype=torch.int32, device="cuda"), t, l, r,
                       pda.page_workspace(p1, R, NB, "cuda"), new_tokens=torch.ones(R, dtype=torch.int32, device="cuda"))
    rng = np.random.default_rng(5)
    new = [torch.from_numpy(rng.standard_normal((R, 2, 128)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]
    pda.append_kv(pR, *new, cache, NB, t, l - 1)
    q = torch.from_numpy(rng.standard_normal((R, 16, 128)).astype(np.float32)).cuda().bfloat16()
    want = pda.decode_step(pR, q, cache, NB, t, l, out_dtype=torch.float32)
    # the 18 full blocks are the prefix; the 19th block, copied per row, is each row's own
    pp_, p = pda.shared_plans(R, 1, 2, 8, 16, 18, 6)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = pda.decode_shared(pp_, p, q, cache, NB, i32(0, R), t[:1, :18].contiguous(), i32(288), t[:, 18:].contiguous(), l - 288,
                            out_dtype=torch.float32)
    # P in bf16 (2^-8 of each weight) against the step's 16 bits; |v| < 5
    assert (out - want).abs().max() <= 2.0 ** -8 * 5


def test_every_e4m3_code_in_a_prefix(pda):
    """All 256 codes through the fp8 conversion: a one-hot query reads single key codes as logits, and values are picked out one
    token at a time (a query far along one key's direction)."""
    c = Case(FP8, 1, 8, 16, [256], [1], [0], seed=20)
    data, meta = wl.cache_views(c.w, c.cache)
    codes = np.arange(256, dtype=np.uint8)
    finite = (codes & 0x7F) != 0x7F
    t = np.arange(256)
    blk, slot = c.ptable[0][t // 16], t % 16
    data[blk, slot, 0, 0, :] = 0
    data[blk, slot, 0, 0, 0] = np.where(finite, codes, 0)
    data[blk, slot, 0, 1, :] = np.where(finite, codes, 0)[:, None]
    meta[blk, 0, 0, slot] = 0.25
    meta[blk, 0, 1, slot] = 0.5
    q = np.zeros((1, 8, 128), np.float32)
    q[0, :, 0] = [0.0, 0.1, -0.1, 1.0, -1.0, 0.01, 3.0, -3.0]
    c.q = wl.round_bf16(q)
    check(pda, c)
    for code in (0x7F, 0xFF):                                # a NaN code in V makes its dimension NaN, in K every row that weighs it
        d = c.device()
        keep = c.cache.copy()
        data[c.ptable[0][5], 3, 0, 1, 70] = code
        out = pda.decode_shared(*c.plans(pda), **c.device(), out_dtype=torch.float32).cpu().numpy()
        assert np.isnan(out[0, :, 70]).all() and np.isfinite(np.delete(out, 70, axis=2)).all()
        c.cache[:] = keep
        data[c.ptable[0][5], 3, 0, 0, 1] = code
        assert np.isnan(pda.decode_shared(*c.plans(pda), **c.device(), out_dtype=torch.float32).cpu().numpy()).all()
        c.cache[:] = keep


def test_groups_that_jump_back_and_forth_do_no_work(pda):
    # a table of 4001 overlapping groups names far more rows than there are: an error bit, and no prefix at all
    B, NG = 64, 4001
    pp_, p = pda.shared_plans(B, NG, 8, 16, 16, 60000, 4)
    starts = torch.zeros(NG + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = B
    plens = torch.full((NG,), 60000 * 16, dtype=torch.int32, device="cuda")
    cache = torch.zeros(8 * p.cache_block_bytes, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, 128, 128), dtype=torch.bfloat16, device="cuda")
    out = pda.decode_shared(pp_, p, q, cache, 8, starts, i32(NG, 60000), plens, i32(B, 4), i32(B), err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pda.ERRW_BAD_GROUP and (out == 0).all()


@pytest.mark.parametrize("kv", [BF16, FP8])
def test_outputs_behind_the_last_sequence_stay(pda, kv):
    c = Case(kv, 2, 6, 16, [100], [5], [9] * 5, seed=21)
    out = torch.full((7, 12, 128), 3.0, device="cuda")
    pda.decode_shared(*c.plans(pda), **c.device(), out=out)
    ref, bound = c.reference()
    assert (out[5:] == 3.0).all() and (np.abs(out[:5].cpu().numpy() - ref) <= bound).all()
