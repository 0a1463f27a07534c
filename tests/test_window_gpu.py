"""The decode step over a sliding window and first tokens, against attention in 64 bits."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_tokens as pt

pytestmark = pytest.mark.gpu

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4
KVS = [BF16, FP8, TQ4]


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def poison(c, lens, window, first):
    """What no query sees: NaN, and table entries of blocks that hold nothing else are no block's."""
    for b, n in enumerate(lens):
        start = max(0, n - window)
        if start <= first:
            continue
        t = np.arange(first, start)
        data, meta = wl.cache_views(c.w, c.cache)
        data[c.table[b, t // c.BS], t % c.BS] = 0xFFFF if c.kv == BF16 else 0xFF
        if meta is not None:
            meta[c.table[b, t // c.BS], :, :, t % c.BS] = np.nan if c.kv == FP8 else 0xFFFF
        for j in range(-(-first // c.BS), start // c.BS):
            c.table[b, j] = -1 if j % 2 else c.NB + j


def case(pda, kv, Hk, QG, BS, lens, window, first, seed=0):
    c = pt.Pool(kv, Hk, QG, BS, lens, seed=seed, v_spread=0.5)
    poison(c, lens, window, first)
    c.q = wl.round_bf16(c.rng.standard_normal((c.B, Hk * QG, 128)).astype(np.float32))
    c.lens, c.window, c.first = lens, window, first
    c.p = pda.plan(c.B, Hk, QG, BS, c.MB, kv_dtype=kv)
    c.d = dict(query=torch.from_numpy(c.q.view(np.int16)).cuda().view(torch.bfloat16), kv_cache=torch.from_numpy(c.cache).cuda(),
               num_cache_blocks=c.NB, block_table=i32(c.table), context_lens=i32(lens), window=window, num_first=first,
               centroids=None if c.book is None else torch.from_numpy(c.book).cuda())
    return c


def reference(c):
    out, bound = np.zeros((c.B, c.Hk * c.QG, 128)), np.zeros((c.B, c.Hk * c.QG, 128))
    q = wl.bf16_bits_to_f32(c.q).astype(np.float64)
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        t = t[(t < c.first) | (n - 1 - t < c.window)]
        for h in range(c.Hk if n else 0):
            k, v, vs, vz = pt.token_values(c.w, c.cache, c.table[b, t // c.BS], t % c.BS, h, c.book)
            r = slice(h * c.QG, (h + 1) * c.QG)
            out[b, r], bound[b, r] = pt.attend(q[b, r], k, v, np.ones((c.QG, len(t)), bool), c.kv, tree=False, vscale=vs, vzero=vz)
    return out, bound


def check(pda, c, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pda.decode_window(c.p, **c.d, out_dtype=torch.float32, err_word=err, **kw)
    out16 = pda.decode_window(c.p, **c.d, err_word=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, bound = reference(c)
    off = np.abs(out.cpu().double().numpy() - want)
    assert np.isfinite(off).all() and (off <= bound).all(), (float((off / np.maximum(bound, 1e-30)).max()), float(off.max()))
    assert torch.equal(out16, out.to(torch.bfloat16))
    return out


SIZES = [   # lengths, window, first
    ([1, 2, 15, 16, 17, 33], 1, 0),
    ([1, 2, 15, 16, 17, 33], 2, 1),
    ([0, 5, 40, 64, 65, 100], 16, 4),
    ([0, 3, 300, 47, 48, 49, 81], 17, 33),
    ([700, 1023, 1024, 1025, 1100], 1000, 4),
    ([2000, 100, 513], 400, 100),
    ([5000], 4096, 4),
    ([900, 1000], 1 << 30, 0),
    ([900, 1000], 2147483647, 2147483647),
    ([600, 77, 450], 64, 300),
]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("QG,BS", [(8, 16), (6, 32), (16, 32)])
@pytest.mark.parametrize("lens,window,first", SIZES)
def test_against_64_bits(pda, kv, QG, BS, lens, window, first):
    check(pda, case(pda, kv, 2, QG, BS, lens, window, first, seed=len(lens) + QG))


@pytest.mark.parametrize("kv", KVS)
def test_every_border(pda, kv):
    """Lengths and windows that begin and end at every place of a block, first tokens up to past a tile."""
    for first in (0, 3, 16, 21):
        for window in (1, 7, 16, 30, 33):
            check(pda, case(pda, kv, 1, 8, 32, list(range(40, 110)), window, first, seed=window))


@pytest.mark.parametrize("kv", KVS)
def test_many_units(pda, kv):
    """More units than one round of the clusters holds, lengths of all sizes."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 130))]
    check(pda, case(pda, kv, 8, 8, 16, lens, 512, 4, seed=1))


def test_a_window_past_the_context_is_the_whole_step(pda):
    """Where nothing is cut, the step is the one over selected blocks that are all blocks, bit for bit."""
    for kv in KVS:
        c = case(pda, kv, 2, 8, 16, [200, 31], 4096, 4)
        out = check(pda, c)
        table = c.d["block_table"][:, None].expand(c.B, c.Hk, c.MB).contiguous()
        lens = c.d["context_lens"][:, None].expand(c.B, c.Hk).contiguous()
        full = pda.decode_selected(c.p, c.d["query"], c.d["kv_cache"], c.NB, table, lens, out_dtype=torch.float32,
                                   centroids=c.d["centroids"])
        assert torch.allclose(out, full, rtol=0, atol=0) or c.MB * c.BS > 4096


def test_data_errors(pda):
    for kv in KVS:
        c = case(pda, kv, 2, 8, 16, [300, 300, 300], 40, 4, seed=2)
        want, _ = reference(c)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.d["context_lens"] = i32([300, -1, c.MB * c.BS + 1])
        out = pda.decode_window(c.p, **c.d, out_dtype=torch.float32, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pda.ERRW_BAD_CONTEXT_LEN
        assert bool((out[1:] == 0).all()) and np.abs(out[0].cpu().numpy() - want[0]).max() < 0.05
        err.zero_()
        c.d["context_lens"] = i32([300, 300, 300])
        c.d["block_table"][1, 17] = c.NB
        out2 = pda.decode_window(c.p, **c.d, out_dtype=torch.float32, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pda.ERRW_BAD_BLOCK_ID and torch.equal(out2[0], out[0]) and bool(torch.isfinite(out2).all())


def test_graph_stream_and_pinned_memory(pda):
    c = case(pda, FP8, 4, 8, 16, [900, 200, 30], 256, 4, seed=4)
    want = check(pda, c)
    out = torch.zeros_like(want)
    pda.decode_window(c.p, **c.d, out=out)
    torch.cuda.synchronize()
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pda.decode_window(c.p, **c.d, out=out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    got = pda.decode_window(c.p, **c.d, out_dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    host = {k: c.d[k].cpu().pin_memory() for k in ("query", "block_table", "context_lens")}
    hout = torch.zeros(want.shape).pin_memory()
    pda.decode_window(c.p, **{**c.d, **host}, out=hout)
    torch.cuda.synchronize()
    assert torch.equal(hout, want.cpu())
