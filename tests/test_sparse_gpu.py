"""Block summaries, scores, selection and the decode over selected blocks, against 64-bit definitions."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp
from tests.gpu_helpers import to_device

pytestmark = pytest.mark.gpu

FORMATS = [wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4]
TOL = {wl.KV_BF16: 2e-3, wl.KV_FP8_E4M3: 1e-2, wl.KV_TQ4: 1e-2}      # the library's decode bounds


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def outward(x, up):
    """fp32 to bf16 values, up or down."""
    x = np.asarray(x, np.float32)
    t = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)                # towards zero
    away = (t.view(np.uint32) + 0x10000).view(np.float32)
    return np.where((t != x) & ((x > 0) == up), away, t)


def stored_keys32(w, inp):
    """Every block's keys as the fp32 products code x factor."""
    data, meta = wl.cache_views(w, inp.cache)
    with np.errstate(invalid="ignore"):
        if w.kv_dtype == wl.KV_BF16:
            return wl.bf16_bits_to_f32(data[..., 0, :])
        if w.kv_dtype == wl.KV_FP8_E4M3:
            x = torch.from_numpy(np.ascontiguousarray(data[..., 0, :])).view(torch.float8_e4m3fn).float().numpy()
            return x * np.asarray(meta[:, :, 0], np.float32).transpose(0, 2, 1)[..., None]
        packed = np.asarray(data[..., 0, :])
        codes = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 128)
        norm = np.ascontiguousarray(meta[:, :, 0]).view(np.float16).astype(np.float32).transpose(0, 2, 1)
        return inp.extra["centroids"][codes] * norm[..., None]


def plan_of(pda, w, **kw):
    return pda.plan(w.num_seqs, w.num_kv_heads, w.query_group_size, w.kv_block_size, w.max_blocks_per_seq,
                    kv_dtype=w.kv_dtype, **kw)


def expected_summaries(w, inp, ctx, since, before):
    keys, out = stored_keys32(w, inp), before.copy()
    for b in range(w.num_seqs):
        n = int(ctx[b])
        for j in range(max(0, int(since[b])) // w.kv_block_size, -(-n // w.kv_block_size)):
            i = int(inp.block_table[b, j])
            k = keys[i, :min(w.kv_block_size, n - j * w.kv_block_size)]
            out[i, :, 0], out[i, :, 1] = outward(k.max(0), True), outward(k.min(0), False)
    return out


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("BS,Hk", [(16, 1), (32, 3)])
def test_summaries(pda, kv, BS, Hk):
    ctx = (0, 1, BS, BS + 1, 5 * BS - 3, 9 * BS)
    w = wl.small(num_seqs=len(ctx), num_kv_heads=Hk, kv_block_size=BS, ctx=ctx, kv_dtype=kv, seed=BS + kv)
    inp = wl.generate(w)                                     # slots past each context hold NaN
    d, p = to_device(inp), plan_of(pda, w)
    NB = w.num_cache_blocks
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for since in (None, [-4, 0, BS - 1, BS, 2 * BS + 1, 9 * BS - 1], [0, 1, 0, 99999, 0, 9 * BS]):
        summ = torch.full((NB + 1, Hk, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        before = summ[:NB].float().cpu().numpy()
        s = None if since is None else torch.tensor(since, dtype=torch.int32, device="cuda")
        pda.summarize_blocks(p, d["cache"], NB, d["block_table"], d["context_lens"], summ, since=s,
                             centroids=d.get("centroids"), err_word=err)
        want = expected_summaries(w, inp, ctx, [0] * len(ctx) if since is None else since, before)
        assert np.array_equal(summ[:NB].float().cpu().numpy(), want) and (summ[NB] == 7.0).all()
    assert int(err.item()) == 0
    bt = d["block_table"].clone()                            # blocks outside the pool are skipped
    bt[4, 1], bt[5, 3] = NB, -1
    bad = d["context_lens"].clone()
    bad[3] = w.max_blocks_per_seq * BS + 1
    summ.fill_(7.0)
    pda.summarize_blocks(p, d["cache"], NB, bt, bad, summ, centroids=d.get("centroids"), err_word=err)
    inp.block_table, keep = bt.cpu().numpy(), inp.block_table
    skip = {int(keep[4, 1]), int(keep[5, 3])} | {int(keep[3, j]) for j in range(2)}
    want = expected_summaries(w, wl.Inputs(w, inp.query, inp.cache, keep, inp.context_lens, inp.extra), ctx, [0] * 6, before)
    for i in skip:
        want[i] = 7.0
    assert np.array_equal(summ[:NB].float().cpu().numpy(), want)
    assert int(err.item()) == pda.ERRW_BAD_BLOCK_ID | pda.ERRW_BAD_CONTEXT_LEN


def scored(pda, w, inp, p, d, summ, err=None, table=None):
    scores = torch.full((w.num_seqs, w.num_kv_heads, w.max_blocks_per_seq), 55.0, device="cuda")
    pda.score_blocks(p, d["query"], summ, w.num_cache_blocks, d["block_table"] if table is None else table, d["context_lens"],
                     scores, err_word=err)
    return scores.cpu().numpy()


@pytest.mark.parametrize("QG", [6, 8, 16])
@pytest.mark.parametrize("BS,Hk,scale", [(16, 2, 0.0), (32, 1, 0.3)])
def test_scores(pda, QG, BS, Hk, scale):
    ctx = (0, 1, 16 * BS, 16 * BS + 1, 77 * BS - 5)
    w = wl.small(num_seqs=5, num_kv_heads=Hk, query_group_size=QG, kv_block_size=BS, ctx=ctx, seed=QG, k_bias_std=1.0)
    inp = wl.generate(w)
    d, p = to_device(inp), plan_of(pda, w, softmax_scale=scale)
    summ = pda.block_summaries(p, w.num_cache_blocks, "cuda")
    pda.summarize_blocks(p, d["cache"], w.num_cache_blocks, d["block_table"], d["context_lens"], summ)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = scored(pda, w, inp, p, d, summ, err)
    q = wl.bf16_bits_to_f32(inp.query).astype(np.float64).reshape(5, Hk, QG, 128)
    s64 = summ.double().cpu().numpy()
    sc = p.resolved_softmax_scale
    kst, _ = pp.block_values(w, inp.cache)
    for b in range(5):
        n = -(-ctx[b] // BS)
        x = s64[inp.block_table[b, :n]]
        for h in range(Hk):
            terms = np.concatenate([np.maximum(q[b, h], 0)[:, None] * x[None, :, h, 0],
                                    np.minimum(q[b, h], 0)[:, None] * x[None, :, h, 1]], -1)      # [QG][n][256]
            # products of two bf16 values are exact in fp32; 256 additions, each off by at most one
            # step (2^-23: the tensor cores may truncate), one more for the two chains' sum, one scaling
            bound = sc * (np.abs(terms).sum(-1) * 258 * 2.0 ** -23)
            want = sc * terms.sum(-1)
            assert np.all(np.abs(got[b, h, :n] - want.max(0)) <= bound.max(0) + 1e-30)
            assert np.all(got[b, h, n:] == 55.0)
            for j in range(n):                               # it bounds every logit of the block
                t = min(BS, ctx[b] - j * BS)
                logits = sc * q[b, h] @ kst[inp.block_table[b, j], :t, h].T
                assert logits.max() <= got[b, h, j] + bound[:, j].max()
    assert int(err.item()) == 0
    bt = d["block_table"].clone()
    bt[4, 3] = w.num_cache_blocks
    again = scored(pda, w, inp, p, d, summ, err, bt)
    assert (again[4, :, 3] == -np.inf).all() and int(err.item()) == pda.ERRW_BAD_BLOCK_ID
    again[4, :, 3] = got[4, :, 3]
    assert np.array_equal(again, got)


@pytest.mark.parametrize("K,first,last", [(1, 0, 0), (1, 1, 0), (4, 1, 2), (4, 2, 2), (16, 0, 1), (64, 1, 2), (300, 3, 5)])
@pytest.mark.parametrize("BS", [16, 32])
def test_select(pda, K, first, last, BS):
    rng = np.random.default_rng(K + BS)
    lens = np.array([0, 1, BS, 2 * BS - 1, 5 * BS, K * BS, K * BS + 1, 257 * BS - 3, 1000 * BS, 1100 * BS - 7], np.int32)
    B, Hk, MB = len(lens), 6, 1100
    scores = rng.standard_normal((B, Hk, MB)).astype(np.float32)
    scores[:, 1] = np.round(scores[:, 1])                    # many ties
    scores[:, 2] = 3.0                                       # all equal
    scores[:, 3] = np.where(rng.random((B, MB)) < 0.5, 0.0, -0.0)          # +0 and -0 are equal
    scores[:, 4, ::3] = np.inf
    scores[:, 4, 1::3] = -np.inf
    scores[:, 5, rng.integers(0, MB, 700)] = np.nan
    table = rng.integers(0, 1 << 30, (B, MB)).astype(np.int32)
    p = pda.plan(B, Hk, 8, BS, MB)
    sel = torch.full((B, Hk, K), 9, dtype=torch.int32, device="cuda")
    blocks, tokens = sel.clone(), torch.full((B, Hk), 9, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.from_numpy(x).cuda()
    pda.select_blocks(p, dev(scores), dev(table), dev(lens), K, first, last, sel, tokens, sel_blocks=blocks)
    want = pp.select(scores, lens, BS, K, first, last)
    sel2, tokens2 = sel.clone().fill_(9), tokens.clone().fill_(9)
    pda.select_blocks(p, dev(scores), dev(table), dev(lens), K, first, last, sel2, tokens2)
    assert torch.equal(sel, sel2) and torch.equal(tokens, tokens2)
    for b in range(B):
        for h in range(Hk):
            js = want[b * Hk + h]
            pad = [-1] * (K - len(js))
            assert blocks[b, h].tolist() == js + pad, (b, h)
            assert sel[b, h].tolist() == [int(table[b, j]) for j in js] + pad
            assert int(tokens[b, h]) == sum(min(BS, int(lens[b]) - j * BS) for j in js)


def test_select_of_a_row_longer_than_the_staging(pda):
    rng = np.random.default_rng(0)
    MB = 30011                                               # keys re-read instead of staged
    lens = np.array([MB * 16 - 5, 12000 * 16], np.int32)
    scores = np.round(rng.standard_normal((2, 1, MB)) * 50).astype(np.float32)
    table = rng.permutation(2 * MB).astype(np.int32).reshape(2, MB)
    p = pda.plan(2, 1, 8, 16, MB)
    sel, tokens = torch.empty((2, 1, 500), dtype=torch.int32, device="cuda"), torch.empty((2, 1), dtype=torch.int32, device="cuda")
    blocks = torch.empty_like(sel)
    dev = lambda x: torch.from_numpy(x).cuda()
    pda.select_blocks(p, dev(scores), dev(table), dev(lens), 500, 2, 1, sel, tokens, sel_blocks=blocks)
    want = pp.select(scores, lens, 16, 500, 2, 1)
    assert blocks[0, 0].tolist() == want[0] and blocks[1, 0].tolist() == want[1]
    assert tokens.flatten().tolist() == [500 * 16 - 5, 500 * 16]


def test_select_bad_length(pda):
    p = pda.plan(2, 2, 8, 16, 4)
    scores = torch.zeros((2, 2, 4), device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda")
    sel, tokens = torch.full((2, 2, 2), 9, dtype=torch.int32, device="cuda"), torch.full((2, 2), 9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pda.select_blocks(p, scores, table, torch.tensor([65, 40], dtype=torch.int32, device="cuda"), 2, 0, 1, sel, tokens, err_word=err)
    assert int(err.item()) == pda.ERRW_BAD_CONTEXT_LEN
    assert sel[0].flatten().tolist() == [-1] * 4 and tokens.tolist() == [[0, 0], [24, 24]]
    assert sel[1].tolist() == [[4, 6], [4, 6]]


def check_selected(pda, w, inp, lists, p, d, K, out_dtype=torch.float32, err=None):
    """decode_selected over the given logical blocks against the definition."""
    B, Hk, QG, BS = w.num_seqs, w.num_kv_heads, w.query_group_size, w.kv_block_size
    sel = np.full((B, Hk, K), -1, np.int32)
    lens = np.zeros((B, Hk), np.int32)
    for b in range(B):
        for h in range(Hk):
            js = lists[b * Hk + h]
            sel[b, h, :len(js)] = inp.block_table[b, js]
            lens[b, h] = sum(min(BS, int(inp.context_lens[b]) - j * BS) for j in js)
    out = pda.decode_selected(p, d["query"], d["cache"], w.num_cache_blocks, torch.from_numpy(sel).cuda(), torch.from_numpy(lens).cuda(),
                              out_dtype=out_dtype, centroids=d.get("centroids"), err_word=err)
    got = out.double().cpu().numpy()
    q = wl.bf16_bits_to_f32(inp.query).astype(np.float64)
    kst, vst = pp.block_values(w, inp.cache, inp.extra.get("centroids"))
    for b in range(B):
        for h in range(Hk):
            n = lens[b, h]
            ids = sel[b, h, :-(-n // BS)]
            ref = pp.attention(q[b, h * QG:(h + 1) * QG], kst[ids, :, h].reshape(-1, 128)[:n], vst[ids, :, h].reshape(-1, 128)[:n],
                               p.resolved_softmax_scale)
            tol = TOL[w.kv_dtype] + (np.abs(ref) * 2.0 ** -8 if out_dtype == torch.bfloat16 else 0)
            assert np.all(np.abs(got[b, h * QG:(h + 1) * QG] - ref) <= tol), (b, h)
    return out


@pytest.mark.parametrize("variant", [0, 1])                  # one launch of clusters; partition pass and reduce
@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("QG,BS,Hk,G", [(6, 16, 3, 1), (8, 32, 2, 2), (16, 16, 1, 1)])
def test_decode_selected(pda, kv, QG, BS, Hk, G, variant):
    ctx = (0, 1, BS + 3, 40 * BS, 61 * BS - 2)
    w = wl.small(num_seqs=5, num_kv_heads=Hk, query_group_size=QG, kv_block_size=BS, ctx=ctx, kv_dtype=kv, seed=QG + kv)
    inp = wl.generate(w)
    d, K = to_device(inp), 37
    p = pda.plan(5, Hk, QG, BS, K, tile_groups_per_partition=G, kv_dtype=kv, kernel_variant=variant)
    rng = np.random.default_rng(kv)
    lists = []
    for b in range(5):
        nb = -(-ctx[b] // BS)
        for h in range(Hk):                                  # other blocks for every head, none for one
            take = sorted(rng.permutation(nb)[:rng.integers(0, min(K, nb) + 1)].tolist())
            lists.append(take if (b, h) != (3, 0) else [])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_selected(pda, w, inp, lists, p, d, K, err=err)
    check_selected(pda, w, inp, lists, p, d, K, out_dtype=torch.bfloat16, err=err)
    assert int(err.item()) == 0


def test_decode_selected_of_every_block_is_the_plain_step(pda):
    w = wl.small(num_seqs=3, num_kv_heads=2, ctx=(300, 77, 512), seed=5)
    inp = wl.generate(w)
    d, p = to_device(inp), plan_of(pda, w, kernel_variant=1)
    plain = pda.decode_step(p, d["query"], d["cache"], w.num_cache_blocks, d["block_table"], d["context_lens"], out_dtype=torch.float32)
    table = d["block_table"][:, None].expand(-1, 2, -1).contiguous()
    lens = d["context_lens"][:, None].expand(-1, 2).contiguous()
    out = pda.decode_selected(p, d["query"], d["cache"], w.num_cache_blocks, table, lens, out_dtype=torch.float32)
    assert torch.equal(out, plain)                           # the same partitions
    out = pda.decode_selected(plan_of(pda, w), d["query"], d["cache"], w.num_cache_blocks, table, lens, out_dtype=torch.float32)
    # other runs of tokens: each weight is off by at most 2^-16 (P as two bf16) and a few steps of 2^-23, |V| < 6
    assert (out - plain).abs().max() <= 2 * 6 * 2.0 ** -16 * 1.1


@pytest.mark.parametrize("kv,QG", [(wl.KV_BF16, 8), (wl.KV_BF16, 16), (wl.KV_FP8_E4M3, 6), (wl.KV_TQ4, 8), (wl.KV_FP8_E4M3, 16)])
@pytest.mark.parametrize("B,K", [(1, 70), (37, 9), (150, 33), (700, 2)])
def test_decode_selected_shapes(pda, kv, QG, B, K):
    # few long units (clusters of eight), many short ones (single CTAs), lists shorter than the warps, blocks shared by units
    rng = np.random.default_rng(B)
    w = wl.small(num_seqs=1, num_kv_heads=2, query_group_size=QG, ctx=(16 * 80,), kv_dtype=kv, seed=B)
    inp = wl.generate(w)
    d = to_device(inp)
    p = pda.plan(B, 2, QG, 16, K, kv_dtype=kv)
    sel, lens = np.full((B, 2, K), -1, np.int32), np.zeros((B, 2), np.int32)
    for b in range(B):
        for h in range(2):
            n = rng.integers(0, K + 1) if b else K
            sel[b, h, :n] = inp.block_table[0, rng.permutation(80)[:n]]
            lens[b, h] = max(0, n * 16 - rng.integers(0, 16))
    q = wl.round_bf16(rng.standard_normal((B, 2 * QG, 128)).astype(np.float32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pda.decode_selected(p, torch.from_numpy(q.view(np.int16)).cuda().view(torch.bfloat16), d["cache"], w.num_cache_blocks,
                              torch.from_numpy(sel).cuda(), torch.from_numpy(lens).cuda(), out_dtype=torch.float32,
                              centroids=d.get("centroids"), err_word=err)
    got, q64 = out.double().cpu().numpy(), wl.bf16_bits_to_f32(q).astype(np.float64)
    kst, vst = pp.block_values(w, inp.cache, inp.extra.get("centroids"))
    for b in range(B):
        for h in range(2):
            ids, n, rows = sel[b, h, :-(-lens[b, h] // 16)], lens[b, h], slice(h * QG, (h + 1) * QG)
            ref = pp.attention(q64[b, rows], kst[ids, :, h].reshape(-1, 128)[:n], vst[ids, :, h].reshape(-1, 128)[:n], 128 ** -0.5)
            assert np.abs(got[b, rows] - ref).max() <= TOL[kv], (b, h)
    assert int(err.item()) == 0


def test_decode_selected_timeout_sets_the_error_bit_and_the_next_call_is_correct(pda):
    w = wl.small(num_seqs=16, num_kv_heads=8, ctx=(4096,) * 16, seed=61, extra_blocks=0)
    inp = wl.generate(w)
    d = to_device(inp)
    table = d["block_table"][:, None].expand(-1, 8, -1).contiguous()
    lens = torch.full((16, 8), 4096, dtype=torch.int32, device="cuda")
    args = (d["query"], d["cache"], w.num_cache_blocks, table, lens)
    for variant in (0, 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pda.decode_selected(plan_of(pda, w, wait_timeout_ns=1, kernel_variant=variant), *args, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) & pda.ERRW_PIPELINE_TIMEOUT
        err.zero_()
        out = pda.decode_selected(plan_of(pda, w, kernel_variant=variant), *args, out_dtype=torch.float32, err_word=err)
        plain = pda.decode_step(plan_of(pda, w), d["query"], d["cache"], w.num_cache_blocks, d["block_table"], d["context_lens"],
                                out_dtype=torch.float32)
        assert int(err.item()) == 0 and (out - plain).abs().max() <= 2 * 6 * 2.0 ** -16 * 1.1


def test_decode_selected_data_errors(pda):
    w = wl.small(num_seqs=2, num_kv_heads=2, ctx=(64, 64), seed=6)
    inp = wl.generate(w)
    d, p = to_device(inp), plan_of(pda, w)
    table = d["block_table"][:, None].expand(-1, 2, -1).contiguous()
    table[0, 1, 2] = w.num_cache_blocks + 9
    lens = torch.tensor([[64, 64], [65, 0]], dtype=torch.int32, device="cuda")
    for variant in (0, 1):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pda.decode_selected(plan_of(pda, w, kernel_variant=variant), d["query"], d["cache"], w.num_cache_blocks, table, lens,
                                  out_dtype=torch.float32, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pda.ERRW_BAD_BLOCK_ID | pda.ERRW_BAD_CONTEXT_LEN
        assert (out[1] == 0).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("kv", FORMATS)
def test_the_steps_together(pda, kv):
    """As a decode loop runs them: append, renew the newest summary, score, select, attend; twice, on
    another stream, and again from a captured graph."""
    ctx0 = (700, 15, 16, 333)
    w = wl.small(num_seqs=4, num_kv_heads=2, ctx=ctx0, kv_dtype=kv, seed=17, max_blocks_per_seq=48)
    inp = wl.generate(w)
    d, p, K = to_device(inp), plan_of(pda, w), 12
    ps = pda.plan(4, 2, 8, 16, K, kv_dtype=kv)
    NB, cent = w.num_cache_blocks, d.get("centroids")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = d["context_lens"]
    if kv == wl.KV_TQ4:                                      # no encoder: the last token stands for the new one
        ctx.sub_(1)
    summ = pda.block_summaries(p, NB, "cuda")
    pda.summarize_blocks(p, d["cache"], NB, d["block_table"], ctx, summ, centroids=cent, err_word=err)
    scores = torch.empty((4, 2, 48), device="cuda")
    sel, blocks = (torch.empty((4, 2, K), dtype=torch.int32, device="cuda") for _ in range(2))
    lens, since = torch.empty((4, 2), dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    ws, out = pda.workspace(ps, "cuda"), torch.empty((4, 16, 128), device="cuda")
    rng = np.random.default_rng(3)
    new = [torch.from_numpy(rng.standard_normal((4, 2, 128)).astype(np.float32)).cuda().bfloat16() for _ in range(2)]

    def step():
        since.copy_(ctx)
        if kv != wl.KV_TQ4:
            pda.append_kv(p, new[0], new[1], d["cache"], NB, d["block_table"], ctx, err_word=err)
        ctx.add_(1)
        pda.summarize_blocks(p, d["cache"], NB, d["block_table"], ctx, summ, since=since, centroids=cent, err_word=err)
        pda.score_blocks(p, d["query"], summ, NB, d["block_table"], ctx, scores, err_word=err)
        pda.select_blocks(p, scores, d["block_table"], ctx, K, 1, 1, sel, lens, sel_blocks=blocks, err_word=err)
        pda.decode_selected(ps, d["query"], d["cache"], NB, sel, lens, ws=ws, out=out, centroids=cent, err_word=err)

    def check():
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        now = wl.Inputs(w, inp.query, d["cache"].cpu().numpy(), inp.block_table, ctx.cpu().numpy(), inp.extra)
        fresh = torch.empty_like(summ)
        pda.summarize_blocks(p, d["cache"], NB, d["block_table"], ctx, fresh, centroids=cent)
        for b in range(4):
            ids = torch.from_numpy(inp.block_table[b, :-(-int(ctx[b]) // 16)]).long()
            assert torch.equal(summ[ids], fresh[ids])
        lists = pp.select(scores.cpu().numpy(), now.context_lens, 16, K, 1, 1)
        for i, js in enumerate(lists):
            assert blocks.view(8, K)[i].tolist() == js + [-1] * (K - len(js))
        assert torch.equal(check_selected(pda, w, now, lists, ps, d, K), out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    check()
    if kv == wl.KV_TQ4:
        return
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for _ in range(3):
        g.replay()
        check()
