"""The step for drafted tokens, in chains, trees and other masks, against attention in 64 bits."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests.tree_cases import TreeCase

pytestmark = pytest.mark.gpu

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4
KVS = [BF16, FP8, TQ4]


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


SIZES = [   # cached lengths, drafted counts
    ([0], [1]),
    ([250], [4]),
    ([0, 1, 127, 128, 129, 255], [1, 2, 3, 4, 5, 6]),
    ([126, 127, 128, 120], [2, 2, 2, 9]),
    ([300, 40, 0, 700], [0, 33, 17, 0]),
    ([1000, 513], [64, 65]),
    ([90], [130]),
    ([2500, 3, 640], [7, 40, 1]),
]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("kind", ["chain", "tree", "anything"])
@pytest.mark.parametrize("lens,counts", SIZES)
def test_against_64_bits(pda, kv, kind, lens, counts):
    TreeCase(kv, 2, 8, 16, lens, counts, kind, seed=len(lens) + sum(counts)).check(pda)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("QG,BS,Hk", [(6, 16, 3), (6, 32, 1), (16, 32, 2), (8, 32, 5)])
def test_heads_and_blocks(pda, kv, QG, BS, Hk):
    TreeCase(kv, Hk, QG, BS, [400, 31, 0, 129], [9, 50, 3, 16], "tree", seed=QG + BS).check(pda)


WINDOWS = [(1, 0), (2, 1), (100, 4), (128, 0), (129, 130), (40, 300), (600, 17), (1 << 30, 4), (2147483647, 2147483647)]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("window,first", WINDOWS)
@pytest.mark.parametrize("kind", ["chain", "tree", "anything"])
def test_windows(pda, kv, window, first, kind):
    TreeCase(kv, 2, 8, 16, [1000, 130, 0, 383, 2], [5, 20, 3, 33, 1], kind, window, first, seed=window % 97).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_window_borders(pda, kv):
    """Windows that begin at every place of a block, first tokens that end anywhere."""
    for first in (0, 5, 127, 128, 160):
        TreeCase(kv, 1, 8, 32, list(range(470, 530, 3)), [1 + i % 4 for i in range(20)], "tree", 97, first, seed=first).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_rows_that_see_nothing(pda, kv):
    """No cached token, and masks that name none: zeros, whatever the neighbours see."""
    t = TreeCase(kv, 2, 8, 16, [0, 0, 64], [5, 1, 3], "anything", seed=1)
    t.masks = [[[], [0, 1], [], [4], []], [[]], [[], [0], []]]
    t.see = [np.zeros((5, 5), bool), np.zeros((1, 1), bool), np.zeros((3, 67), bool)]
    t.see[0][1, :2] = t.see[0][3, 4] = True
    t.see[2][:, :64] = t.see[2][1, 64] = True
    out = t.check(pda)
    assert bool((out[[0, 2, 4, 5]] == 0).all())


@pytest.mark.parametrize("kv", KVS)
def test_padded_rows_stay(pda, kv):
    t = TreeCase(kv, 2, 6, 16, [100, 0, 300], [4, 0, 9], "tree", seed=2, before=3, after=5)
    out = t.check(pda)
    assert bool((out[:3] == 7).all()) and bool((out[-5:] == 7).all())


@pytest.mark.parametrize("kv", KVS)
def test_masks_shorter_than_the_tree(pda, kv):
    """Tokens past the masks' bits are seen by none, their own rows included."""
    TreeCase(kv, 1, 8, 16, [70], [100], "tree", seed=3, words=1).check(pda)
    TreeCase(kv, 1, 8, 16, [70], [9], "tree", seed=3, words=4).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_many_sequences(pda, kv):
    """More sequences than a warp has lanes, lengths of all sizes, several row tiles."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(2000), 90)) - 1]
    counts = [int(x) for x in rng.integers(0, 9, 90)]
    TreeCase(kv, 2, 8, 16, lens, counts, "tree", seed=4).check(pda)
    TreeCase(kv, 4, 16, 32, [700, 0, 4000], [100, 60, 40], "tree", seed=4).check(pda)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("window,first", [(0, 0), (200, 3)])
def test_unlike_trees(pda, kv, window, first):
    """Several units per SM, of one row, of a tile's 128, one more, two tiles' 256 and one more, in every order."""
    rng = np.random.default_rng(11)
    counts = [int(x) for x in rng.choice([1, 3, 15, 16, 17, 31, 32, 33, 40], 90)]
    lens = [int(x) for x in rng.integers(0, 520, 90)]
    TreeCase(kv, 8, 8, 16, lens, counts, "tree", window, first, seed=12).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_many_pieces(pda, kv):
    """One long sequence over every SM: more than 32 pieces for the join."""
    TreeCase(kv, 1, 8, 32, [20000], [3], "tree", seed=6).check(pda)
    TreeCase(kv, 1, 8, 32, [20000, 10], [3, 2], "chain", 9000, 200, seed=6).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_long_chains(pda, kv):
    """A chain longer than its window, and than several steps: the last part of a prompt."""
    TreeCase(kv, 1, 6, 16, [37], [400], "chain", seed=7).check(pda)
    TreeCase(kv, 1, 6, 16, [300], [300], "chain", 50, 20, seed=7).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_peaked_weights(pda, kv):
    TreeCase(kv, 2, 8, 16, [900, 60], [12, 3], "tree", seed=8, q_scale=8.0, v_spread=2.0).check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_peaked_weights_in_units_of_every_size(pda, kv):
    """References that move, in the first and the second half of a step, in rows held twice (up to 64), in one tile and in two."""
    lens, counts = [900, 60, 1300, 700, 1024, 411, 1500, 640], [12, 8, 16, 17, 1, 33, 9, 40]
    TreeCase(kv, 4, 8, 16, lens, counts, "tree", seed=13, q_scale=8.0, v_spread=2.0).check(pda)
    TreeCase(kv, 4, 8, 32, lens, counts, "anything", 500, 4, seed=14, q_scale=8.0, v_spread=2.0).check(pda)


def test_one_token_is_the_plain_step(pda):
    """Chains of one token over n cached ones are a plain step over n + 1."""
    for kv in KVS:
        t = TreeCase(kv, 2, 8, 16, [100, 0, 555], [1, 1, 1], "chain", seed=9)
        out = t.check(pda)
        d = t.device()
        ref = pda.decode_step(t.plan(pda), d["query"], d["kv_cache"], t.c.NB, d["block_table"], d["context_lens"] + 1,
                              out_dtype=torch.float32, centroids=d["centroids"])
        _, bound = t.reference()
        assert bool(((out - ref).abs().cpu().numpy() <= 2 * bound + 1e-6).all())


def test_data_errors(pda):
    for kv in KVS:
        t = TreeCase(kv, 2, 8, 16, [100, 60, 33, 90], [4, 9, 2, 5], "tree", seed=10)
        want, bound = t.reference()
        d = t.device()
        room = t.c.MB * 16
        d["context_lens"] = torch.tensor([100, -1, room + 1, room - 4], dtype=torch.int32, device="cuda")
        out, err = t.run(pda, d)
        assert err == pda.ERRW_BAD_CONTEXT_LEN | pda.ERRW_BAD_POSITION
        assert (np.abs(out[:4].cpu().numpy() - want[:4]) <= bound[:4]).all() and bool((out[4:] == 0).all())
        d = t.device()
        d["block_table"][1, 2] = t.c.NB
        d["block_table"][2, 0] = -3
        out, err = t.run(pda, d)
        assert err == pda.ERRW_BAD_BLOCK_ID and bool(torch.isfinite(out).all())
        for rows in (slice(0, 4), slice(15, 20)):
            assert (np.abs(out[rows].cpu().numpy() - want[rows]) <= bound[rows]).all()


@pytest.mark.parametrize("starts", [[0, 4, 3, 15, 20], [-1, 4, 13, 15, 20], [0, 4, 13, 15, 21], [5, 4, 4, 4, 4]])
def test_starts_that_do_not_ascend(pda, starts):
    for kv in (BF16, FP8):
        t = TreeCase(kv, 2, 8, 16, [100, 60, 33, 90], [4, 9, 2, 5], "tree", seed=10)
        d = t.device()
        d["token_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out, err = t.run(pda, d)
        assert err == pda.ERRW_BAD_TOKENS and bool((out == 7).all())


def test_graph_and_streams(pda):
    """One workspace, a captured step replayed with other lengths and masks, and the same call on a stream of its own."""
    t = TreeCase(BF16, 4, 8, 16, [700, 90, 0], [9, 30, 2], "tree", seed=11)
    d, p = t.device(), t.plan(pda)
    want = t.check(pda)
    ws = pda.tree_workspace(p, t.N, "cuda")
    out = torch.zeros_like(want)
    pda.decode_tree(p, **d, ws=ws, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pda.decode_tree(p, **d, ws=ws, out=out)
    for _ in range(3):
        ws.fill_(0xFF)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens, masks = d["context_lens"].clone(), d["tree_masks"].clone()
    d["context_lens"].copy_(torch.tensor([300, 90, 0]))
    d["tree_masks"].copy_(masks.roll(1, 0))
    g.replay()
    other = out.clone()
    assert torch.equal(pda.decode_tree(p, **d, out_dtype=torch.float32), other) and not torch.equal(other, want)
    d["context_lens"].copy_(lens)
    d["tree_masks"].copy_(masks)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pda.decode_tree(p, **d, out_dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_short_waits_end(pda):
    """A wait limit below a copy's latency sets the bit and leaves the context usable."""
    t = TreeCase(BF16, 2, 8, 16, [2000], [9], "tree", seed=12)
    out, err = t.run(pda, p=t.plan(pda, wait_timeout_ns=1))
    assert err in (0, pda.ERRW_PIPELINE_TIMEOUT)
    t.check(pda)


# ---------------------------------------------------------------------------- the operators together
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("window,first", [(0, 0), (48, 4)])
def test_a_round_of_speculative_decoding(pda, kv, window, first):
    """A prompt is written, trees are drafted behind it and verified, their paths accepted; the next single-token step and
    another round see the same cache as one that was written token by token."""
    rng = np.random.default_rng(13)
    Hk, QG, BS, MB, B = 2, 8, 16, 12, 3
    NB = B * MB
    p = pda.plan(B, Hk, QG, BS, MB, kv_dtype=kv)
    book = torch.from_numpy(wl.tq4_codebook()).cuda() if kv == TQ4 else None
    i32 = lambda x: torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")
    table = i32(rng.permutation(NB).reshape(B, MB))
    cache, plain = (torch.full((NB * p.cache_block_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))

    def draw(n):
        return [torch.from_numpy(rng.standard_normal((n, Hk, 128)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2)]

    def put(pool, kv_rows, starts, positions):
        pda.write_kv(p, *kv_rows, pool, NB, table, i32(starts), positions, centroids=book)

    prompt = [60, 17, 100]
    starts = np.concatenate([[0], np.cumsum(prompt)])
    rows = draw(starts[-1])
    put(cache, rows, starts, i32([0, 0, 0]))
    put(plain, rows, starts, i32([0, 0, 0]))
    lens = i32(prompt)
    for _ in range(2):
        counts, paths = [6, 3, 7], [[0, 2, 5], [1], [0, 1, 4, 6]]
        starts = np.concatenate([[0], np.cumsum(counts)])
        rows = draw(starts[-1])
        put(cache, rows, starts, lens)
        masks = np.zeros((starts[-1], 1), np.int64)
        for b, path in enumerate(paths):
            for i in range(counts[b]):
                masks[starts[b] + i, 0] = sum(1 << j for j in path if j < i) | 1 << i
        q = torch.from_numpy(rng.standard_normal((starts[-1], Hk * QG, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
        out = pda.decode_tree(p, q, cache, NB, table, lens, i32(starts), tree_masks=torch.from_numpy(masks).cuda(),
                              window=window, num_first=first, centroids=book, out_dtype=torch.float32)
        new_lens = torch.empty_like(lens)
        width = max(map(len, paths))
        pda.accept_tokens(p, cache, NB, table, lens, i32([x + [-1] * (width - len(x)) for x in paths]), i32([len(x) for x in paths]),
                          new_lens)
        # token by token, the accepted ones only
        at = lens.clone()
        for step in range(width):
            live = [step < len(x) for x in paths]
            pick = [starts[b] + x[step] if step < len(x) else 0 for b, x in enumerate(paths)]
            one = [r[pick].contiguous() for r in rows]
            pos = torch.where(torch.tensor(live, device="cuda"), at, torch.full_like(at, -1))
            if kv == TQ4:
                put(plain, one, [0, 1, 2, 3], pos)
            else:
                pda.append_kv(p, *one, plain, NB, table, pos)
            at = at + i32(live)
            size = torch.where(torch.tensor(live, device="cuda"), at, torch.zeros_like(at))
            if window:
                ref = pda.decode_window(p, q[pick].contiguous(), plain, NB, table, size, window, num_first=first, centroids=book,
                                        out_dtype=torch.float32)
            else:
                ref = pda.decode_step(p, q[pick].contiguous(), plain, NB, table, size, out_dtype=torch.float32, centroids=book)
            for b in range(B):
                if live[b]:
                    # both are within the weights' rounding of the result: 2^-8 and 2^-16 of a mean of |v| < 5
                    assert float((out[pick[b]] - ref[b]).abs().max()) < 5 * 2 ** -7
        assert torch.equal(at, new_lens)
        lens = new_lens
        starts = np.concatenate([[0], np.cumsum(lens.tolist())])
        back = [[torch.zeros(starts[-1], Hk, 128, device="cuda") for _ in range(2)] for _ in range(2)]
        for pool, o in zip((cache, plain), back):
            pda.read_kv(p, pool, NB, table, i32(starts), i32([0, 0, 0]), *o, centroids=book)
        assert torch.equal(back[0][0], back[1][0]) and torch.equal(back[0][1], back[1][1])


def test_pinned_query_and_out(pda):
    for kv in KVS:
        t = TreeCase(kv, 2, 8, 16, [300, 40, 0], [5, 33, 9], "tree", seed=15)
        for dtype in (torch.float32, torch.bfloat16):
            d = t.device()
            want, err = t.run(pda, d, dtype)
            assert err == 0
            d["query"] = d["query"].cpu().pin_memory()
            out = torch.full(want.shape, 7.0, dtype=dtype).pin_memory()
            pda.decode_tree(t.plan(pda), **d, out=out)
            torch.cuda.synchronize()
            assert torch.equal(out, want.cpu())


def test_two_calls_at_once(pda):
    """On two streams, each with a workspace of its own."""
    cases = [TreeCase(kv, 8, 8, 16, [2000] * 20, [4, 33] * 10, "tree", seed=16 + kv) for kv in (BF16, FP8)]
    ds, plans = [t.device() for t in cases], [t.plan(pda) for t in cases]
    want = [t.run(pda, d)[0] for t, d in zip(cases, ds)]
    wss = [pda.tree_workspace(p, t.N, "cuda") for p, t in zip(plans, cases)]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, d, ws, out, s in zip(plans, ds, wss, outs, streams):
            pda.decode_tree(p, **d, ws=ws, out=out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("kv", KVS)
def test_pools_past_4_gb(pda, kv):
    """Block offsets past 32 bits: the same blocks at a large pool's end."""
    t = TreeCase(kv, 8, 8, 32, [300, 40, 0], [5, 33, 9], "tree", seed=17)
    d, p = t.device(), t.plan(pda)
    want, err = t.run(pda, d)
    assert err == 0
    size, n = p.cache_block_bytes, d["num_cache_blocks"]
    far = 5 * 10 ** 9 // size
    big = torch.empty((far + n) * size, dtype=torch.uint8, device="cuda")
    big[far * size:] = d["kv_cache"].view(-1)[:n * size]
    table = d["block_table"]
    d.update(kv_cache=big, num_cache_blocks=far + n, block_table=torch.where(table >= 0, table + far, table))
    out, err = t.run(pda, d)
    assert err == 0 and torch.equal(out, want)
