"""Copying, forking, growing, freeing and compacting pages: exact against the definition."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import oracle_helpers as oh
from tests import plain_pages as pp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def pool(rng, NB, block_bytes):
    return rng.integers(0, 256, NB * block_bytes, dtype=np.uint8)


def batch(rng, lens, BS, MB, NB, shared=0):
    """Tables of a batch whose first `shared` full blocks are common, and the pool's counts."""
    ids, at = rng.permutation(NB).astype(np.int32), 0
    table, refs = np.full((len(lens), MB), -1, np.int32), np.zeros(NB, np.int32)
    common = ids[:shared]
    at = shared
    for b, n in enumerate(lens):
        h = -(-max(int(n), 0) // BS)
        s = min(shared, int(n) // BS)
        table[b, :s] = common[:s]
        table[b, s:h] = ids[at:at + h - s]
        at += h - s
        np.add.at(refs, table[b, :h], 1)
    assert at <= NB
    return table, refs


def run_fork(pda, p, cache, NB, table, lens, refs, parents, grow, extra=3):
    d = dict(cache=dev(cache), table=dev(table), lens=dev(lens), refs=dev(refs))
    R, MB = len(parents), table.shape[1]
    out = dict(table=torch.full((R + extra, MB), 77, dtype=torch.int32, device="cuda"),
               lens=torch.full((R + extra,), 77, dtype=torch.int32, device="cuda"),
               refs=torch.full((NB + extra,), 77, dtype=torch.int32, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pda.page_workspace(p, R, NB, "cuda")
    pda.fork_sequences(p, d["cache"], NB, d["table"], d["lens"], d["refs"], dev(np.asarray(parents, np.int32)),
                       out["table"], out["lens"], out["refs"], ws,
                       new_tokens=None if grow is None else dev(np.asarray(grow, np.int32)), err_word=err)
    torch.cuda.synchronize()
    assert (out["table"][R:] == 77).all() and (out["lens"][R:] == 77).all() and (out["refs"][NB:] == 77).all()
    for k, v in (("table", table), ("lens", lens), ("refs", refs)):
        assert np.array_equal(d[k].cpu().numpy(), v), f"{k} was changed"
    return (d["cache"].cpu().numpy(), out["table"][:R].cpu().numpy(), out["lens"][:R].cpu().numpy(),
            out["refs"][:NB].cpu().numpy(), int(err.item()))


def check_fork(pda, p, cache, NB, table, lens, refs, parents, grow):
    got = run_fork(pda, p, cache, NB, table, lens, refs, parents, grow)
    want = pp.fork(cache, p.cache_block_bytes, p.kv_block_size, table, lens, refs, parents, grow)
    for name, g, w in zip(("cache", "table", "lens", "refs", "error word"), got, want):
        assert np.array_equal(g, w), name
    return got


@pytest.mark.parametrize("kv,BS,Hk", [(wl.KV_BF16, 16, 1), (wl.KV_FP8_E4M3, 16, 3), (wl.KV_TQ4, 16, 1),
                                      (wl.KV_BF16, 32, 5), (wl.KV_TQ4, 32, 7)])
@pytest.mark.parametrize("shared", [0, 3])
def test_fork_of_ragged_rows(pda, kv, BS, Hk, shared):
    rng = np.random.default_rng(BS + Hk + shared)
    lens = np.array([0, 1, BS - 1, BS, BS + 1, 5 * BS, 7 * BS + 3, 4 * BS - 1], np.int32)
    MB, NB = 11, 120
    p = pda.plan(len(lens), Hk, 8, BS, MB, kv_dtype=kv)
    table, refs = batch(rng, lens, BS, MB, NB, shared)
    cache = pool(rng, NB, p.cache_block_bytes)
    B = len(lens)
    for parents, grow in (([*range(B)], None), ([*range(B)], [1] * B), ([6, 6, 6, -1, 2, 7, 7, 1, 0, 4, 4, 2], None),
                          ([7, 3, 3, 6, 6], [0, 1, BS, 2 * BS + 5, 3 * BS]), ([-1, -1], [4, 4]), ([2], [0]),
                          (rng.integers(-1, B, 40), rng.integers(0, BS + 2, 40))):
        assert check_fork(pda, p, cache, NB, table, lens, refs, parents, grow)[4] & ~pp.NO_BLOCKS == 0


def test_fork_copies_a_partial_block_that_something_else_holds(pda):
    rng = np.random.default_rng(1)
    lens = np.array([20, 16], np.int32)
    p = pda.plan(2, 1, 8, 16, 4)
    table, refs = batch(rng, lens, 16, 4, 12)
    cache = pool(rng, 12, p.cache_block_bytes)
    refs[table[0, 1]] += 1                                   # a prefix cache keeps the partial block too
    out = check_fork(pda, p, cache, 12, table, lens, refs, [0, 1], None)
    assert out[1][0, 1] != table[0, 1] and out[3][table[0, 1]] == 1


@pytest.mark.parametrize("NB", [5, 1023, 8192, 8193, 40001])
def test_fork_and_compact_over_pool_sizes(pda, NB):
    # one scan CTA up to 8192 blocks, a cluster above; odd pools; many free and many used blocks
    rng = np.random.default_rng(NB)
    p = pda.plan(3, 1, 8, 16, 64, kv_dtype=wl.KV_TQ4)
    lens = np.minimum(np.array([min(1000, NB // 3 * 16), 7, 0]), NB // 4 * 16).astype(np.int32)
    table, refs = batch(rng, lens, 16, 64, NB)
    others = rng.permutation(np.flatnonzero(refs == 0))      # blocks of another batch, spread over the pool
    refs[others[:len(others) // 2]] = rng.integers(1, 4, len(others) // 2)
    cache = pool(rng, NB, p.cache_block_bytes)
    check_fork(pda, p, cache, NB, table, lens, refs, [0, 0, 1, 2], [3, 0, 30, 5])
    check_compact(pda, p, cache, NB, table, lens, refs)


def test_fork_with_too_few_blocks_leaves_the_old_batch_valid(pda):
    rng = np.random.default_rng(2)
    lens = np.array([33, 40, 5], np.int32)
    p = pda.plan(3, 2, 8, 16, 8)
    table, refs = batch(rng, lens, 16, 8, 9)                 # 7 blocks used, 2 free
    cache = pool(rng, 9, p.cache_block_bytes)
    got = check_fork(pda, p, cache, 9, table, lens, refs, [0, 0, 1, 1, 2, 2], None)
    assert got[4] == pp.NO_BLOCKS and list(got[2]) == [33, 33, 40, 40, 5, 0]
    used = refs > 0
    assert np.array_equal(got[0].reshape(9, -1)[used], cache.reshape(9, -1)[used])


def test_a_first_child_without_blocks_is_not_an_heir(pda):
    # row 0 would inherit the sequence's blocks but asks for more than there are; row 1 shares them
    # and their counts stay
    rng = np.random.default_rng(3)
    lens = np.array([32], np.int32)
    p = pda.plan(1, 1, 8, 16, 8)
    table, refs = batch(rng, lens, 16, 8, 5)
    cache = pool(rng, 5, p.cache_block_bytes)
    got = check_fork(pda, p, cache, 5, table, lens, refs, [0, 0], [90, 0])
    assert list(got[2]) == [0, 32] and np.array_equal(got[3], refs)
    got = check_fork(pda, p, cache, 5, table, lens, refs, [0, -1], [90, 0])
    assert list(got[2]) == [0, 0] and not got[3].any()


def test_fork_data_errors(pda):
    rng = np.random.default_rng(4)
    lens = np.array([20, 30, 999, 17], np.int32)             # 999 > 8 * 16
    p = pda.plan(4, 1, 8, 16, 8)
    table, refs = batch(rng, np.array([20, 30, 0, 17]), 16, 8, 30)
    cache = pool(rng, 30, p.cache_block_bytes)
    t = table.copy()
    t[1, 0], t[1, 1] = -5, 1 << 30                           # full and partial block outside the pool
    got = check_fork(pda, p, cache, 30, t, lens, refs, [0, 1, 1, 2, 3, 4, 1 << 30, 0, 0], [0, 0, 1, 2, 200, 0, 0, -1, 108])
    assert got[4] == pp.BAD_LEN | pp.BAD_ID | pp.BAD_POS | pp.BAD_SEQ


def test_fork_of_many_rows(pda):
    rng = np.random.default_rng(5)
    B, R, MB, NB = 37, 2500, 3, 4000                         # more rows than one pass of the scan's CTA
    lens = rng.integers(0, 48, B).astype(np.int32)
    p = pda.plan(B, 1, 6, 16, MB, kv_dtype=wl.KV_TQ4)
    table, refs = batch(rng, lens, 16, MB, NB)
    cache = pool(rng, NB, p.cache_block_bytes)
    check_fork(pda, p, cache, NB, table, lens, refs, rng.integers(-2, B, R), rng.integers(0, 3, R))


def check_compact(pda, p, cache, NB, table, lens, refs):
    d = dict(cache=dev(cache), table=dev(table), lens=dev(lens), refs=dev(refs))
    full = lambda n: torch.full(n if isinstance(n, tuple) else (n,), 77, dtype=torch.int32, device="cuda")
    out_table, out_refs, remap, used = full(table.shape), full(NB + 2), full(NB + 2), full(2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pda.page_workspace(p, 0, NB, "cuda")
    pda.compact_blocks(p, d["cache"], NB, d["table"], d["lens"], d["refs"], out_table, out_refs, remap, used, ws,
                       err_word=err)
    torch.cuda.synchronize()
    want = pp.compact(cache, p.cache_block_bytes, p.kv_block_size, table, lens, refs)
    got = (d["cache"].cpu().numpy(), out_table.cpu().numpy(), out_refs[:NB].cpu().numpy(), remap[:NB].cpu().numpy(),
           int(used[0]), int(err.item()))
    for name, g, w in zip(("cache", "table", "refs", "remap", "used", "error word"), got, want):
        assert np.array_equal(g, w), name
    assert (out_refs[NB:] == 77).all() and (remap[NB:] == 77).all() and used[1] == 77
    assert np.array_equal(d["refs"].cpu().numpy(), refs) and np.array_equal(d["table"].cpu().numpy(), table)
    return got


@pytest.mark.parametrize("kv,BS,Hk", [(wl.KV_BF16, 16, 2), (wl.KV_FP8_E4M3, 32, 3), (wl.KV_TQ4, 16, 1)])
def test_compact(pda, kv, BS, Hk):
    rng = np.random.default_rng(BS + Hk)
    lens = np.array([0, 1, 5 * BS, 3 * BS + 1, 8 * BS], np.int32)
    p = pda.plan(len(lens), Hk, 8, BS, 8, kv_dtype=kv)
    for NB in (18, 40, 300):                                 # 18: every block used, nothing moves
        table, refs = batch(rng, lens, BS, 8, NB)
        check_compact(pda, p, pool(rng, NB, p.cache_block_bytes), NB, table, lens, refs)
    empty = np.zeros(300, np.int32)
    assert check_compact(pda, p, pool(rng, 300, p.cache_block_bytes), 300, table, np.zeros(5, np.int32), empty)[4] == 0


def test_compact_data_errors(pda):
    rng = np.random.default_rng(6)
    lens = np.array([40, -3, 20], np.int32)
    p = pda.plan(3, 1, 8, 16, 4)
    table, refs = batch(rng, np.array([40, 0, 20]), 16, 4, 50)
    table[0, 1], table[2, 0] = 1 << 29, np.flatnonzero(refs == 0)[0]      # outside the pool; a free block
    got = check_compact(pda, p, pool(rng, 50, p.cache_block_bytes), 50, table, lens, refs)
    assert got[5] == pp.BAD_LEN | pp.BAD_ID


@pytest.mark.parametrize("kv,BS,Hk,n", [(wl.KV_BF16, 16, 1, 1), (wl.KV_TQ4, 16, 1, 7), (wl.KV_FP8_E4M3, 32, 5, 60),
                                        (wl.KV_BF16, 32, 4, 150)])
def test_copy(pda, kv, BS, Hk, n):
    rng = np.random.default_rng(n)
    p = pda.plan(1, Hk, 8, BS, 1, kv_dtype=kv)
    cbb, NB = p.cache_block_bytes, 2 * n + 5
    src, dst = pool(rng, NB, cbb), pool(rng, NB - 1, cbb)
    pairs = np.stack([rng.integers(0, NB, n), rng.permutation(NB - 1)[:n]], 1).astype(np.int32)   # sources repeat
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for host in (None, "src", "dst"):
        s, d = dev(src), dev(dst)
        if host == "src":
            s = torch.from_numpy(src).pin_memory()
        if host == "dst":
            d = torch.from_numpy(dst.copy()).pin_memory()
        pda.copy_blocks(p, s, NB, d, NB - 1, dev(pairs), err_word=err)
        torch.cuda.synchronize()
        want, _ = pp.copy(src, dst, pairs, cbb, False)
        assert np.array_equal(d.cpu().numpy(), want) and int(err.item()) == 0
    ids = rng.permutation(NB)                                # within one pool
    inside = np.stack([ids[:n], ids[n:2 * n]], 1).astype(np.int32)
    s = dev(src)
    pda.copy_blocks(p, s, NB, s, NB, dev(inside))
    assert np.array_equal(s.cpu().numpy(), pp.copy(src, src, inside, cbb, True)[0])


def test_copy_data_errors(pda):
    rng = np.random.default_rng(7)
    p = pda.plan(1, 1, 8, 16, 1)
    src, dst = pool(rng, 4, p.cache_block_bytes), pool(rng, 3, p.cache_block_bytes)
    pairs = np.array([[0, 1], [-1, 0], [2, -7], [4, 0], [1, 3], [1 << 30, 1 << 30]], np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = dev(dst)
    pda.copy_blocks(p, dev(src), 4, d, 3, dev(pairs), err_word=err)
    want, e = pp.copy(src, dst, pairs, p.cache_block_bytes, False)
    assert np.array_equal(d.cpu().numpy(), want) and int(err.item()) == e == pp.BAD_ID
    pda.copy_blocks(p, dev(src), 4, d, 3, dev(np.zeros((0, 2), np.int32)), err_word=err)     # nothing to do
    assert np.array_equal(d.cpu().numpy(), want)


def test_blocks_past_4_gib(pda):
    # ids whose byte offsets need 64 bits, in all three operations
    p = pda.plan(1, 8, 8, 32, 2)
    cbb = p.cache_block_bytes                                # 128 KB
    NB = (5 << 30) // cbb
    cache = torch.empty(NB * cbb, dtype=torch.uint8, device="cuda")
    blocks = cache.view(NB, cbb)
    blocks[:8].random_(0, 256)
    blocks[-8:].random_(0, 256)
    last = blocks[NB - 1].clone()
    pda.copy_blocks(p, cache, NB, cache, NB, torch.tensor([[NB - 1, NB - 3]], dtype=torch.int32, device="cuda"))
    assert torch.equal(blocks[NB - 3], last)
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    refs[NB - 1] = 1
    table = torch.tensor([[NB - 1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    ws = pda.page_workspace(p, 2, NB, "cuda")
    out_t, out_l, out_r = torch.empty((2, 2), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(refs)
    refs[:NB - 2] = 1                                        # only block NB - 2 is free
    pda.fork_sequences(p, cache, NB, table, lens, refs, torch.zeros(2, dtype=torch.int32, device="cuda"), out_t, out_l, out_r, ws)
    assert out_t[:, 0].tolist() == [NB - 1, NB - 2] and torch.equal(blocks[NB - 2], last)
    refs.zero_()
    refs[NB - 1] = 3
    remap, used = torch.empty_like(refs), torch.empty(1, dtype=torch.int32, device="cuda")
    pda.compact_blocks(p, cache, NB, table, lens, refs, out_t[:1], out_r, remap, used, ws)
    assert torch.equal(blocks[0], last) and out_t[0, 0] == 0 and out_r[0] == 3 and int(used) == 1


def test_fork_append_decode_together(oracle_mod, pda):
    """A serving step as it is used: two beams fork and grow by one token, both append their own
    token, decode, are compacted, and decode the same."""
    w = wl.small(num_seqs=3, num_kv_heads=2, ctx=(37, 50, 16), seed=91, max_blocks_per_seq=6, extra_blocks=12)
    inp = wl.generate(w)
    refs = np.zeros(w.num_cache_blocks, np.int32)
    for b, n in enumerate(inp.context_lens):
        refs[inp.block_table[b, :-(-int(n) // 16)]] += 1
    p3 = pda.plan(3, 2, 8, 16, 6)
    parents, R = np.array([1, 0, 0, 1], np.int32), 4
    cache = dev(inp.cache)
    lens, table = dev(inp.context_lens), dev(inp.block_table)
    out_t, out_l = torch.empty((R, 6), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    out_r = torch.empty(w.num_cache_blocks, dtype=torch.int32, device="cuda")
    ws = pda.page_workspace(p3, R, w.num_cache_blocks, "cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p4 = pda.plan(R, 2, 8, 16, 6)
    rng = np.random.default_rng(8)
    k, v = (rng.standard_normal((R, 2, 128)).astype(np.float32) for _ in range(2))
    q = wl.round_bf16(rng.standard_normal((R, 16, 128)).astype(np.float32))
    as_bf16 = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    NB = w.num_cache_blocks
    pda.fork_sequences(p3, cache, NB, table, lens, dev(refs), dev(parents), out_t, out_l, out_r, ws,
                       new_tokens=torch.ones(R, dtype=torch.int32, device="cuda"), err_word=err)
    pda.append_kv(p4, as_bf16(wl.round_bf16(k)), as_bf16(wl.round_bf16(v)), cache, NB, out_t, out_l - 1, err_word=err)
    out = pda.decode_step(p4, as_bf16(q), cache, NB, out_t, out_l, out_dtype=torch.float32, err_word=err)
    t2, r2, remap, used = torch.empty_like(out_t), torch.empty_like(out_r), torch.empty_like(out_r), torch.empty(1, dtype=torch.int32, device="cuda")
    pda.compact_blocks(p4, cache, NB, out_t, out_l, out_r, t2, r2, remap, used, ws, err_word=err)
    again = pda.decode_step(p4, as_bf16(q), cache, int(used), t2, out_l, out_dtype=torch.float32, err_word=err)
    assert int(err.item()) == 0 and torch.equal(out, again)
    kst, vst = pp.block_values(w, inp.cache)
    for r, pa in enumerate(parents):
        n = int(inp.context_lens[pa])
        ids = inp.block_table[pa, :-(-n // 16)]
        for h in range(2):
            kk = np.concatenate([kst[ids, :, h].reshape(-1, 128)[:n], wl.bf16_bits_to_f32(wl.round_bf16(k[r, h]))[None]])
            vv = np.concatenate([vst[ids, :, h].reshape(-1, 128)[:n], wl.bf16_bits_to_f32(wl.round_bf16(v[r, h]))[None]])
            ref = pp.attention(wl.bf16_bits_to_f32(q[r, 8 * h:8 * h + 8]).astype(np.float64), kk, vv, 128 ** -0.5)
            assert np.abs(out[r, 8 * h:8 * h + 8].cpu().numpy() - ref).max() <= 2e-3     # the library's bf16 bound


def test_fork_in_a_graph_and_on_another_stream(pda):
    rng = np.random.default_rng(9)
    lens = np.array([20, 37], np.int32)
    p = pda.plan(2, 1, 8, 16, 4)
    table, refs = batch(rng, lens, 16, 4, 12)
    cache = pool(rng, 12, p.cache_block_bytes)
    d = dict(cache=dev(cache), table=dev(table), lens=dev(lens), refs=dev(refs), par=dev(np.array([1, 1, 0], np.int32)))
    ot, ol, orf = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((3, 4), (3,), (12,)))
    ws = pda.page_workspace(p, 3, 12, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pda.fork_sequences(p, d["cache"], 12, d["table"], d["lens"], d["refs"], d["par"], ot, ol, orf, ws)
    for par in ([1, 1, 0], [0, 0, 0], [-1, 1, 1]):           # the captured step follows what it reads
        d["cache"].copy_(torch.from_numpy(cache))
        d["par"].copy_(torch.tensor(par, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = pp.fork(cache, p.cache_block_bytes, 16, table, lens, refs, par, None)
        for a, b in zip((d["cache"], ot, ol, orf), want):
            assert np.array_equal(a.cpu().numpy(), b)
    with torch.cuda.stream(s):
        pda.fork_sequences(p, d["cache"], 12, d["table"], d["lens"], d["refs"], d["par"], ot, ol, orf, ws, stream=s)
    s.synchronize()
    assert np.array_equal(ot.cpu().numpy(), want[1])


def test_fork_into_nothing_frees_everything_and_from_nothing_stays_empty(pda):
    rng = np.random.default_rng(11)
    lens = np.array([20, 37], np.int32)
    p = pda.plan(2, 1, 8, 16, 4)
    table, refs = batch(rng, lens, 16, 4, 12)
    cache = pool(rng, 12, p.cache_block_bytes)
    assert not check_fork(pda, p, cache, 12, table, lens, refs, [], None)[3].any()
    p0 = pda.plan(0, 1, 8, 16, 4)
    got = check_fork(pda, p0, cache, 12, np.zeros((0, 4), np.int32), np.zeros(0, np.int32), refs, [-1, -1], [5, 0])
    assert not got[2].any() and np.array_equal(got[3], refs)


def test_two_forks_at_once_with_workspaces_of_their_own(pda):
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 200, 40).astype(np.int32)
    p = pda.plan(40, 2, 8, 16, 16)
    sides = []
    for k in range(2):
        table, refs = batch(rng, lens, 16, 16, 900)
        sides.append(dict(cache=pool(rng, 900, p.cache_block_bytes), table=table, refs=refs, par=rng.integers(-1, 40, 50).astype(np.int32),
                          s=torch.cuda.Stream(), ws=pda.page_workspace(p, 50, 900, "cuda"),
                          out=[torch.empty(n, dtype=torch.int32, device="cuda") for n in ((50, 16), (50,), (900,))]))
    dv = [{k: dev(x[k]) for k in ("cache", "table", "refs", "par")} for x in sides]
    L = dev(lens)
    torch.cuda.synchronize()
    for _ in range(10):
        for x, d in zip(sides, dv):
            pda.fork_sequences(p, d["cache"], 900, d["table"], L, d["refs"], d["par"], *x["out"], x["ws"], stream=x["s"])
    torch.cuda.synchronize()
    for x, d in zip(sides, dv):
        want = pp.fork(x["cache"], p.cache_block_bytes, 16, x["table"], lens, x["refs"], x["par"], None)
        for a, b in zip((d["cache"], *x["out"]), want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_the_binding_refuses(pda):
    p = pda.plan(2, 1, 8, 16, 4)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    cache = torch.zeros(12 * p.cache_block_bytes, dtype=torch.uint8, device="cuda")
    ws = pda.page_workspace(p, 3, 12, "cuda")
    good = dict(kv_cache=cache, num_cache_blocks=12, block_table=i32(2, 4), context_lens=i32(2), refcounts=i32(12), parents=i32(3),
                out_table=i32(3, 4), out_lens=i32(3), out_refcounts=i32(12), workspace=ws)
    pda.fork_sequences(p, **good)
    for name, bad, what in (("block_table", i32(8, 2).t(), "contiguous"), ("block_table", i32(7), "too small"),
                            ("parents", i32(3).long(), "dtype"), ("out_refcounts", i32(12).cpu(), "cuda:0"),
                            ("kv_cache", cache[:-1], "too small"), ("context_lens", None, "CUDA tensor")):
        with pytest.raises(ValueError, match=what):
            pda.fork_sequences(p, **{**good, name: bad})
    for name, bad, status in (("workspace", ws[:-16], -3), ("workspace", torch.cat([ws, ws])[8:], -1), ("out_table", good["block_table"], None),
                              ("out_refcounts", good["refcounts"], -1)):
        with pytest.raises((pda.PdaError, ValueError)) as e:
            pda.fork_sequences(p, **{**good, name: bad})
        assert status is None or e.value.status == status
    with pytest.raises(ValueError, match="pair"):
        pda.copy_blocks(p, cache, 12, cache, 12, i32(3))
    with pytest.raises(pda.PdaError):
        pda.copy_blocks(p, cache, 6, cache[5 * p.cache_block_bytes:], 6, i32(1, 2))      # pools that overlap
