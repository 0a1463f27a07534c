"""Many tokens per sequence written into the cache and read back, against the generator's quantisers bit for bit, and the
accepted paths of drafted tokens."""
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


def rows(rng, n, Hk):
    """K, V [n][Hk][128] as bf16 values: of all sizes, with rows of zeros, of one value, and of one large among small."""
    x = rng.standard_normal((2, n, Hk, 128)) * np.exp(2 * rng.standard_normal((2, n, Hk, 1)))
    kind = rng.integers(0, 12, (2, n, Hk))
    x[kind == 0] = 0
    x[kind == 1] = 1.5
    x[kind == 2, 5] = 300
    x[kind == 3] *= 1e-4
    bits = wl.round_bf16(x.astype(np.float32))
    return wl.bf16_bits_to_f32(bits), bits


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def setup(pda, kv, Hk, BS, positions, counts, seed=0, before=0, after=0, MB=None):
    """A pool with the sequences' blocks, new tokens of each from its position on, and rows of nobody around them."""
    total = [max(0, p) + n for p, n in zip(positions, counts)]
    c = pt.Pool(kv, Hk, 8, BS, total, seed=seed, MB=MB)
    c.starts = before + np.concatenate([[0], np.cumsum(counts)])
    c.N = int(c.starts[-1]) + after
    c.positions = list(positions)
    c.x, c.bits = rows(c.rng, c.N, Hk)
    c.p = pda.plan(c.B, Hk, 8, BS, c.MB, kv_dtype=kv)
    c.cent = None if c.book is None else torch.from_numpy(c.book).cuda()
    return c


def places(c, b):
    n = int(c.starts[b + 1] - c.starts[b])
    t = c.positions[b] + np.arange(n)
    return c.table[b, t // c.BS], t % c.BS


def expected_write(c):
    cache = c.cache.copy()
    data, fields = pt.quantised(c.kv, c.x[0], c.x[1], c.book)
    for b in range(c.B):
        if c.positions[b] >= 0 and c.starts[b + 1] > c.starts[b]:
            r = slice(c.starts[b], c.starts[b + 1])
            pt.store(c.w, cache, *places(c, b), data[r], None if fields is None else fields[r])
    return cache


def write(pda, c, cache, k=None, v=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pda.write_kv(c.p, bf16(c.bits[0]) if k is None else k, bf16(c.bits[1]) if v is None else v, cache, c.NB,
                 kw.pop("table", i32(c.table)), kw.pop("starts", i32(c.starts)), kw.pop("positions", i32(c.positions)),
                 centroids=c.cent, err_word=err, **kw)
    torch.cuda.synchronize()
    return int(err.item())


SHAPES = [   # Hk, BS, positions, counts, rows before, rows after
    (1, 16, [0], [1], 0, 0),
    (8, 16, [5, 0, 100, 31, 7], [3, 16, 1, 0, 33], 0, 0),
    (5, 32, [0, 1, 15, 16, 17, 31, 32, 33], [64, 1, 2, 16, 17, 1, 1, 95], 0, 0),
    (4, 32, [0, -1, 40, -7], [7, 5, 9, 2], 3, 4),
    (2, 16, [1000, 0], [700, 1300], 0, 17),
    (3, 16, list(range(70)), [i % 4 for i in range(70)], 2, 0),
]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("Hk,BS,positions,counts,before,after", SHAPES)
def test_bytes_are_the_quantisers(pda, kv, Hk, BS, positions, counts, before, after):
    c = setup(pda, kv, Hk, BS, positions, counts, seed=len(counts), before=before, after=after)
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    assert np.array_equal(cache.cpu().numpy(), expected_write(c))


@pytest.mark.parametrize("kv", KVS)
def test_a_token_has_the_bytes_of_the_single_token_call(pda, kv):
    """bf16 and fp8: pda_append_kv's.  TQ4, which that call refuses: those of a write of its own."""
    c = setup(pda, kv, 8, 16, [9, 0, 33], [1, 1, 1], seed=5)
    one, many = (torch.from_numpy(c.cache).cuda() for _ in range(2))
    assert write(pda, c, many) == 0
    if kv == TQ4:
        for b in range(c.B):
            starts = np.where(np.arange(c.B + 1) > b, c.starts[b + 1], c.starts[b])
            assert write(pda, c, one, starts=i32(starts)) == 0
    else:
        pda.append_kv(c.p, bf16(c.bits[0]), bf16(c.bits[1]), one, c.NB, i32(c.table), i32(c.positions))
        torch.cuda.synchronize()
    assert torch.equal(one, many)


@pytest.mark.parametrize("kv", KVS)
def test_rows_of_a_fused_projection(pda, kv):
    """K and V as column ranges of wider rows, and K behind V in memory."""
    c = setup(pda, kv, 4, 16, [3, 20], [18, 5], seed=2)
    wide = torch.full((c.N, 4 * 3 + 1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 9:13], wide[:, 2:6] = bf16(c.bits[0]), bf16(c.bits[1])
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache, wide[:, 9:13], wide[:, 2:6]) == 0
    assert np.array_equal(cache.cpu().numpy(), expected_write(c))


@pytest.mark.parametrize("order", ["descending", "shuffled"])
def test_a_codebook_in_any_order(pda, order):
    c = setup(pda, TQ4, 2, 16, [0], [40], seed=3)
    perm = np.arange(16)[::-1].copy() if order == "descending" else np.random.default_rng(1).permutation(16)
    kc, _ = pt.tq4_keys(c.x[0], c.book)
    code_of = np.argsort(perm)                       # the given book is book[perm]: sorted code i is its index code_of[i]
    want = c.cache.copy()
    data, fields = pt.quantised(TQ4, c.x[0], c.x[1], c.book)
    data[:, :, 0] = wl.pack_nibbles(code_of[kc].astype(np.uint8))
    pt.store(c.w, want, *places(c, 0), data, fields)
    c.cent = torch.from_numpy(np.ascontiguousarray(c.book[perm])).cuda()
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    assert np.array_equal(cache.cpu().numpy(), want)


def test_norms_next_to_a_border_of_f16(pda):
    """Rows whose norm lies within 2^-22 of the middle between two f16 values: only the exact sum of squares decides."""
    rng = np.random.default_rng(7)
    found = []
    while len(found) < 24:
        x = wl.bf16_bits_to_f32(wl.round_bf16(rng.standard_normal((20000, 128)).astype(np.float32)))
        norm = np.sqrt((x.astype(np.float64) ** 2).sum(-1))
        f = norm.astype(np.float16).astype(np.float64)
        half = 2.0 ** (np.floor(np.log2(norm)) - 11)
        found += list(x[np.abs(np.abs(norm - f) / half - 1) < 2.0 ** -10])
    x = np.array(found[:24], np.float32).reshape(24, 1, 128)
    c = setup(pda, TQ4, 1, 16, [0], [24], seed=1)
    c.x = np.stack([x, x])
    c.bits = wl.round_bf16(c.x)
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    assert np.array_equal(cache.cpu().numpy(), expected_write(c))


def test_tq4_values_past_f16(pda):
    """Norms and ranges past f16's are kept at 65504."""
    c = setup(pda, TQ4, 1, 16, [0], [4], seed=1)
    x = np.ones((4, 1, 128), np.float32)
    x[0] *= 1e30
    x[1, 0, ::2] = -1e6
    x[2] *= 60000
    x[3, 0, 0] = 3e38
    c.x, c.bits = np.stack([x, x]), wl.round_bf16(np.stack([x, x]))
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    _, meta = wl.cache_views(c.w, cache.cpu().numpy())
    f = meta[c.table[0, 0], 0, :, :4].view(np.float16).astype(np.float64)
    assert np.isfinite(f).all()
    assert f[0].tolist() == [65504] * 4
    assert f[1].tolist() == [0, 65504, 0, 65504] and f[2, 0] == 65504 and f[2, 1] == -65504


# ---------------------------------------------------------------------------- reading
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("Hk,BS,positions,counts,before,after", SHAPES)
def test_values_come_back(pda, kv, dtype, Hk, BS, positions, counts, before, after):
    c = setup(pda, kv, Hk, BS, positions, counts, seed=len(counts), before=before, after=after)
    out = [torch.full((c.N, Hk, 128), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c.p, torch.from_numpy(c.cache).cuda(), c.NB, i32(c.table), i32(c.starts), i32(c.positions))
    pda.read_kv(*args, *out, centroids=c.cent, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want = np.full((2, c.N, Hk, 128), 7.0)
    for b in range(c.B):
        if c.positions[b] >= 0:
            for h in range(Hk):
                k, v, _, _ = pt.token_values(c.w, c.cache, *places(c, b), h, c.book)
                want[0, c.starts[b]:c.starts[b + 1], h], want[1, c.starts[b]:c.starts[b + 1], h] = k, v
    want = torch.from_numpy(want).float().to(dtype)      # one fp32 product, or one sum: rounded once, then to the type
    for w in range(2):
        assert torch.equal(out[w].cpu(), want[w])
    alone = [torch.full((c.N, Hk, 128), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    pda.read_kv(*args, alone[0], None, centroids=c.cent)
    pda.read_kv(*args, None, alone[1], centroids=c.cent)
    assert torch.equal(alone[0], out[0]) and torch.equal(alone[1], out[1])


# ---------------------------------------------------------------------------- data errors
def test_data_errors_move_nothing_of_the_row(pda):
    for kv in KVS:
        c = setup(pda, kv, 2, 16, [0, 30, 5, 2], [20, 4, 20, 3], seed=9, MB=3)
        c.table[2, 1] = c.NB              # block ids outside the pool: positions 16 .. 24 of sequence 2
        c.table[3, 0] = -5
        c.positions[1] = 45               # rows 45 .. 47 fit, 48 does not
        good = expected_rows(c)
        cache = torch.from_numpy(c.cache).cuda()
        assert write(pda, c, cache) == pda.ERRW_BAD_BLOCK_ID | pda.ERRW_BAD_POSITION
        assert np.array_equal(cache.cpu().numpy(), good)
        out = torch.full((c.N, 2, 128), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pda.read_kv(c.p, cache, c.NB, i32(c.table), i32(c.starts), i32(c.positions), out, None, centroids=c.cent, err_word=err)
        assert int(err.item()) == pda.ERRW_BAD_BLOCK_ID | pda.ERRW_BAD_POSITION
        kept = (out == 7.0).all(-1).all(-1).cpu().numpy()
        assert kept[[23, 24 + 11, 24 + 19, 44, 46]].all() and not kept[[0, 19, 22, 24, 24 + 10]].any()


def expected_rows(c):
    """As expected_write, row by row, without those that have no place."""
    cache = c.cache.copy()
    data, fields = pt.quantised(c.kv, c.x[0], c.x[1], c.book)
    for b in range(c.B):
        for i in range(c.starts[b], c.starts[b + 1]):
            t = c.positions[b] + i - c.starts[b]
            if t < c.MB * c.BS and 0 <= c.table[b, t // c.BS] < c.NB:
                pt.store(c.w, cache, [c.table[b, t // c.BS]], [t % c.BS], data[i:i + 1], None if fields is None else fields[i:i + 1])
    return cache


@pytest.mark.parametrize("starts", [[0, 5, 4, 9], [-1, 2, 4, 9], [0, 2, 4, 10], [3, 2, 2, 2], [9, 9, 9, 8]])
def test_starts_that_do_not_ascend(pda, starts):
    for kv in KVS:
        c = setup(pda, kv, 2, 16, [0, 0, 0], [4, 4, 1], seed=4)
        cache = torch.from_numpy(c.cache).cuda()
        assert write(pda, c, cache, starts=i32(starts)) == pda.ERRW_BAD_TOKENS
        assert np.array_equal(cache.cpu().numpy(), c.cache)
        out = torch.full((c.N, 2, 128), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pda.read_kv(c.p, cache, c.NB, i32(c.table), i32(starts), i32(c.positions), out, out.clone(), centroids=c.cent, err_word=err)
        assert int(err.item()) == pda.ERRW_BAD_TOKENS and bool((out == 7.0).all())


def test_many_sequences_and_none(pda):
    c = setup(pda, FP8, 1, 16, [i % 50 for i in range(3000)], [i % 3 for i in range(3000)], seed=6)
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    assert np.array_equal(cache.cpu().numpy(), expected_write(c))
    empty = pda.plan(0, 1, 8, 16, 4, kv_dtype=FP8)
    pda.write_kv(empty, bf16(c.bits[0]), bf16(c.bits[1]), cache, c.NB, i32([]), i32([0]), i32([]))
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    pda.write_kv(c.p, none, none, cache, c.NB, i32(c.table), i32(np.zeros(3001)), i32(c.positions))
    pda.read_kv(c.p, cache, c.NB, i32(c.table), i32(np.zeros(3001)), i32(c.positions), none, none)
    torch.cuda.synchronize()
    assert np.array_equal(cache.cpu().numpy(), expected_write(c))


def test_pools_past_4_gb(pda):
    """Block offsets past 32 bits, in all three calls."""
    BS, Hk, NB = 32, 8, 36000                                # 131 KB per block: 4.7 GB
    p = pda.plan(1, Hk, 8, BS, 4)
    cache = torch.zeros(NB * p.cache_block_bytes, dtype=torch.uint8, device="cuda")
    table = i32([[35999, 3, 35000, 34000]])
    rng = np.random.default_rng(0)
    _, bits = rows(rng, 100, Hk)
    pda.write_kv(p, bf16(bits[0]), bf16(bits[1]), cache, NB, table, i32([0, 100]), i32([20]))
    k, v = (torch.zeros(100, Hk, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pda.read_kv(p, cache, NB, table, i32([0, 100]), i32([20]), k, v)
    assert torch.equal(k, bf16(bits[0])) and torch.equal(v, bf16(bits[1]))
    lens = i32([0])
    pda.accept_tokens(p, cache, NB, table, i32([20]), i32([[3, 40, 99]]), i32([3]), lens)
    pda.read_kv(p, cache, NB, table, i32([0, 3]), i32([20]), k, v)
    assert torch.equal(k[:3], bf16(bits[0][[3, 40, 99]])) and torch.equal(v[:3], bf16(bits[1][[3, 40, 99]]))
    assert lens.item() == 23


# ---------------------------------------------------------------------------- accepting
def accept_case(pda, kv, Hk, BS, lens, paths, A=None, seed=0, MB=None):
    total = [n + (max(p) + 1 if p else 0) for n, p in zip(lens, paths)]
    c = pt.Pool(kv, Hk, 8, BS, total, seed=seed, MB=MB)
    c.lens, c.paths = list(lens), paths
    c.A = max([1] + [len(p) for p in paths]) if A is None else A
    c.path = np.full((c.B, c.A), -1, np.int32)
    for b, p in enumerate(paths):
        c.path[b, :len(p)] = p
    c.p = pda.plan(c.B, Hk, 8, BS, c.MB, kv_dtype=kv)
    return c


def accept(pda, c, path_lens=None, **kw):
    cache = torch.from_numpy(c.cache).cuda()
    out = torch.full((c.B,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pda.accept_tokens(c.p, cache, c.NB, i32(c.table), i32(c.lens), i32(c.path),
                      i32([len(p) for p in c.paths] if path_lens is None else path_lens), out, err_word=err)
    torch.cuda.synchronize()
    return cache.cpu().numpy(), out.tolist(), int(err.item())


def expected_accept(c):
    cache = c.cache.copy()
    data, meta = wl.cache_views(c.w, c.cache)
    d2, m2 = wl.cache_views(c.w, cache)
    for b, p in enumerate(c.paths):
        for k, j in enumerate(p):
            s, t = c.lens[b] + j, c.lens[b] + k
            (i0, s0), (i1, s1) = ((c.table[b, x // c.BS], x % c.BS) for x in (s, t))
            d2[i1, s1] = data[i0, s0]
            if meta is not None:
                m2[i1, :, :, s1] = meta[i0, :, :, s0]
    return cache


PATHS = [
    (8, 16, [100, 0, 15, 31], [[0, 2, 5], [1], [], [0, 1, 2, 3]]),
    (1, 32, [0], [[63]]),
    (5, 16, [7], [[0, 1, 2, 9, 10, 11, 12, 13, 14, 15, 16, 30]]),
    (2, 32, [33, 1, 62], [list(range(1, 300, 2)), list(range(40)), [5, 6, 7, 40]]),       # longer than a chunk of the kernel
    (40, 16, [17], [[1, 3, 5, 6]]),                                                        # more bytes than one CTA's threads
]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("Hk,BS,lens,paths", PATHS)
def test_paths_move(pda, kv, Hk, BS, lens, paths):
    c = accept_case(pda, kv, Hk, BS, lens, paths, seed=len(paths))
    cache, out, err = accept(pda, c)
    assert err == 0 and out == [n + len(p) for n, p in zip(lens, paths)]
    assert np.array_equal(cache, expected_accept(c))


def test_paths_in_error_stay(pda):
    lens = [10, 10, 10, 10, 10, 500, 10]
    paths = [[0, 3], [2, 2], [-1, 4], [1, 5], [0, 2], [0, 1], [1, 2]]
    c = accept_case(pda, FP8, 2, 16, [10] * 7, [[0, 1, 2, 3, 4, 5]] * 7, seed=3, MB=4)
    c.lens, c.paths = lens, paths
    c.path[:] = -1
    for b, p in enumerate(paths):
        c.path[b, :2] = p
    c.path[4, 1] = 54                     # position 64: past the table
    plens = [2, 2, 2, 9, 2, 2, -1]
    cache, out, err = accept(pda, c, plens)
    assert err == pda.ERRW_BAD_TOKENS | pda.ERRW_BAD_POSITION | pda.ERRW_BAD_CONTEXT_LEN
    assert out == [12, 10, 10, 10, 10, 500, 10]
    c.paths = [[0, 3]] + [[]] * 6
    c.lens[5] = 10
    assert np.array_equal(cache, expected_accept(c))


def test_paths_over_bad_blocks(pda):
    c = accept_case(pda, BF16, 2, 16, [14, 3], [[1, 4, 20], [2]], seed=3)
    good = c.table.copy()
    c.table[0, 2] = c.NB + 7              # token 20 of the first: position 34
    cache, out, err = accept(pda, c)
    assert err == pda.ERRW_BAD_BLOCK_ID and out == [17, 4]
    c.table, c.paths = good, [[1, 4], [2]]
    assert np.array_equal(cache, expected_accept(c))


def test_graphs_and_other_streams(pda):
    """Captured, and replayed with the lengths, paths and rows of the next step, on a stream of its own."""
    c = setup(pda, FP8, 4, 16, [10, 40], [6, 9], seed=8)
    cache = torch.from_numpy(c.cache).cuda()
    k, v, pos, starts, table = bf16(c.bits[0]), bf16(c.bits[1]), i32(c.positions), i32(c.starts), i32(c.table)
    path, plens, out = i32([[0, 2, 5], [1, 8, -1]]), i32([3, 2]), i32([0, 0])
    s = torch.cuda.Stream()

    def step(stream=None):
        pda.write_kv(c.p, k, v, cache, c.NB, table, starts, pos, stream=stream)
        pda.accept_tokens(c.p, cache, c.NB, table, pos, path, plens, out, stream=stream)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    want = None
    for shift in (0, 1):
        pos.copy_(i32([10 - shift, 40 - shift]))
        path.copy_(i32([[0, 2, 5 - shift], [1, 8 - shift, -1]]))
        cache.copy_(torch.from_numpy(c.cache))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got, lens = cache.clone(), out.tolist()
        cache.copy_(torch.from_numpy(c.cache))
        torch.cuda.synchronize()
        step(s)
        torch.cuda.synchronize()
        assert torch.equal(cache, got) and lens == out.tolist() == [13 - shift, 42 - shift]
        assert want is None or not torch.equal(got, want)
        want = got


def test_every_quotient_of_e4m3(pda):
    """Rows of scale 1, 3/7, 2^-40, .. and of every bf16 value up to their largest: next to every border of the codes, the smallest
    ones and both zeros among them; rows with infinities, NaN and of the smallest values have the bytes of the single-token call."""
    bits = np.arange(0x10000, dtype=np.uint32)
    finite = bits[(bits & 0x7F80) != 0x7F80].astype(np.uint16)
    rows_ = []
    for top in (448.0, 192.0, 3.0, 1.0, 0.4921875, 2.0 ** -40, 2.0 ** -90, 2.0 ** -100, 2.0 ** -126, 2.0 ** 120):
        big = wl.round_bf16(np.float32([top]))[0]
        vals = finite[(finite & 0x7FFF) <= big]
        near = vals[(vals & 0x7FFF) >= max(0, int(big) - 128 * 22)]       # the others' codes are 0
        near = near[: len(near) // 127 * 127].reshape(-1, 127)
        rows_.append(np.concatenate([np.full((len(near), 1), big, np.uint16), near], 1))
    odd = np.zeros((4, 128), np.uint16)
    odd[0, 3], odd[0, 5] = 0x7F80, 0x3F80          # +inf
    odd[1, 3], odd[1, 5] = 0xFFC1, 0xBF80          # a negative NaN
    odd[2, 7], odd[2, 9] = 0xFF80, 0x7FC0
    odd[3, 1], odd[3, 2] = 0x0001, 0x8000          # the smallest value, and -0
    x = np.concatenate(rows_ + [odd])
    n = len(x)
    c = setup(pda, FP8, 1, 16, [0], [n], seed=1)
    c.bits = np.stack([x.reshape(n, 1, 128), x[::-1].reshape(n, 1, 128)])
    one, many = (torch.from_numpy(c.cache).cuda() for _ in range(2))
    assert write(pda, c, many) == 0
    p = pda.plan(n, 1, 8, 16, c.MB, kv_dtype=FP8)
    table = i32(np.repeat(c.table, n, 0))
    pda.append_kv(p, bf16(c.bits[0]), bf16(c.bits[1]), one, c.NB, table, i32(np.arange(n)))
    torch.cuda.synchronize()
    assert torch.equal(one, many)


def test_zeros_keep_their_sign(pda):
    """Zeros of either sign, and values whose code is a zero, among ordinary ones: the bytes of the single-token call."""
    c = setup(pda, FP8, 8, 16, [3, 0], [40, 21], seed=2)
    kind = c.rng.integers(0, 6, c.bits.shape)
    for k, v in ((0, 0x8000), (1, 0x0000), (2, 0x8001), (3, 0xA000)):     # the last: -2^-63
        c.bits[kind == k] = v
    one, many = (torch.from_numpy(c.cache).cuda() for _ in range(2))
    assert write(pda, c, many) == 0
    n = int(c.starts[-1])
    p = pda.plan(n, 8, 8, 16, c.MB, kv_dtype=FP8)
    owner = np.repeat([0, 1], [40, 21])
    pos = np.concatenate([3 + np.arange(40), np.arange(21)])
    pda.append_kv(p, bf16(c.bits[0]), bf16(c.bits[1]), one, c.NB, i32(c.table[owner]), i32(pos))
    torch.cuda.synchronize()
    assert torch.equal(one, many)
