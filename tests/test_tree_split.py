"""Which rows and tokens the passes over drafted tokens take, and which tiles a window, run on the host (no GPU needed): the
kernels' own code, with a warp of 32 contexts in the place of the GPU's."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import paged_kv_gqa_block_gb300 as pda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("cta", "g", "h", "rt", "seq0", "rows", "len", "step0", "steps", "rot", "slot", "pieces")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("tree") / "tree.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "paged_kv_gqa_block_gb300", "serving"), os.path.join(ROOT, "tests", "host", "tree.cpp"),
                           "-o", so])
    return ctypes.CDLL(so)


def pieces(lib, starts, lens, QG, Hk, MB, BS, P, window, first, ctas, tokens=None):
    NG, cap = len(lens), 200000
    out, scalars = np.zeros((cap, 12), np.int32), np.zeros(5, np.int32)
    starts, lens = np.asarray(starts, np.int32), np.asarray(lens, np.int32)
    ptr = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    n = lib.tree_pieces_of(NG, ptr(starts), ptr(lens), int(starts[-1]) if tokens is None else tokens, QG, Hk, MB, BS, P, window, first,
                           ctas, ptr(out), cap, ptr(scalars))
    assert n >= 0
    return [dict(zip(FIELDS, map(int, r))) for r in out[:n]], [int(x) for x in scalars]


def seen_steps(ctx, n, window, first):
    """The steps of 128 tokens that hold a token which the first drafted token's position leaves visible."""
    start = max(0, ctx + 1 - window) if window else 0
    t = np.arange(ctx + n)
    return sorted(set((t[(t < first) | (t >= start)] // 128).tolist()))


def check(lib, starts, lens, QG, Hk, MB, BS, P, window, first, ctas, err=0):
    units, (e, per, total, whole, refused) = pieces(lib, starts, lens, QG, Hk, MB, BS, P, window, first, ctas)
    assert e == err and not refused
    want = {}
    for g, ctx in enumerate(lens):
        n = int(starts[g + 1] - starts[g])
        if n and 0 <= ctx and ctx + n <= MB * BS:
            for h in range(Hk):
                for rt in range(-(-n * QG // 256)):
                    want[g, h, rt] = seen_steps(ctx, n, window, first)
    taken = {k: [] for k in want}
    sight = np.zeros(6, np.int32)
    for u in units:
        key = u["g"], u["h"], u["rt"]
        assert key in want, u
        n = int(starts[u["g"] + 1] - starts[u["g"]])
        assert u["seq0"] == starts[u["g"]] and u["rows"] == n * QG and u["len"] == lens[u["g"]] + n
        assert 0 <= u["rot"] < u["steps"] and 0 <= u["slot"] < u["pieces"] <= P + 1
        lib.tree_sight(window, first, u["len"], n, sight.ctypes.data_as(ctypes.c_void_p))
        at, skip = int(sight[4]), int(sight[5])
        taken[key].append((u["slot"], u["pieces"], [i if i < at else i + skip for i in range(u["step0"], u["step0"] + u["steps"])]))
    for key, steps in want.items():
        got = sorted(taken[key])
        assert [x[0] for x in got] == list(range(got[0][1])) and len({x[1] for x in got}) == 1
        assert [s for x in got for s in x[2]] == steps, (key, lens[key[0]])
    assert per >= 1 and (not want or total <= per * ctas)


@pytest.mark.parametrize("NG,ctas", [(1, 152), (2, 152), (33, 152), (70, 152), (7, 3), (4, 1)])
@pytest.mark.parametrize("seed", range(5))
def test_random_batches(lib, NG, ctas, seed):
    rng = np.random.default_rng(100 * NG + seed)
    BS, QG, Hk = int(rng.choice([16, 32])), int(rng.choice([6, 8, 16])), int(rng.choice([1, 2, 5, 8]))
    longest = int(np.exp(rng.uniform(np.log(20), np.log(40000))))
    lens = np.maximum(0, np.exp(rng.uniform(0, np.log(longest + 1), NG)).astype(int) - 1)
    counts = rng.integers(0, int(rng.choice([2, 9, 70])), NG)
    starts = int(rng.integers(0, 3)) + np.concatenate([[0], np.cumsum(counts)])
    MB = max(1, -(-int((lens + counts).max()) // BS))
    window = int(rng.choice([0, 1, 64, 129, 1000, 5000, 2147483647]))
    first = int(rng.choice([0, 4, 128, 300, 2147483647])) if window else 0
    check(lib, starts, lens, QG, Hk, MB, BS, int(rng.integers(1, 40)), window, first, ctas)


def test_lengths_in_error_have_no_pieces(lib):
    check(lib, [0, 3, 5, 6, 8], [100, -1, 700, 639], 8, 2, 40, 16, 4, 0, 0, 152, pda.ERRW_BAD_CONTEXT_LEN | pda.ERRW_BAD_POSITION)


def test_starts_that_do_not_ascend_have_no_pieces(lib):
    for starts, tokens in (([0, 5, 3, 8], 8), ([-1, 2, 3, 8], 8), ([0, 2, 3, 9], 8)):
        units, (err, _, total, _, refused) = pieces(lib, starts, [100, 100, 100], 8, 2, 40, 16, 4, 0, 0, 152, tokens)
        assert not units and total == 0 and refused and err == pda.ERRW_BAD_TOKENS


def test_what_all_rows_miss(lib):
    """Sight: hole0 .. hole1-1 are the cached tokens that the first position misses, and skipped steps lie within them."""
    sight = np.zeros(6, np.int32)
    for ctx in (0, 1, 127, 128, 129, 500, 1000):
        for window in (0, 1, 2, 127, 128, 129, 500, 2000, 2147483647):
            for first in (0, 1, 4, 127, 128, 129, 400, 2147483647):
                for n in (1, 5, 200):
                    lib.tree_sight(window, first, ctx + n, n, sight.ctypes.data_as(ctypes.c_void_p))
                    c, d, h0, h1, at, skip = map(int, sight)
                    t = np.arange(ctx)
                    missed = (ctx - t >= window) & (t >= first) if window else np.zeros(ctx, bool)
                    assert (c, d) == (ctx, n)
                    assert np.flatnonzero(missed).tolist() == list(range(h0, h1))
                    if skip:
                        assert h0 <= at * 128 and (at + skip) * 128 <= h1 and at * 128 < h0 + 128 and (at + skip + 1) * 128 > h1


def test_window_tiles(lib):
    out = np.zeros((4000, 2), np.int32)
    for ctx in list(range(0, 70)) + [300, 1000, 4097, 50000]:
        for window in (1, 2, 15, 16, 17, 40, 1000, 2147483647):
            for first in (0, 1, 4, 16, 17, 33, 999, 2147483647):
                n = lib.window_tiles(ctx, window, first, out.ctypes.data_as(ctypes.c_void_p), 4000)
                assert n <= 4000
                got = []
                for a, k in out[:n].tolist():
                    assert 1 <= k <= 16 and a // 16 == (a + k - 1) // 16      # within one aligned tile, so within one block
                    got += range(a, a + k)
                assert got == [t for t in range(ctx) if t < first or ctx - 1 - t < window]
                assert n <= -(-min(first, ctx) // 16) + -(-(min(window, ctx) + 15) // 16)


def test_row_tiles_stay_whole_where_that_costs_little(lib):
    """128 row tiles of 33 steps on 152 CTAs: cut evenly they would end two steps earlier, and every one would be in pieces."""
    starts, lens = np.arange(17) * 32, [4096] * 16
    check(lib, starts, lens, 8, 8, 260, 16, 40, 0, 0, 152)
    units, (_, per, total, whole, _) = pieces(lib, starts, lens, 8, 8, 260, 16, 40, 0, 0, 152)
    assert len(units) == 128 and whole == per == 33 and all(u["pieces"] == 1 and u["steps"] == 33 for u in units)
    units, (_, per, _, whole, _) = pieces(lib, starts, [12288] * 16, 8, 8, 1000, 16, 40, 0, 0, 152)   # here 15 steps earlier
    assert not whole and per < 97 and max(u["pieces"] for u in units) > 1
