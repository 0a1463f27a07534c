"""The split of the shared prefixes' steps over the CTAs, run on the host (no GPU needed): the kernel's own code, with a warp of
32 contexts in the place of the GPU's."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import paged_kv_gqa_block_gb300 as pda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("cta", "g", "h", "rt", "seq0", "rows", "len", "step0", "steps", "rot", "slot", "pieces")
BAD_LEN, BAD_GROUP = pda.ERRW_BAD_CONTEXT_LEN, pda.ERRW_BAD_GROUP


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "paged_kv_gqa_block_gb300", "serving"), os.path.join(ROOT, "tests", "host", "split.cpp"),
                           "-o", so])
    lib = ctypes.CDLL(so)

    def run(starts, plens, B, QG, Hk, MP, BS, P, ctas):
        NG, cap = len(plens), 200000
        out, scalars = np.zeros((cap, 12), np.int32), np.zeros(4, np.int32)
        starts, plens = np.asarray(starts, np.int32), np.asarray(plens, np.int32)
        ptr = lambda x: x.ctypes.data_as(ctypes.c_void_p)
        n = lib.split_pieces(NG, ptr(starts), ptr(plens), B, QG, Hk, MP, BS, P, ctas, ptr(out), cap, ptr(scalars))
        assert n >= 0
        return [dict(zip(FIELDS, map(int, r))) for r in out[:n]], [int(x) for x in scalars]

    return run


def check(split, starts, plens, B, QG, Hk, MP, BS, P, ctas, err=0):
    """Every step of every row tile is taken once, by pieces numbered as the join expects them."""
    units, (e, per, total, whole) = split(starts, plens, B, QG, Hk, MP, BS, P, ctas)
    assert e == err
    want = {}
    for g, n in enumerate(plens):
        n = n if 0 <= n <= MP * BS else 0
        rows = (starts[g + 1] - starts[g]) * QG
        for h in range(Hk):
            for rt in range(-(-rows // 256) if n else 0):
                want[g, h, rt] = -(-n // 128)
    taken = {k: [] for k in want}
    for u in units:
        key = u["g"], u["h"], u["rt"]
        assert key in want, u
        assert u["seq0"] == starts[u["g"]] and u["rows"] == (starts[u["g"] + 1] - starts[u["g"]]) * QG and u["len"] == plens[u["g"]]
        assert 0 <= u["step0"] and u["steps"] > 0 and u["step0"] + u["steps"] <= want[key]
        assert 0 <= u["rot"] < u["steps"]
        assert 0 <= u["slot"] < u["pieces"] <= P + 1         # the workspace's slots
        taken[key].append(u)
    for key, ns in want.items():
        pieces = sorted(taken[key], key=lambda u: u["slot"])
        assert pieces, key
        assert [u["slot"] for u in pieces] == list(range(pieces[0]["pieces"])), key
        assert len({u["pieces"] for u in pieces}) == 1
        at = 0
        for u in pieces:                                     # slots in the order of the tokens, without a gap or an overlap
            assert u["step0"] == at, (key, u)
            at += u["steps"]
        assert at == ns
    assert per >= 1 and (not want or total <= per * ctas)
    return units


SIZES = [(1, 152), (2, 152), (5, 152), (33, 152), (70, 152), (7, 3), (4, 1), (40, 148)]


@pytest.mark.parametrize("NG,ctas", SIZES)
@pytest.mark.parametrize("seed", range(6))
def test_random_groups(split, NG, ctas, seed):
    rng = np.random.default_rng(1000 * NG + seed)
    BS, QG, Hk = int(rng.choice([16, 32])), int(rng.choice([6, 8, 16])), int(rng.choice([1, 2, 5, 8]))
    longest = int(np.exp(rng.uniform(np.log(20), np.log(40000))))
    plens = np.maximum(0, np.exp(rng.uniform(0, np.log(longest + 1), NG)).astype(int) - 1)
    if seed == 0:
        plens[:] = longest
    sizes = rng.integers(0, 1 + max(1, 200 // NG), NG)
    before = int(rng.integers(0, 3))
    starts = before + np.concatenate([[0], np.cumsum(sizes)])
    MP = -(-max(1, longest) // BS)
    for G in (1, 2, 1 + MP * BS // 256 // 7, 5000):          # pieces as long as P allows, and as the SMs suggest
        check(split, starts.tolist(), plens.tolist(), int(starts[-1]) + 2, QG, Hk, MP, BS, -(-MP * BS // (G * 256)), ctas)


def test_one_row_tile_and_many(split):
    for n in (1, 127, 128, 129, 255, 256, 257, 128 * 152, 128 * 152 + 1, 128 * 303):
        for B in (1, 16, 17, 32, 33, 100):
            check(split, [0, B], [n], B, 16, 1, -(-n // 16), 16, max(1, -(-n // 512)), 152)


def test_groups_without_rows_or_tokens(split):
    assert check(split, [0, 0, 0], [100, 100], 4, 8, 2, 10, 16, 1, 152) == []
    assert check(split, [0, 2, 4], [0, 0], 4, 8, 2, 10, 16, 1, 152) == []
    check(split, [1, 1, 3, 3, 4], [100, 0, 5, 160], 4, 8, 2, 10, 16, 1, 152)


def test_lengths_out_of_range_count_as_empty(split):
    check(split, [0, 1, 2, 3], [100, 161, -1], 3, 8, 2, 10, 16, 1, 152, err=BAD_LEN)


@pytest.mark.parametrize("starts", [(0, 2, 1, 6), (-1, 2, 4, 6), (0, 2, 4, 7), (0, 9, 4, 6), (6, 5, 4, 3), (0, 2 ** 31 - 1, 0, 2 ** 31 - 1)])
def test_groups_that_do_not_ascend_give_no_pieces(split, starts):
    units, scalars = split(list(starts), [100, 100, 100], 6, 8, 2, 10, 16, 1, 152)
    assert units == [] and scalars[0] == BAD_GROUP


def test_thousands_of_overlapping_groups_end(split):
    NG = 4001
    starts = np.zeros(NG + 1, np.int32)
    starts[1::2] = 64
    units, scalars = split(starts, np.full(NG, 60000 * 16), 64, 16, 8, 60000, 16, 3750, 8)
    assert units == [] and scalars[0] == BAD_GROUP


def test_the_largest_step_numbers(split):
    """As many steps as the host lets through: places stay within an int."""
    B, QG, Hk, BS, MP = 16, 16, 1, 32, 1 << 25               # 2^30 tokens
    tiles = 1
    assert tiles * Hk * (MP * BS // 128) * 4 <= 2000000000
    for P in (1, 2, 152, 4096):
        check(split, [0, B], [MP * BS], B, QG, Hk, MP, BS, P, 152)
    # 58 row tiles of the longest: 486 million of the 500 million steps that are allowed
    B = 58 * 16
    units = check(split, [0, B], [MP * BS], B, QG, Hk, MP, BS, 1, 152)
    assert len(units) >= 58
    # one long group beside many short ones
    starts = [0, 16] + [16 + i for i in range(1, 40)]
    check(split, starts, [MP * BS] + [1] * 39, 56, QG, Hk, MP, BS, 1, 152)
