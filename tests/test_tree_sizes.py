"""Sizes of pda_decode_tree's workspace, and numbers of tokens whose arithmetic would not fit.  No GPU needed."""
import ctypes

import pytest

from paged_kv_gqa_block_gb300 import _build

INVALID = -1
BASE = 1 << 20


@pytest.fixture(scope="module")
def pda():
    _build.build()
    import paged_kv_gqa_block_gb300 as pda
    pda.lib()
    return pda


def size(pda, p, n):
    return pda.lib().pda_tree_workspace_size(ctypes.byref(p), n)


@pytest.mark.parametrize("QG", [6, 8, 16])
def test_numbers_of_tokens_past_every_range(pda, QG):
    """Among them those whose rows are 0, or few, modulo 2^64."""
    p = pda.plan(3, 2, QG, 16, 4)
    assert size(pda, p, (1 << 30) // QG) > 0
    many = [(1 << 30) // QG + 1, 1 << 31, 1 << 59, 1 << 60, (1 << 60) + 9, 1 << 61, 1 << 62, (1 << 64) // QG + 1, (1 << 63) - 1]
    at = lambda k: ctypes.c_void_p(BASE * (k + 1))
    for n in [x for x in many if x < 1 << 63]:
        assert size(pda, p, n) == -1, n
        rc = pda.lib().pda_decode_tree(ctypes.byref(p), at(0), n, at(1), 100, None, at(2), at(3), at(4), None, 0, 0, 0, at(6),
                                       (1 << 63) - 1, at(8), 0, None, None)
        assert rc == INVALID, n


def test_heads_past_every_range(pda):
    """Row tiles times steps modulo 2^64."""
    p = pda.plan(1, (1 << 31) - 1, 16, 32, 1, tile_groups_per_partition=1 << 20)
    assert size(pda, p, 1 << 26) == -1
    q = pda.plan(1, 1 << 20, 16, 32, 1 << 25, tile_groups_per_partition=1 << 20)
    for n in (1 << 26, (1 << 26) - 16, 1 << 25):
        assert size(pda, q, n) == -1
