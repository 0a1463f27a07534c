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


def need(B, Hk, QG, MB, BS, n, sms=152):
    """Bytes that a call of n tokens takes: partials of every row in as many slots as its sequences may be cut into, one more than
    runs, pieces, marks."""
    up = lambda x: -(-x // 256) * 256
    tiles = max(-(-n * QG // 256), min(B, n)) * Hk
    steps = -(-MB * BS // 128)
    slots = min(-(-4 * sms // tiles), (steps + 1) // 2) + 1
    rows = n * Hk * QG
    return up(rows * slots * 512) + 2 * up(rows * slots * 4) + up(rows * 4) + up(n) + 256


@pytest.mark.parametrize("B,Hk,QG,BS,MB", [(1, 1, 8, 16, 16), (1, 8, 8, 16, 2048), (3, 2, 6, 32, 1000), (64, 8, 8, 16, 1024),
                                           (200, 1, 16, 32, 4096), (7, 5, 16, 16, 77), (1, 1, 6, 32, 1 << 20)])
def test_a_workspace_serves_fewer_tokens(pda, B, Hk, QG, BS, MB):
    """One made for n tokens is as large as that of any call of at most n, and no larger than the largest of those."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    p = pda.plan(B, Hk, QG, BS, MB)
    most = 0
    for n in range(1, 1500):
        most = max(most, need(B, Hk, QG, MB, BS, n, sms))
        assert size(pda, p, n) == most, n
