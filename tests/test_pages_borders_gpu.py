"""Page operators at the borders of their code paths."""
import numpy as np
import pytest

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp
from tests.test_pages_gpu import batch, check_compact, check_fork, dev, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


# One scan CTA up to 4096 blocks, eight above; a CTA's slice is one tile, and stays in registers, up to 4096 blocks, 32768 in all;
# slices that end inside a thread's four entries; CTAs without any.
@pytest.mark.parametrize("NB", [1, 4, 4095, 4096, 4097, 4099, 32761, 32767, 32768, 32769, 32777, 65541])
@pytest.mark.parametrize("full", [0.0, 0.5, 0.97])
def test_pool_sizes_at_the_borders_of_the_scan(pda, NB, full):
    rng = np.random.default_rng(NB + int(10 * full))
    p = pda.plan(3, 1, 8, 16, 64, kv_dtype=wl.KV_TQ4)
    most = min(64, NB // 4)
    lens = np.array([most * 16, max(0, most * 16 - 9), 0], np.int32)
    table, refs = batch(rng, lens, 16, 64, NB)
    others = rng.permutation(np.flatnonzero(refs == 0))
    others = others[:int(len(others) * full)]
    refs[others] = rng.integers(1, 4, len(others))
    cache = pool(rng, NB, p.cache_block_bytes)
    check_fork(pda, p, cache, NB, table, lens, refs, [0, 0, 1, 2], [3, 0, 30, 5])
    check_compact(pda, p, cache, NB, table, lens, refs)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 1500, 3001])
def test_fork_of_a_large_old_batch(pda, B):
    # up to 1024 old sequences their first rows are kept in shared memory, above in the workspace
    rng = np.random.default_rng(B)
    MB, NB, R = 2, 7000, 2500
    lens = rng.integers(0, 33, B).astype(np.int32)
    p = pda.plan(B, 1, 6, 16, MB, kv_dtype=wl.KV_TQ4)
    table, refs = batch(rng, lens, 16, MB, NB)
    cache = pool(rng, NB, p.cache_block_bytes)
    refs[rng.permutation(np.flatnonzero(refs == 0))[:(NB - B) // 3]] = 1      # blocks that others hold
    parents = rng.integers(-1, B, R)
    parents[:700] = rng.integers(max(0, B - 40), B, 700)     # the highest old sequences, often
    got = check_fork(pda, p, cache, NB, table, lens, refs, parents, rng.integers(0, 4, R))
    assert got[4] & ~(pp.NO_BLOCKS | pp.BAD_POS) == 0        # (a row of 32 tokens, the table's room, cannot grow)
    few = np.where(refs == 0, rng.random(NB) < 0.93, refs).astype(np.int32)   # rows refused for lack of blocks, first ones among them
    got = check_fork(pda, p, cache, NB, table, lens, few, parents, rng.integers(0, 9, R))
    assert got[4] & pp.NO_BLOCKS and (got[2] > 0).any()


def test_fork_from_an_empty_batch_and_to_an_empty_one(pda):
    rng = np.random.default_rng(8)
    p = pda.plan(0, 1, 8, 16, 4)
    refs = np.array([0, 2, 0, 1, 0], np.int32)
    cache = pool(rng, 5, p.cache_block_bytes)
    none = np.zeros((0, 4), np.int32)
    got = check_fork(pda, p, cache, 5, none, np.zeros(0, np.int32), refs, [-1, 0, -1], [1, 1, 1])
    assert got[4] == pp.BAD_SEQ and not got[2].any()
    p = pda.plan(2, 1, 8, 16, 4)
    lens = np.array([20, 3], np.int32)
    table, refs = batch(rng, lens, 16, 4, 5)
    got = check_fork(pda, p, cache, 5, table, lens, refs, [], None)
    assert not got[3].any()
