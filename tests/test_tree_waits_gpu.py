"""Wait limits of the steps for drafted tokens and over windows: below the copies' latency every format and every size of unit gives
up, says so, and leaves the context usable; a step that says nothing is right."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests.gpu_helpers import to_device
from tests.test_wait_limits_gpu import sweep
from tests.tree_cases import TreeCase

pytestmark = pytest.mark.gpu

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4

# rows held twice, one tile, two tiles, two and a further row tile, and units of all these by turns
COUNTS = {"twice": [4] * 20, "tile": [12] * 20, "tiles": [30] * 20, "row tiles": [40] * 20, "mixed": [1, 40, 9, 16, 17, 33, 4, 64, 8, 2] * 2}


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


@pytest.mark.parametrize("kv", [BF16, FP8, TQ4])
@pytest.mark.parametrize("units", list(COUNTS))
def test_limits_around_the_latency(pda, kv, units):
    t = TreeCase(kv, 8, 8, 16, [1500] * 20, COUNTS[units], "tree", seed=21)
    d = t.device()
    want, bound = t.reference(fill=7.0)
    assert t.run(pda, d)[1] == 0
    seen = []
    for limit in [1] * 6 + [1500, 3000, 6000, 12000, 30000, 100000, 1000000]:
        out, err = t.run(pda, d, p=t.plan(pda, wait_timeout_ns=limit))
        assert err in (0, pda.ERRW_PIPELINE_TIMEOUT), (limit, err)
        if err == 0:
            assert (np.abs(out.cpu().double().numpy() - want) <= bound).all(), limit
        seen.append(err)
    assert pda.ERRW_PIPELINE_TIMEOUT in seen[:6]
    out, err = t.run(pda, d)
    assert err == 0 and (np.abs(out.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("kv", [BF16, FP8, TQ4])
@pytest.mark.parametrize("B", [2, 64])                       # clusters of several CTAs, and single ones
def test_windows_around_the_latency(pda, kv, B):
    w = wl.small(num_seqs=B, num_kv_heads=8, query_group_size=8, ctx=(2048,) * B, kv_dtype=kv, seed=4, extra_blocks=0)
    d = to_device(wl.generate(w))

    def run(limit, err):
        p = pda.plan(B, 8, 8, 16, w.max_blocks_per_seq, kv_dtype=kv, wait_timeout_ns=limit)
        return pda.decode_window(p, d["query"], d["cache"], w.num_cache_blocks, d["block_table"], d["context_lens"], 1003, num_first=20,
                                 out_dtype=torch.float32, centroids=d.get("centroids"), err_word=err)

    sweep(pda, run)
