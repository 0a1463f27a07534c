"""One workspace for steps of any number of drafted tokens up to the number that it was made for."""
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests.tree_cases import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


@pytest.mark.parametrize("kv", [wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4])
def test_steps_of_all_sizes(pda, kv):
    """Few tokens over a long context are cut into the most pieces, and need more than many; what lies behind is left alone."""
    ws = None
    for counts in ([90, 64, 140], [33, 3, 1], [1, 0, 0], [4, 8, 40], [0, 2, 0]):
        t = TreeCase(kv, 2, 8, 16, [5000, 20, 300], counts, "tree", seed=sum(counts), MB=360)
        p = t.plan(pda)
        if ws is None:
            n = pda.tree_workspace(p, t.N, "cuda").nbytes
            assert n > pda.lib().pda_tree_workspace_size(p, t.N // 20) > 0
            whole = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
            ws = whole[:n]
        t.check(pda, ws=ws)
        assert bool((whole[n:] == 0xA5).all())
