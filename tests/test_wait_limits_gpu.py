"""Wait limits around the time that the waits take: whatever a limit cuts off, the call ends, a call whose waits all ended in time
gives the results of one without a limit, another sets the timeout bit, and the next call is right.  The limits pass from
far below a copy's latency to above it, so that many of them end while a warp's copy is landing."""
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests.gpu_helpers import to_device

pytestmark = pytest.mark.gpu

LIMITS = [*range(1, 40, 13), *range(100, 3000, 97), 4000, 6000, 9000, 15000, 40000, 200000]


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def sweep(pda, run):
    """run(limit, err) -> out; limit 0 is the default of a second."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = run(0, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    seen = set()
    for limit in LIMITS:
        err.zero_()
        out = run(limit, err)
        torch.cuda.synchronize()
        e = int(err.item())
        assert e in (0, pda.ERRW_PIPELINE_TIMEOUT), limit
        seen.add(e)
        if e == 0:
            assert torch.equal(out, want), limit
    err.zero_()
    assert torch.equal(run(0, err), want) and int(err.item()) == 0
    return seen


@pytest.mark.parametrize("kv,QG,variant", [(wl.KV_BF16, 8, 1), (wl.KV_BF16, 16, 1), (wl.KV_BF16, 16, 3), (wl.KV_FP8_E4M3, 8, 1),
                                           (wl.KV_FP8_E4M3, 6, 2), (wl.KV_FP8_E4M3, 16, 2), (wl.KV_TQ4, 8, 1)])
def test_plain_steps(pda, kv, QG, variant):
    w = wl.small(num_seqs=8, num_kv_heads=4, query_group_size=QG, ctx=(4096,) * 8, kv_dtype=kv, seed=3, extra_blocks=0)
    d = to_device(wl.generate(w))
    def run(limit, err):
        p = pda.plan(8, 4, QG, 16, w.max_blocks_per_seq, kv_dtype=kv, wait_timeout_ns=limit, kernel_variant=variant)
        return pda.decode_step(p, d["query"], d["cache"], w.num_cache_blocks, d["block_table"], d["context_lens"],
                               out_dtype=torch.float32, err_word=err, centroids=d.get("centroids"))
    sweep(pda, run)


@pytest.mark.parametrize("kv,QG", [(wl.KV_BF16, 8), (wl.KV_BF16, 16), (wl.KV_FP8_E4M3, 8), (wl.KV_TQ4, 8)])
@pytest.mark.parametrize("B", [2, 32])                       # clusters of several CTAs, and single ones
def test_selected_blocks(pda, kv, QG, B):
    w = wl.small(num_seqs=B, num_kv_heads=8, query_group_size=QG, ctx=(2048,) * B, kv_dtype=kv, seed=4, extra_blocks=0)
    d = to_device(wl.generate(w))
    table = d["block_table"][:, None].expand(-1, 8, -1).contiguous()
    lens = torch.full((B, 8), 2048, dtype=torch.int32, device="cuda")
    def run(limit, err):
        p = pda.plan(B, 8, QG, 16, w.max_blocks_per_seq, kv_dtype=kv, wait_timeout_ns=limit)
        return pda.decode_selected(p, d["query"], d["cache"], w.num_cache_blocks, table, lens, out_dtype=torch.float32,
                                   centroids=d.get("centroids"), err_word=err)
    sweep(pda, run)


@pytest.mark.parametrize("kv", [wl.KV_BF16, wl.KV_FP8_E4M3])
@pytest.mark.parametrize("B,prefix", [(4, 512), (64, 2048)])           # the prefix before the own tokens, and after
def test_shared_prefixes(pda, kv, B, prefix):
    w = wl.small(num_seqs=B + 1, num_kv_heads=4, ctx=(prefix,) + (64,) * B, kv_dtype=kv, seed=5, extra_blocks=0)
    d = to_device(wl.generate(w))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ptable, table = d["block_table"][:1].contiguous(), d["block_table"][1:, :4].contiguous()
    starts, plens, lens = i32(0, B), i32(prefix), d["context_lens"][1:].contiguous()
    q = d["query"][1:].contiguous()
    def run(limit, err):
        p2 = pda.shared_plans(B, 1, 4, 8, 16, prefix // 16, 4, kv_dtype=kv, wait_timeout_ns=limit)
        return pda.decode_shared(*p2, q, d["cache"], w.num_cache_blocks, starts, ptable, plens, table, lens,
                                 out_dtype=torch.float32, err_word=err)
    sweep(pda, run)
