"""What the page and block-selection entry points refuse, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from paged_kv_gqa_block_gb300 import _build

OK, INVALID, UNSUPPORTED, SMALL = 0, -1, -2, -3
BASE = 1 << 20


@pytest.fixture(scope="module")
def pda():
    _build.build()
    import paged_kv_gqa_block_gb300 as pda
    pda.lib()
    return pda


def at(k):
    """Distinct, 16-byte aligned addresses a megabyte apart (never read: every call here is refused)."""
    return ctypes.c_void_p(BASE * (k + 1))


def refused(fn, plan, good, cases):
    for changes, status in cases:
        args = list(good)
        for i, v in changes.items():
            args[i] = v
        assert fn(None if plan is None else ctypes.byref(plan), *args) == status, changes


def edited(pda, p):
    q = pda.Plan.from_buffer_copy(p)
    q.cache_block_bytes += 16
    return q


def test_copy_blocks(pda):
    L, p = pda.lib(), pda.plan(1, 2, 8, 16, 4)
    good = [at(0), 4, at(1), 4, at(2), 3, None, None]
    off = ctypes.c_void_p
    refused(L.pda_copy_blocks, p, good, [
        ({0: None}, INVALID), ({2: None}, INVALID), ({4: None}, INVALID), ({1: 0}, INVALID), ({3: 1 << 31}, INVALID),
        ({5: -1}, INVALID), ({0: off(BASE + 8)}, INVALID), ({2: off(BASE + 4)}, INVALID), ({4: off(BASE + 2)}, INVALID),
        ({6: off(3)}, INVALID), ({2: off(BASE + p.cache_block_bytes)}, INVALID),      # pools that overlap
        ({5: 0}, OK)])
    refused(L.pda_copy_blocks, edited(pda, p), good, [({}, INVALID)])
    refused(L.pda_copy_blocks, None, good, [({}, INVALID)])


def test_fork_sequences(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    need = L.pda_page_workspace_size(ctypes.byref(p), 5, 100)
    good = [at(0), 100, at(1), at(2), at(3), 5, at(4), at(5), at(6), at(7), at(8), at(9), need, None, None]
    off = ctypes.c_void_p
    cases = [({i: None}, INVALID) for i in (0, 2, 3, 4, 6, 8, 9, 10, 11)]
    cases += [({1: 0}, INVALID), ({1: 1 << 31}, INVALID), ({5: -1}, INVALID), ({12: need - 1}, SMALL), ({5: 6}, SMALL)]
    cases += [({i: off(BASE * 20 + 2)}, INVALID) for i in (2, 3, 4, 6, 7, 8, 9, 10, 13)]
    cases += [({0: off(BASE * 20 + 8)}, INVALID), ({11: off(BASE * 20 + 4)}, INVALID)]
    cases += [({8: at(1)}, INVALID), ({9: off(BASE * 3 + 8)}, INVALID), ({10: off(BASE * 4 + 396)}, INVALID)]   # in place
    refused(L.pda_fork_sequences, p, good, cases)
    refused(L.pda_fork_sequences, edited(pda, p), good, [({}, INVALID)])
    assert L.pda_page_workspace_size(None, 1, 100) == -1 and L.pda_page_workspace_size(ctypes.byref(p), -1, 100) == -1
    assert L.pda_page_workspace_size(ctypes.byref(p), 1, 0) == -1


def test_compact_blocks(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    need = L.pda_page_workspace_size(ctypes.byref(p), 0, 100)
    good = [at(0), 100, at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), need, None, None]
    off = ctypes.c_void_p
    cases = [({i: None}, INVALID) for i in (0, 2, 3, 4, 5, 6, 7, 8, 9)]
    cases += [({1: 0}, INVALID), ({10: need - 1}, SMALL), ({5: at(1)}, INVALID), ({6: at(3)}, INVALID), ({7: at(3)}, INVALID),
              ({7: at(5)}, INVALID)]
    cases += [({i: off(BASE * 20 + 2)}, INVALID) for i in (2, 3, 4, 5, 6, 7, 8, 11)]
    refused(L.pda_compact_blocks, p, good, cases)


def test_summaries_and_scores(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    off = ctypes.c_void_p
    good = [at(0), 100, at(1), at(2), None, None, at(3), None, None]
    refused(L.pda_summarize_blocks, p, good, [({i: None}, INVALID) for i in (0, 2, 3, 6)] + [
        ({1: 0}, INVALID), ({5: at(9)}, INVALID), ({0: off(BASE + 8)}, INVALID), ({6: off(BASE + 8)}, INVALID),
        ({4: off(BASE + 2)}, INVALID), ({7: off(BASE + 1)}, INVALID)])
    tq = pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4)
    refused(L.pda_summarize_blocks, tq, good, [({}, INVALID)])                         # its centroids are missing
    good = [at(0), at(1), 100, at(2), at(3), at(4), None, None]
    refused(L.pda_score_blocks, p, good, [({i: None}, INVALID) for i in (0, 1, 3, 4, 5)] + [
        ({2: 0}, INVALID), ({0: off(BASE + 8)}, INVALID), ({1: off(BASE + 8)}, INVALID), ({5: off(BASE + 2)}, INVALID)])
    empty = pda.plan(0, 2, 8, 16, 4)
    assert L.pda_score_blocks(ctypes.byref(empty), *good) == OK
    assert L.pda_summary_size(ctypes.byref(p), 100) == 100 * 2 * 512 and L.pda_summary_size(ctypes.byref(p), 0) == -1


def test_select_and_decode_selected(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    off = ctypes.c_void_p
    good = [at(0), at(1), at(2), 8, 1, 2, at(3), at(4), None, None, None]
    refused(L.pda_select_blocks, p, good, [({i: None}, INVALID) for i in (0, 1, 2, 6, 7)] + [
        ({3: 0}, INVALID), ({4: -1}, INVALID), ({5: -1}, INVALID), ({3: 2}, INVALID), ({4: 1 << 30, 5: 1 << 30, 3: 1 << 20}, INVALID),
        ({3: 1 << 27}, INVALID), ({8: off(BASE + 2)}, INVALID)])
    good = [at(0), at(1), 100, None, at(2), at(3), at(4), at(5), at(6), at(7), 0, None, None]
    warps = pda.plan(3, 2, 8, 16, 4, kernel_variant=pda.VARIANT_HEAD_WARPS)            # needs its partials
    refused(L.pda_decode_selected, warps, good, [({i: None}, INVALID) for i in (0, 1, 4, 5, 6, 7, 8, 9)])
    refused(L.pda_decode_selected, p, good, [({i: None}, INVALID) for i in (0, 1, 4, 5, 9)] + [
        ({2: 0}, INVALID), ({3: at(9)}, INVALID), ({10: 2}, INVALID), ({0: off(BASE + 8)}, INVALID), ({6: off(BASE + 8)}, INVALID),
        ({9: off(BASE + 4)}, INVALID), ({9: off(BASE + 8), 10: 1}, INVALID)])
    grouped = pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_FP8_E4M3, kernel_variant=pda.VARIANT_HEAD_GROUPS)
    refused(L.pda_decode_selected, grouped, good, [({}, UNSUPPORTED)])
    tq = pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4)
    refused(L.pda_decode_selected, tq, good, [({}, INVALID)])
    assert L.pda_decode_selected(ctypes.byref(pda.plan(0, 2, 8, 16, 4)), *good) == OK


def test_decode_shared(pda):
    L = pda.lib()
    pp, p = pda.shared_plans(6, 2, 2, 8, 16, 40, 4)
    need = L.pda_shared_workspace_size(ctypes.byref(pp), ctypes.byref(p))
    assert need > 0
    good = [ctypes.byref(p)] + [at(k) for k in range(2)] + [100] + [at(k) for k in range(2, 8)] + [need, at(8), 0, None, None]
    off = ctypes.c_void_p
    refused(L.pda_decode_shared, pp, good, [({i: None}, INVALID) for i in (0, 1, 2, 4, 5, 6, 7, 8, 9, 11)] + [
        ({3: 0}, INVALID), ({10: need - 1}, SMALL), ({12: 5}, INVALID), ({1: off(BASE + 8)}, INVALID), ({2: off(BASE + 8)}, INVALID),
        ({9: off(BASE + 16)}, INVALID), ({4: off(BASE + 2)}, INVALID), ({11: off(BASE + 4)}, INVALID), ({13: off(BASE + 2)}, INVALID)])
    for other in (dict(num_kv_heads=1), dict(query_group_size=6), dict(kv_block_size=32), dict(kv_dtype=1), dict(softmax_scale=0.5)):
        args = dict(num_seqs=6, num_kv_heads=2, query_group_size=8, kv_block_size=16, max_blocks_per_seq=4)
        q = pda.plan(**{**args, **other})
        assert L.pda_shared_workspace_size(ctypes.byref(pp), ctypes.byref(q)) == -1
        refused(L.pda_decode_shared, pp, [ctypes.byref(q)] + good[1:], [({}, INVALID)])
    tpp, tp = pda.shared_plans(6, 2, 2, 8, 16, 40, 4, kv_dtype=pda.KV_TQ4)
    refused(L.pda_decode_shared, tpp, [ctypes.byref(tp)] + good[1:10] + [1 << 30] + good[11:], [({}, UNSUPPORTED)])
    none = pda.plan(0, 2, 8, 16, 40, 2)                                                # no groups
    refused(L.pda_decode_shared, none, good[:10] + [1 << 30] + good[11:], [({}, INVALID)])
    empty = pda.plan(0, 2, 8, 16, 4)
    refused(L.pda_decode_shared, pp, [ctypes.byref(empty)] + good[1:], [({}, OK)])
    huge = pda.shared_plans(1 << 20, 1 << 16, 8, 16, 32, 1 << 20, 1)                   # more steps than an int counts
    big = L.pda_shared_workspace_size(ctypes.byref(huge[0]), ctypes.byref(huge[1]))
    refused(L.pda_decode_shared, huge[0], [ctypes.byref(huge[1])] + good[1:10] + [big] + good[11:], [({}, INVALID)])


def test_shared_plans(pda):
    for B, NG, Hk, QG, BS, blocks in ((2, 1, 1, 8, 16, 16), (64, 1, 8, 6, 16, 251), (128, 1, 8, 8, 32, 1024), (32, 4, 4, 16, 32, 256),
                                      (1, 1, 1, 6, 16, 100000)):
        pp, p = pda.shared_plans(B, NG, Hk, QG, BS, blocks, 4)
        assert pp.num_seqs == NG and p.num_seqs == B and pp.max_blocks_per_seq == blocks
        assert pp.partition_tokens >= 256 and pp.num_partitions * pp.partition_tokens >= blocks * BS
        assert pp.num_partitions <= max(1, 2 * 152)
    assert pda.lib().pda_shared_tile_groups(None, 1, 1) == INVALID
    assert pda.lib().pda_shared_tile_groups(ctypes.byref(p), 0, 1) == INVALID
    assert pda.lib().pda_shared_tile_groups(ctypes.byref(p), 1, 0) == INVALID
    pp, _ = pda.shared_plans(8, 1, 8, 8, 16, 1000, 4, prefix_tile_groups=3)
    assert pp.resolved_tile_groups == 3


def test_the_binding_refuses_host_tensors(pda):
    p = pda.plan(1, 1, 8, 16, 4)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pda.copy_blocks(p, torch.zeros(100), 1, torch.zeros(100), 1, i32(1, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        pda.select_blocks(p, torch.zeros(1, 1, 4), i32(1, 4), i32(1), 2, 0, 1, i32(1, 1, 2), i32(1, 1))
    with pytest.raises(ValueError, match="CUDA tensor"):
        pda.score_blocks(p, torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(4, 1, 2, 128, dtype=torch.bfloat16), 4, i32(1, 4), i32(1),
                         torch.zeros(1, 1, 4))
