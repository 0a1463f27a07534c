"""What the token operators refuse, before anything is launched (no GPU needed)."""
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


def at(k, off=0):
    """Distinct, 16-byte aligned addresses a megabyte apart (never read: every call here is refused, or has nothing to do)."""
    return ctypes.c_void_p(BASE * (k + 1) + off)


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


def all_plans(pda, fn, p, good, null_ok=False):
    refused(fn, edited(pda, p), good, [({}, INVALID)])
    refused(fn, None, good, [({}, INVALID)])


def test_write_kv(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    #       k      v      ks   vs   N  cache  NB   book  table  starts pos    err   stream
    good = [at(0), at(1), 256, 256, 9, at(2), 100, None, at(3), at(4), at(5), None, None]
    refused(L.pda_write_kv, p, good, [({i: None}, INVALID) for i in (0, 1, 5, 8, 9, 10)] + [
        ({2: 248}, INVALID), ({3: 248}, INVALID), ({2: 260}, INVALID), ({3: 257}, INVALID), ({2: -256}, INVALID), ({4: -1}, INVALID),
        ({4: 1 << 31}, INVALID), ({6: 0}, INVALID), ({6: 1 << 31}, INVALID), ({7: at(9)}, INVALID),
        ({0: at(0, 8)}, INVALID), ({1: at(1, 2)}, INVALID), ({5: at(2, 8)}, INVALID), ({8: at(3, 2)}, INVALID),
        ({9: at(4, 1)}, INVALID), ({10: at(5, 2)}, INVALID), ({11: at(6, 2)}, INVALID), ({4: 0}, OK), ({4: 0, 0: None}, OK)])
    all_plans(pda, L.pda_write_kv, p, good)
    tq = pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4)
    refused(L.pda_write_kv, tq, good, [({}, INVALID), ({7: at(9, 2)}, INVALID), ({7: at(9), 4: 0}, OK)])
    refused(L.pda_write_kv, pda.plan(0, 2, 8, 16, 4), good, [({}, OK)])


def test_read_kv(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_FP8_E4M3)
    #       cache  NB   book  table  starts pos    N  k      v      dtype err   stream
    good = [at(0), 100, None, at(1), at(2), at(3), 9, at(4), at(5), 0, None, None]
    refused(L.pda_read_kv, p, good, [({i: None}, INVALID) for i in (0, 3, 4, 5)] + [
        ({7: None, 8: None}, INVALID), ({9: 2}, INVALID), ({1: 0}, INVALID), ({2: at(9)}, INVALID), ({6: -1}, INVALID),
        ({7: at(4, 8)}, INVALID), ({8: at(5, 4)}, INVALID), ({0: at(0, 4)}, INVALID), ({3: at(1, 2)}, INVALID), ({4: at(2, 2)}, INVALID),
        ({5: at(3, 2)}, INVALID), ({10: at(9, 2)}, INVALID), ({6: 0}, OK)])
    all_plans(pda, L.pda_read_kv, p, good)
    refused(L.pda_read_kv, pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4), good, [({}, INVALID)])
    refused(L.pda_read_kv, pda.plan(0, 2, 8, 16, 4), good, [({}, OK)])


def test_decode_tree(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    need = L.pda_tree_workspace_size(ctypes.byref(p), 9)
    assert need > 0
    #       q      N  cache  NB   book  table  lens   starts masks words win first ws     bytes out    dtype err   stream
    good = [at(0), 9, at(1), 100, None, at(2), at(3), at(4), at(5), 1, 0, 0, at(6), need, at(8), 0, None, None]
    cases = [({i: None}, INVALID) for i in (0, 2, 5, 6, 7, 12, 14)]
    cases += [({8: None}, INVALID), ({9: 0}, INVALID), ({9: -1}, INVALID), ({10: -1}, INVALID), ({11: -1}, INVALID), ({15: 2}, INVALID),
              ({3: 0}, INVALID), ({3: 1 << 31}, INVALID), ({4: at(9)}, INVALID), ({1: -1}, INVALID), ({1: 1 << 28}, INVALID),
              ({13: need - 1}, SMALL), ({13: 0}, SMALL)]
    cases += [({0: at(0, 8)}, INVALID), ({2: at(1, 8)}, INVALID), ({5: at(2, 2)}, INVALID), ({6: at(3, 2)}, INVALID), ({7: at(4, 2)}, INVALID),
              ({8: at(5, 4)}, INVALID), ({12: at(6, 16)}, INVALID), ({14: at(8, 4)}, INVALID), ({14: at(8, 8), 15: 1}, INVALID),
              ({14: at(8, 8)}, INVALID), ({16: at(9, 2)}, INVALID), ({1: 0}, OK)]
    refused(L.pda_decode_tree, p, good, cases)
    all_plans(pda, L.pda_decode_tree, p, good)
    refused(L.pda_decode_tree, pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4), good, [({}, INVALID), ({4: at(9, 2)}, INVALID)])
    refused(L.pda_decode_tree, pda.plan(0, 2, 8, 16, 4), good, [({}, OK)])
    assert L.pda_tree_workspace_size(None, 9) == -1 and L.pda_tree_workspace_size(ctypes.byref(p), -1) == -1
    assert L.pda_tree_workspace_size(ctypes.byref(p), 0) == 0 and L.pda_tree_workspace_size(ctypes.byref(edited(pda, p)), 9) == -1
    # steps that would not fit an int
    big = pda.plan(60000, 8, 16, 32, 1 << 20)
    assert L.pda_tree_workspace_size(ctypes.byref(big), 60000) == -1
    refused(L.pda_decode_tree, big, good, [({1: 60000}, INVALID)])


def test_accept_tokens(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    #       cache  NB   table  lens   path   plens  A  out    err   stream
    good = [at(0), 100, at(1), at(2), at(3), at(4), 5, at(5), None, None]
    refused(L.pda_accept_tokens, p, good, [({i: None}, INVALID) for i in (0, 2, 3, 4, 5, 7)] + [
        ({1: 0}, INVALID), ({6: -1}, INVALID), ({0: at(0, 8)}, INVALID), ({8: at(9, 2)}, INVALID)] + [
        ({i: at(9, 2)}, INVALID) for i in (2, 3, 4, 5, 7)] + [
        ({7: at(2)}, INVALID), ({7: at(2, 8)}, INVALID), ({7: at(4)}, INVALID)])      # in place
    all_plans(pda, L.pda_accept_tokens, p, good)
    refused(L.pda_accept_tokens, pda.plan(0, 2, 8, 16, 4), good, [({}, OK)])


def test_decode_window(pda):
    L, p = pda.lib(), pda.plan(3, 2, 8, 16, 4)
    #       q      cache  NB   book  table  lens   win first out   dtype err   stream
    good = [at(0), at(1), 100, None, at(2), at(3), 16, 4, at(4), 0, None, None]
    refused(L.pda_decode_window, p, good, [({i: None}, INVALID) for i in (0, 1, 4, 5, 8)] + [
        ({6: 0}, INVALID), ({6: -3}, INVALID), ({7: -1}, INVALID), ({9: 2}, INVALID), ({2: 0}, INVALID), ({3: at(9)}, INVALID),
        ({0: at(0, 8)}, INVALID), ({1: at(1, 8)}, INVALID), ({4: at(2, 2)}, INVALID), ({5: at(3, 2)}, INVALID), ({8: at(4, 4)}, INVALID),
        ({8: at(4, 8), 9: 1}, INVALID), ({10: at(9, 2)}, INVALID)])
    all_plans(pda, L.pda_decode_window, p, good)
    refused(L.pda_decode_window, pda.plan(3, 2, 8, 16, 4, kernel_variant=1), good, [({}, UNSUPPORTED)])
    refused(L.pda_decode_window, pda.plan(3, 2, 8, 16, 4, kv_dtype=pda.KV_TQ4), good, [({}, INVALID), ({3: at(9, 2)}, INVALID)])
    refused(L.pda_decode_window, pda.plan(0, 2, 8, 16, 4), good, [({}, OK)])


def test_the_binding_refuses(pda):
    """Tensors that are not on a GPU, before the library is called."""
    p = pda.plan(2, 2, 8, 16, 4)
    z = torch.zeros(4, dtype=torch.int32)
    rows, cache = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(100 * p.cache_block_bytes, dtype=torch.uint8)
    for call in (lambda: pda.write_kv(p, rows, rows, cache, 100, z, z, z), lambda: pda.read_kv(p, cache, 100, z, z, z, rows, rows),
                 lambda: pda.decode_tree(p, rows, cache, 100, z, z, z), lambda: pda.accept_tokens(p, cache, 100, z, z, z, z, z),
                 lambda: pda.decode_window(p, rows, cache, 100, z, z, 16)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    with pytest.raises(pda.PdaError):
        pda.tree_workspace(p, -1, "cpu")
