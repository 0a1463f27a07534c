"""paged_kv_gqa_block_gb300: single-token paged-KV GQA decode attention for GB300 (sm_103a).

Thin binding over the C ABI of ``libpda.so`` (declared in ``include/pda.h``): it checks and
marshals torch tensors into device pointers and calls the library.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and a
missing library raises.  PyTorch provides device memory and streams only.

    p   = plan(num_seqs=..., num_kv_heads=..., query_group_size=8, kv_block_size=16,
               max_blocks_per_seq=..., tile_groups_per_partition=1)
    ws  = workspace(p, device)                    # partial_out, exp_sums, max_logits
    decode(p, query, kv_cache, num_cache_blocks, block_table, context_lens, **ws)
    reduce(p, context_lens, out=out, **ws)        # or decode_step(...) for both

A pool of blocks with counts on the device: fork_sequences lays a batch out anew (forks, reorders, grows,
frees), append_kv writes the new tokens, copy_blocks and compact_blocks move blocks.

    fork_sequences(p, kv_cache, NB, table, lens, refs, parents, new_table, new_lens, new_refs,
                   page_workspace(p, rows, NB, device), new_tokens=ones)

Sequences that share prefixes, and long contexts of which a step attends to selected blocks only:

    pp, p = shared_plans(B, groups, Hk, QG, BS, prefix_blocks, max_blocks_per_seq)
    decode_shared(pp, p, query, kv_cache, NB, group_starts, prefix_table, prefix_lens, table, lens)

    summarize_blocks(p, kv_cache, NB, table, lens, summaries, since=appended_at)
    score_blocks(p, query, summaries, NB, table, lens, scores)
    select_blocks(p, scores, table, lens, K, 1, 1, sel_table, sel_lens)
    decode_selected(plan(..., max_blocks_per_seq=K), query, kv_cache, NB, sel_table, sel_lens)

Many tokens per sequence, written in the cache's format and read back; drafted tokens in chains or trees; sliding windows:

    write_kv(p, k, v, kv_cache, NB, table, token_starts, positions)
    read_kv(p, kv_cache, NB, table, token_starts, positions, k_out, v_out)
    decode_tree(p, query, kv_cache, NB, table, lens, token_starts, tree_masks=masks)
    accept_tokens(p, kv_cache, NB, table, lens, path, path_lens, new_lens)
    decode_window(p, query, kv_cache, NB, table, lens, 4096, num_first=4)
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpda.so")

KV_BF16 = 0
KV_FP8_E4M3 = 1
KV_TQ4 = 2
OUT_BF16 = 0
OUT_F32 = 1
ERRW_BAD_CONTEXT_LEN = 1
ERRW_BAD_BLOCK_ID = 2
ERRW_PIPELINE_TIMEOUT = 4
ERRW_BAD_POSITION = 8
ERRW_BAD_SEQUENCE = 16
ERRW_OUT_OF_BLOCKS = 32
ERRW_BAD_GROUP = 64
ERRW_BAD_TOKENS = 128
HEAD_DIM = 128
VARIANT_AUTO = 0
VARIANT_HEAD_WARPS = 1
VARIANT_HEAD_GROUPS = 2
VARIANT_ROW_HALVES = 3

STATUS = {0: "PDA_OK", -1: "PDA_ERR_INVALID_ARG", -2: "PDA_ERR_UNSUPPORTED", -3: "PDA_ERR_WORKSPACE_TOO_SMALL",
          -4: "PDA_ERR_LAUNCH", -5: "PDA_ERR_NOT_IMPLEMENTED", -6: "PDA_ERR_CUDA"}


class PdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class Plan(ctypes.Structure):
    """Mirror of pda_plan_t."""
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("query_group_size", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("kv_block_size", ctypes.c_int), ("max_blocks_per_seq", ctypes.c_int),
        ("tile_groups_per_partition", ctypes.c_int), ("max_partitions", ctypes.c_int), ("kv_dtype", ctypes.c_int),
        ("softmax_scale", ctypes.c_float), ("wait_timeout_ns", ctypes.c_int), ("kernel_variant", ctypes.c_int),
        ("num_partitions", ctypes.c_int), ("partition_tokens", ctypes.c_int), ("resolved_tile_groups", ctypes.c_int),
        ("resolved_softmax_scale", ctypes.c_float),
        ("cache_block_bytes", ctypes.c_longlong), ("meta_offset_bytes", ctypes.c_longlong),
        ("workspace_bytes", ctypes.c_longlong),
    ]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


_lib = None
_lock = threading.Lock()
_VP = ctypes.c_void_p


def lib():
    """The loaded libpda.so.  Raises if it has not been built (no fallback exists)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(LIB_PATH)
            P = ctypes.POINTER(Plan)
            L.pda_plan.argtypes = [P]
            L.pda_plan.restype = ctypes.c_int
            L.pda_decode.argtypes = [P, _VP, _VP, ctypes.c_longlong, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
            L.pda_decode.restype = ctypes.c_int
            L.pda_decode_tq4.argtypes = [P, _VP, _VP, ctypes.c_longlong, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
            L.pda_decode_tq4.restype = ctypes.c_int
            L.pda_reduce.argtypes = [P, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP]
            L.pda_reduce.restype = ctypes.c_int
            L.pda_status_string.argtypes = [ctypes.c_int]
            L.pda_status_string.restype = ctypes.c_char_p
            L.pda_workspace_size.argtypes = [P]
            L.pda_workspace_size.restype = ctypes.c_longlong
            L.pda_append_kv.argtypes = [P, _VP, _VP, _VP, ctypes.c_longlong, _VP, _VP, _VP, _VP]
            L.pda_append_kv.restype = ctypes.c_int
            L.pda_decode_fused.argtypes = [P, _VP, _VP, ctypes.c_longlong, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                           ctypes.c_int, _VP, _VP]
            L.pda_decode_fused.restype = ctypes.c_int
            L.pda_decode_step_noalloc.argtypes = [P, _VP, _VP, ctypes.c_longlong, _VP, _VP, _VP, ctypes.c_int, _VP,
                                                  _VP]
            L.pda_decode_step_noalloc.restype = ctypes.c_int
            CLL, CI = ctypes.c_longlong, ctypes.c_int
            L.pda_copy_blocks.argtypes = [P, _VP, CLL, _VP, CLL, _VP, CLL, _VP, _VP]
            L.pda_page_workspace_size.argtypes = [P, CI, CLL]
            L.pda_page_workspace_size.restype = CLL
            L.pda_fork_sequences.argtypes = [P, _VP, CLL, _VP, _VP, _VP, CI, _VP, _VP, _VP, _VP, _VP, _VP, CLL, _VP,
                                             _VP]
            L.pda_compact_blocks.argtypes = [P, _VP, CLL, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, CLL, _VP, _VP]
            L.pda_summary_size.argtypes = [P, CLL]
            L.pda_summary_size.restype = CLL
            L.pda_summarize_blocks.argtypes = [P, _VP, CLL, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
            L.pda_score_blocks.argtypes = [P, _VP, _VP, CLL, _VP, _VP, _VP, _VP, _VP]
            L.pda_select_blocks.argtypes = [P, _VP, _VP, _VP, CI, CI, CI, _VP, _VP, _VP, _VP, _VP]
            L.pda_decode_selected.argtypes = [P, _VP, _VP, CLL, _VP, _VP, _VP, _VP, _VP, _VP, _VP, CI, _VP, _VP]
            L.pda_shared_tile_groups.argtypes = [P, CI, CI]
            L.pda_shared_tile_groups.restype = CI
            L.pda_shared_workspace_size.argtypes = [P, P]
            L.pda_shared_workspace_size.restype = CLL
            L.pda_decode_shared.argtypes = [P, P, _VP, _VP, CLL, _VP, _VP, _VP, _VP, _VP, _VP, CLL, _VP, CI, _VP, _VP]
            L.pda_decode_shared.restype = CI
            L.pda_write_kv.argtypes = [P, _VP, _VP, CLL, CLL, CLL, _VP, CLL, _VP, _VP, _VP, _VP, _VP, _VP]
            L.pda_read_kv.argtypes = [P, _VP, CLL, _VP, _VP, _VP, _VP, CLL, _VP, _VP, CI, _VP, _VP]
            L.pda_tree_workspace_size.argtypes = [P, CLL]
            L.pda_tree_workspace_size.restype = CLL
            L.pda_decode_tree.argtypes = [P, _VP, CLL, _VP, CLL, _VP, _VP, _VP, _VP, _VP, CI, CI, CI, _VP, CLL, _VP, CI, _VP,
                                          _VP]
            L.pda_accept_tokens.argtypes = [P, _VP, CLL, _VP, _VP, _VP, _VP, CI, _VP, _VP, _VP]
            L.pda_decode_window.argtypes = [P, _VP, _VP, CLL, _VP, _VP, _VP, CI, CI, _VP, CI, _VP, _VP]
            for f in (L.pda_write_kv, L.pda_read_kv, L.pda_decode_tree, L.pda_accept_tokens, L.pda_decode_window):
                f.restype = CI
            for f in (L.pda_copy_blocks, L.pda_fork_sequences, L.pda_compact_blocks, L.pda_summarize_blocks,
                      L.pda_score_blocks, L.pda_select_blocks, L.pda_decode_selected):
                f.restype = CI
            L.pda_kernel_variant.argtypes = [P]
            L.pda_kernel_variant.restype = ctypes.c_int
            L.pda_plan_struct_size.argtypes = []
            L.pda_plan_struct_size.restype = ctypes.c_int
            if L.pda_plan_struct_size() != ctypes.sizeof(Plan):
                raise RuntimeError("pda_plan_t layout mismatch between include/pda.h and the binding")
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pda_status_string(status).decode()


def plan(num_seqs: int, num_kv_heads: int, query_group_size: int, kv_block_size: int, max_blocks_per_seq: int,
         tile_groups_per_partition: int = 1, max_partitions: int = 0, kv_dtype: int = KV_BF16,
         softmax_scale: float = 0.0, head_dim: int = HEAD_DIM, wait_timeout_ns: int = 0,
         kernel_variant: int = 0) -> Plan:
    p = Plan(num_seqs, num_kv_heads, query_group_size, head_dim, kv_block_size, max_blocks_per_seq,
             tile_groups_per_partition, max_partitions, kv_dtype, softmax_scale, wait_timeout_ns, kernel_variant)
    rc = lib().pda_plan(ctypes.byref(p))
    if rc != 0:
        raise PdaError(rc, "pda_plan")
    return p


def kernel_variant(p: Plan) -> int:
    """pda_kernel_variant: the partition-pass layout pda_decode launches for this plan on the
    current device (VARIANT_HEAD_WARPS, VARIANT_HEAD_GROUPS or VARIANT_ROW_HALVES)."""
    rc = lib().pda_kernel_variant(ctypes.byref(p))
    if rc < 0:
        raise PdaError(rc, "pda_kernel_variant")
    return rc


def partial_shapes(p: Plan):
    B, Hk, P, QG = p.num_seqs, p.num_kv_heads, p.num_partitions, p.query_group_size
    return (B, Hk, P, QG, p.head_dim), (B, Hk, P, QG)


def workspace(p: Plan, device, fill: float | None = None) -> dict:
    """partial_out / exp_sums / max_logits for one step (allocated by torch)."""
    so, ss = partial_shapes(p)
    mk = (lambda s: torch.empty(s, dtype=torch.float32, device=device)) if fill is None else \
        (lambda s: torch.full(s, fill, dtype=torch.float32, device=device))
    return {"partial_out": mk(so), "exp_sums": mk(ss), "max_logits": mk(ss)}


def _need(t: torch.Tensor, name: str, dtype, numel: int, host_ok: bool = False):
    """Pointer of a contiguous tensor of at least `numel` bytes.  With host_ok, pinned host memory
    is accepted too: the kernels then read or write it across the host link (unified addressing
    gives pinned memory one address on both sides)."""
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or (host_ok and t.device.type == "cpu" and t.is_pinned())):
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() * t.element_size() < numel:
        raise ValueError(f"{name} is too small ({t.numel() * t.element_size()} < {numel} bytes)")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream if isinstance(s, torch.cuda.Stream) else int(s))


def decode(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, partial_out, exp_sums,
           max_logits, err_word=None, stream=None) -> None:
    """pda_decode: the partition pass (see include/pda.h)."""
    B, Hk, QG, D, P = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim, p.num_partitions
    args = (
        _need(query, "query", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * QG * D * 2, host_ok=True),
        _need(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes),
        ctypes.c_longlong(num_cache_blocks),
        _need(block_table, "block_table", torch.int32, B * p.max_blocks_per_seq * 4, host_ok=True),
        _need(context_lens, "context_lens", torch.int32, B * 4, host_ok=True),
        _need(partial_out, "partial_out", torch.float32, B * Hk * P * QG * D * 4),
        _need(exp_sums, "exp_sums", torch.float32, B * Hk * P * QG * 4),
        _need(max_logits, "max_logits", torch.float32, B * Hk * P * QG * 4),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_decode(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_decode")


def decode_tq4(p: Plan, query, kv_cache, num_cache_blocks: int, centroids, block_table, context_lens, partial_out,
               exp_sums, max_logits, err_word=None, stream=None) -> None:
    """pda_decode_tq4: the partition pass over a TQ4 cache (see include/pda.h); centroids: fp32 [16]."""
    B, Hk, QG, D, P = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim, p.num_partitions
    args = (
        _need(query, "query", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * QG * D * 2, host_ok=True),
        _need(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes),
        ctypes.c_longlong(num_cache_blocks),
        _need(centroids, "centroids", torch.float32, 16 * 4),
        _need(block_table, "block_table", torch.int32, B * p.max_blocks_per_seq * 4, host_ok=True),
        _need(context_lens, "context_lens", torch.int32, B * 4, host_ok=True),
        _need(partial_out, "partial_out", torch.float32, B * Hk * P * QG * D * 4),
        _need(exp_sums, "exp_sums", torch.float32, B * Hk * P * QG * 4),
        _need(max_logits, "max_logits", torch.float32, B * Hk * P * QG * 4),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_decode_tq4(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_decode_tq4")


def reduce(p: Plan, context_lens, partial_out, exp_sums, max_logits, out, err_word=None, stream=None) -> None:
    """pda_reduce: combines the partials into out [B][Hk*QG][D] (bf16 or fp32 by out's dtype)."""
    B, Hk, QG, D, P = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim, p.num_partitions
    out_dtype = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    args = (
        _need(context_lens, "context_lens", torch.int32, B * 4, host_ok=True),
        _need(partial_out, "partial_out", torch.float32, B * Hk * P * QG * D * 4),
        _need(exp_sums, "exp_sums", torch.float32, B * Hk * P * QG * 4),
        _need(max_logits, "max_logits", torch.float32, B * Hk * P * QG * 4),
        _need(out, "out", (torch.float32, torch.bfloat16), B * Hk * QG * D * out.element_size(), host_ok=True),
        ctypes.c_int(out_dtype),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_reduce(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_reduce")


def append_kv(p: Plan, k_new, v_new, kv_cache, num_cache_blocks: int, block_table, positions, err_word=None,
              stream=None) -> None:
    """pda_append_kv: writes one new token per sequence into the paged cache (see include/pda.h).
    k_new, v_new: bf16 [B][Hk][D]; positions: int32 [B] (negative: no write)."""
    B, Hk, D = p.num_seqs, p.num_kv_heads, p.head_dim
    args = (
        _need(k_new, "k_new", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * D * 2),
        _need(v_new, "v_new", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * D * 2),
        _need(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes),
        ctypes.c_longlong(num_cache_blocks),
        _need(block_table, "block_table", torch.int32, B * p.max_blocks_per_seq * 4),
        _need(positions, "positions", torch.int32, B * 4),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_append_kv(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_append_kv")


def counters(p: Plan, device):
    """The fused step's reserved counters argument, int32 [B][Hk], zeroed (the step leaves them zero)."""
    return torch.zeros((p.num_seqs, p.num_kv_heads), dtype=torch.int32, device=device)


def decode_fused(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, partial_out, exp_sums,
                 max_logits, counters, out, err_word=None, stream=None) -> None:
    """pda_decode_fused: the partition pass and the reduce in one launch (see include/pda.h)."""
    B, Hk, QG, D, P = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim, p.num_partitions
    out_dtype = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    args = (
        _need(query, "query", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * QG * D * 2, host_ok=True),
        _need(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes),
        ctypes.c_longlong(num_cache_blocks),
        _need(block_table, "block_table", torch.int32, B * p.max_blocks_per_seq * 4, host_ok=True),
        _need(context_lens, "context_lens", torch.int32, B * 4, host_ok=True),
        _need(partial_out, "partial_out", torch.float32, B * Hk * P * QG * D * 4),
        _need(exp_sums, "exp_sums", torch.float32, B * Hk * P * QG * 4),
        _need(max_logits, "max_logits", torch.float32, B * Hk * P * QG * 4),
        _need(counters, "counters", torch.int32, B * Hk * 4),
        _need(out, "out", (torch.float32, torch.bfloat16), B * Hk * QG * D * out.element_size(), host_ok=True),
        ctypes.c_int(out_dtype),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_decode_fused(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_decode_fused")


def decode_step(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, ws: dict | None = None,
                out=None, out_dtype=torch.bfloat16, err_word=None, stream=None, centroids=None):
    """pda_decode (pda_decode_tq4 for a TQ4 plan, with its centroids) then pda_reduce on one stream;
    returns out [B][Hk*QG][D]."""
    if ws is None:
        ws = workspace(p, query.device)
    if out is None:
        out = torch.empty((p.num_seqs, p.num_kv_heads * p.query_group_size, p.head_dim), dtype=out_dtype,
                          device=query.device)
    if p.kv_dtype == KV_TQ4:
        decode_tq4(p, query, kv_cache, num_cache_blocks, centroids, block_table, context_lens, ws["partial_out"],
                   ws["exp_sums"], ws["max_logits"], err_word=err_word, stream=stream)
    else:
        decode(p, query, kv_cache, num_cache_blocks, block_table, context_lens, ws["partial_out"], ws["exp_sums"],
               ws["max_logits"], err_word=err_word, stream=stream)
    reduce(p, context_lens, ws["partial_out"], ws["exp_sums"], ws["max_logits"], out, err_word=err_word,
           stream=stream)
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20


def decode_step_noalloc(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, out,
                        err_word=None, stream=None) -> None:
    """pda_decode_step_noalloc: a whole step with the partials kept inside the library, for callers
    that cannot allocate a workspace (see include/pda.h).  out [B][Hk*QG][D], bf16 or fp32."""
    B, Hk, QG, D = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim
    out_dtype = OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    args = (
        _need(query, "query", (torch.bfloat16, torch.int16, torch.uint16), B * Hk * QG * D * 2, host_ok=True),
        _need(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes),
        ctypes.c_longlong(num_cache_blocks),
        _need(block_table, "block_table", torch.int32, B * p.max_blocks_per_seq * 4, host_ok=True),
        _need(context_lens, "context_lens", torch.int32, B * 4, host_ok=True),
        _need(out, "out", (torch.float32, torch.bfloat16), B * Hk * QG * D * out.element_size(), host_ok=True),
        ctypes.c_int(out_dtype),
        None if err_word is None else _need(err_word, "err_word", torch.int32, 4),
        _stream(stream),
    )
    rc = lib().pda_decode_step_noalloc(ctypes.byref(p), *args)
    if rc != 0:
        raise PdaError(rc, "pda_decode_step_noalloc")


# ------------------------------------------------------------------------------------------------
# Pages of the cache, attention over selected blocks, and shared prefixes.  Every tensor of a call lies on one GPU,
# which the call makes current; `stream` defaults to that GPU's current stream.
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)


class _Call:
    """Checks the tensors of one call: on the device of the first, contiguous, large enough."""

    __slots__ = ("index",)

    def __init__(self, t: torch.Tensor, name: str):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        self.index = t.get_device()

    def ptr(self, t, name: str, dtype, nbytes: int, host_ok: bool = False):
        # the common case first and short: a step of many short kernels waits for this code
        try:
            if (t.get_device() == self.index and (dtype is None or t.dtype in dtype) and t.is_contiguous()
                    and t.nbytes >= nbytes):
                return t.data_ptr()
        except AttributeError:   # no tensor
            pass
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != self.index and not (host_ok and t.device.type == "cpu" and t.is_pinned()):
            raise ValueError(f"{name} must be on cuda:{self.index}" + (" or pinned host memory" if host_ok else ""))
        if dtype is not None and t.dtype not in dtype:
            raise ValueError(f"{name} has dtype {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.nbytes < nbytes:
            raise ValueError(f"{name} is too small ({t.nbytes} < {nbytes} bytes)")
        return t.data_ptr()

    def opt(self, t, name: str, dtype, nbytes: int):
        return None if t is None else self.ptr(t, name, dtype, nbytes)

    def run(self, what: str, fn, p: Plan, args: tuple, err_word, stream) -> None:
        err = None if err_word is None else self.ptr(err_word, "err_word", _I32, 4)
        if torch._C._cuda_getDevice() == self.index:
            rc = fn(p, *args, err, self._stream(stream))
        else:
            with torch.cuda.device(self.index):
                rc = fn(p, *args, err, self._stream(stream))
        if rc != 0:
            raise PdaError(rc, what)

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.index)
        return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _made(make, index: int, stream):
    """What a call allocates for itself is its stream's: no other stream uses it still, and it comes back in the
    stream's order."""
    if stream is None:
        return make()
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=index)
    with torch.cuda.stream(s):
        return make()


def copy_blocks(p: Plan, src_cache, src_blocks: int, dst_cache, dst_blocks: int, pairs, err_word=None,
                stream=None) -> None:
    """pda_copy_blocks: block pairs[i, 0] of src_cache to block pairs[i, 1] of dst_cache (see
    include/pda.h).  pairs: int32 [n][2].  Either cache may be pinned host memory."""
    c = _Call(pairs, "pairs")
    n = pairs.numel() // 2
    if pairs.numel() != 2 * n:
        raise ValueError("pairs must hold two ids per pair")
    cbb = p.cache_block_bytes
    args = (c.ptr(src_cache, "src_cache", None, src_blocks * cbb, host_ok=True), src_blocks,
            c.ptr(dst_cache, "dst_cache", None, dst_blocks * cbb, host_ok=True), dst_blocks,
            c.ptr(pairs, "pairs", _I32, n * 8), n)
    c.run("pda_copy_blocks", lib().pda_copy_blocks, p, args, err_word, stream)


def page_workspace(p: Plan, num_rows: int, num_cache_blocks: int, device):
    """The workspace of fork_sequences with up to num_rows rows, and of compact_blocks."""
    n = lib().pda_page_workspace_size(p, num_rows, num_cache_blocks)
    if n < 0:
        raise PdaError(-1, "pda_page_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def fork_sequences(p: Plan, kv_cache, num_cache_blocks: int, block_table, context_lens, refcounts, parents, out_table,
                   out_lens, out_refcounts, workspace, new_tokens=None, err_word=None, stream=None) -> None:
    """pda_fork_sequences: row i of the new batch is old sequence parents[i] grown by new_tokens[i]
    positions; sequences that no row names are freed (see include/pda.h, also for what a model's other pools and
    block summaries need).  parents: int32 [R];
    out_table: int32 [R][max_blocks_per_seq]; workspace: page_workspace(p, R, ...) or larger."""
    c = _Call(kv_cache, "kv_cache")
    B, MB, NB, R = p.num_seqs, p.max_blocks_per_seq, num_cache_blocks, parents.numel()
    args = (c.ptr(kv_cache, "kv_cache", None, NB * p.cache_block_bytes), NB,
            c.ptr(block_table, "block_table", _I32, B * MB * 4), c.ptr(context_lens, "context_lens", _I32, B * 4),
            c.ptr(refcounts, "refcounts", _I32, NB * 4), R, c.ptr(parents, "parents", _I32, R * 4),
            c.opt(new_tokens, "new_tokens", _I32, R * 4), c.ptr(out_table, "out_table", _I32, R * MB * 4),
            c.ptr(out_lens, "out_lens", _I32, R * 4), c.ptr(out_refcounts, "out_refcounts", _I32, NB * 4),
            c.ptr(workspace, "workspace", _U8, 0), workspace.nbytes)
    c.run("pda_fork_sequences", lib().pda_fork_sequences, p, args, err_word, stream)


def compact_blocks(p: Plan, kv_cache, num_cache_blocks: int, block_table, context_lens, refcounts, out_table,
                   out_refcounts, remap, num_used, workspace, err_word=None, stream=None) -> None:
    """pda_compact_blocks: moves the blocks in use to the low end of the pool (see include/pda.h).  Block summaries and other
    pools under the same tables are not moved: copy_blocks with the pairs (id, remap[id]); summaries[remap[used]] = summaries[used] with used = remap >= 0."""
    c = _Call(kv_cache, "kv_cache")
    B, MB, NB = p.num_seqs, p.max_blocks_per_seq, num_cache_blocks
    args = (c.ptr(kv_cache, "kv_cache", None, NB * p.cache_block_bytes), NB,
            c.ptr(block_table, "block_table", _I32, B * MB * 4), c.ptr(context_lens, "context_lens", _I32, B * 4),
            c.ptr(refcounts, "refcounts", _I32, NB * 4), c.ptr(out_table, "out_table", _I32, B * MB * 4),
            c.ptr(out_refcounts, "out_refcounts", _I32, NB * 4), c.ptr(remap, "remap", _I32, NB * 4),
            c.ptr(num_used, "num_used", _I32, 4), c.ptr(workspace, "workspace", _U8, 0), workspace.nbytes)
    c.run("pda_compact_blocks", lib().pda_compact_blocks, p, args, err_word, stream)


def block_summaries(p: Plan, num_cache_blocks: int, device):
    """Summaries of every block: bf16 [num_cache_blocks][num_kv_heads][2: max, min][128]."""
    return torch.empty((num_cache_blocks, p.num_kv_heads, 2, p.head_dim), dtype=torch.bfloat16, device=device)


def summarize_blocks(p: Plan, kv_cache, num_cache_blocks: int, block_table, context_lens, summaries, since=None,
                     centroids=None, err_word=None, stream=None) -> None:
    """pda_summarize_blocks: renews the summaries of the blocks with tokens since[b] and later (all
    blocks without `since`; see include/pda.h).  centroids: fp32 [16], for a TQ4 plan."""
    c = _Call(kv_cache, "kv_cache")
    B, MB, NB = p.num_seqs, p.max_blocks_per_seq, num_cache_blocks
    args = (c.ptr(kv_cache, "kv_cache", None, NB * p.cache_block_bytes), NB,
            c.ptr(block_table, "block_table", _I32, B * MB * 4), c.ptr(context_lens, "context_lens", _I32, B * 4),
            c.opt(since, "since", _I32, B * 4), c.opt(centroids, "centroids", _F32, 64),
            c.ptr(summaries, "summaries", _BF16, NB * p.num_kv_heads * 512))
    c.run("pda_summarize_blocks", lib().pda_summarize_blocks, p, args, err_word, stream)


def score_blocks(p: Plan, query, summaries, num_cache_blocks: int, block_table, context_lens, scores, err_word=None,
                 stream=None) -> None:
    """pda_score_blocks: an upper bound of every block's logits, fp32 [B][Hk][max_blocks_per_seq]
    (see include/pda.h)."""
    c = _Call(summaries, "summaries")
    B, Hk, MB, NB = p.num_seqs, p.num_kv_heads, p.max_blocks_per_seq, num_cache_blocks
    args = (c.ptr(query, "query", _BF16, B * Hk * p.query_group_size * p.head_dim * 2),
            c.ptr(summaries, "summaries", _BF16, NB * Hk * 512), NB,
            c.ptr(block_table, "block_table", _I32, B * MB * 4), c.ptr(context_lens, "context_lens", _I32, B * 4),
            c.ptr(scores, "scores", _F32, B * Hk * MB * 4))
    c.run("pda_score_blocks", lib().pda_score_blocks, p, args, err_word, stream)


def select_blocks(p: Plan, scores, block_table, context_lens, num_select: int, num_first: int, num_last: int,
                  sel_table, sel_lens, sel_blocks=None, err_word=None, stream=None) -> None:
    """pda_select_blocks: the blocks each (sequence, KV head) attends to (see include/pda.h).
    sel_table, sel_blocks: int32 [B][Hk][num_select]; sel_lens: int32 [B][Hk]."""
    c = _Call(scores, "scores")
    B, Hk, MB = p.num_seqs, p.num_kv_heads, p.max_blocks_per_seq
    need = B * Hk * max(num_select, 0) * 4
    args = (c.ptr(scores, "scores", _F32, B * Hk * MB * 4),
            c.ptr(block_table, "block_table", _I32, B * MB * 4), c.ptr(context_lens, "context_lens", _I32, B * 4),
            num_select, num_first, num_last, c.ptr(sel_table, "sel_table", _I32, need),
            c.ptr(sel_lens, "sel_lens", _I32, B * Hk * 4), c.opt(sel_blocks, "sel_blocks", _I32, need))
    c.run("pda_select_blocks", lib().pda_select_blocks, p, args, err_word, stream)


def decode_selected(p: Plan, query, kv_cache, num_cache_blocks: int, sel_table, sel_lens, ws: dict | None = None,
                    out=None, out_dtype=torch.bfloat16, centroids=None, err_word=None, stream=None):
    """pda_decode_selected: a decode step over the blocks in sel_table [B][Hk][max_blocks_per_seq],
    sel_lens [B][Hk] tokens (see include/pda.h); returns out [B][Hk*QG][D].  ws: the partials of a plan
    with kernel_variant VARIANT_HEAD_WARPS (made if None); other plans need none."""
    c = _Call(kv_cache, "kv_cache")
    B, Hk, QG, D, P = p.num_seqs, p.num_kv_heads, p.query_group_size, p.head_dim, p.num_partitions
    if out is None:
        out = _made(lambda: torch.empty((B, Hk * QG, D), dtype=out_dtype, device=kv_cache.device), c.index, stream)
    rows = B * Hk * QG
    f32 = out.dtype is torch.float32
    partials = (None, None, None)
    if p.kernel_variant == VARIANT_HEAD_WARPS:
        if ws is None:
            ws = _made(lambda: workspace(p, kv_cache.device), c.index, stream)
        partials = (c.ptr(ws["partial_out"], "partial_out", _F32, rows * P * D * 4),
                    c.ptr(ws["exp_sums"], "exp_sums", _F32, rows * P * 4),
                    c.ptr(ws["max_logits"], "max_logits", _F32, rows * P * 4))
    args = (c.ptr(query, "query", _BF16, rows * D * 2, host_ok=True),
            c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.opt(centroids, "centroids", _F32, 64),
            c.ptr(sel_table, "sel_table", _I32, B * Hk * p.max_blocks_per_seq * 4),
            c.ptr(sel_lens, "sel_lens", _I32, B * Hk * 4), *partials,
            c.ptr(out, "out", (torch.float32, torch.bfloat16), rows * D * (4 if f32 else 2), host_ok=True),
            OUT_F32 if f32 else OUT_BF16)
    c.run("pda_decode_selected", lib().pda_decode_selected, p, args, err_word, stream)
    return out


def shared_plans(num_seqs: int, num_groups: int, num_kv_heads: int, query_group_size: int, kv_block_size: int,
                 prefix_blocks: int, max_blocks_per_seq: int, kv_dtype: int = KV_BF16, softmax_scale: float = 0.0,
                 tile_groups_per_partition: int = 1, prefix_tile_groups: int = 0, wait_timeout_ns: int = 0):
    """The two plans of decode_shared: of the prefixes (num_groups tables of prefix_blocks entries) and of
    the sequences' own tokens.  prefix_tile_groups 0 asks pda_shared_tile_groups."""
    p = plan(num_seqs, num_kv_heads, query_group_size, kv_block_size, max_blocks_per_seq, tile_groups_per_partition,
             kv_dtype=kv_dtype, softmax_scale=softmax_scale, wait_timeout_ns=wait_timeout_ns)
    if prefix_tile_groups == 0:
        prefix_tile_groups = lib().pda_shared_tile_groups(p, num_groups, prefix_blocks)
        if prefix_tile_groups < 0:
            raise PdaError(prefix_tile_groups, "pda_shared_tile_groups")
    pp = plan(num_groups, num_kv_heads, query_group_size, kv_block_size, prefix_blocks, prefix_tile_groups,
              kv_dtype=kv_dtype, softmax_scale=softmax_scale, wait_timeout_ns=wait_timeout_ns)
    return pp, p


def shared_workspace(prefix_plan: Plan, p: Plan, device):
    """The workspace of decode_shared (torch memory is aligned far beyond what it needs)."""
    n = lib().pda_shared_workspace_size(prefix_plan, p)
    if n < 0:
        raise PdaError(-1, "pda_shared_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def decode_shared(prefix_plan: Plan, p: Plan, query, kv_cache, num_cache_blocks: int, group_starts, prefix_table,
                  prefix_lens, block_table, context_lens, ws=None, out=None, out_dtype=torch.bfloat16, err_word=None,
                  stream=None):
    """pda_decode_shared: a decode step over each group's shared prefix and each sequence's own tokens
    (see include/pda.h); returns out [B][Hk*QG][D]."""
    c = _Call(kv_cache, "kv_cache")
    B, NG = p.num_seqs, prefix_plan.num_seqs
    if ws is None:
        ws = _made(lambda: shared_workspace(prefix_plan, p, kv_cache.device), c.index, stream)
    if out is None:
        shape = (B, p.num_kv_heads * p.query_group_size, p.head_dim)
        out = _made(lambda: torch.empty(shape, dtype=out_dtype, device=kv_cache.device), c.index, stream)
    n = B * p.num_kv_heads * p.query_group_size * p.head_dim
    f32 = out.dtype is torch.float32
    args = (p, c.ptr(query, "query", _BF16, n * 2, host_ok=True),
            c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.ptr(group_starts, "group_starts", _I32, (NG + 1) * 4),
            c.ptr(prefix_table, "prefix_table", _I32, NG * prefix_plan.max_blocks_per_seq * 4),
            c.ptr(prefix_lens, "prefix_lens", _I32, NG * 4),
            c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4),
            c.ptr(context_lens, "context_lens", _I32, B * 4), c.ptr(ws, "ws", _U8, 0), ws.nbytes,
            c.ptr(out, "out", (torch.float32, torch.bfloat16), n * (4 if f32 else 2), host_ok=True),
            OUT_F32 if f32 else OUT_BF16)
    c.run("pda_decode_shared", lib().pda_decode_shared, prefix_plan, args, err_word, stream)
    return out


# ------------------------------------------------------------------------------------------------
# Many tokens per sequence, drafted tokens, sliding windows.  Rows token_starts[b] .. token_starts[b+1]-1 of the packed
# arrays are sequence b's.
def _rows(c: _Call, t, name: str, p: Plan):
    """Pointer and row stride (elements) of bf16 [N][Hk][128] whose rows may lie apart."""
    try:   # the common case first and short, as in _Call.ptr
        n, heads, dims = t.shape
        stride, between, step = t.stride()
        if (t.get_device() == c.index and t.dtype in _BF16 and heads == p.num_kv_heads and dims == p.head_dim == between
                and step == 1 and stride >= heads * dims and n > 1):
            return t.data_ptr(), stride
    except (AttributeError, ValueError):   # no tensor, or not of three dimensions
        pass
    if not isinstance(t, torch.Tensor) or t.get_device() != c.index:
        raise ValueError(f"{name} must be on cuda:{c.index}")
    if t.dtype not in _BF16:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if t.dim() != 3 or t.shape[1] != p.num_kv_heads or t.shape[2] != p.head_dim:
        raise ValueError(f"{name} must be [tokens][{p.num_kv_heads}][{p.head_dim}]")
    row = p.num_kv_heads * p.head_dim
    if t.shape[0] <= 1 or t.numel() == 0:
        stride = row
    else:
        stride = t.stride(0)
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != p.head_dim) or stride < row):
        raise ValueError(f"{name} must hold whole rows: only the first stride is free")
    return t.data_ptr(), stride


def _int32(x: int, name: str) -> int:
    """ctypes would take a larger number modulo 2^32."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return x


def _tokens(t, name: str, heads: int, dims: int) -> int:
    """How many tokens of [heads][dims] a packed tensor holds: nothing else may be left, and rows of other heads are refused."""
    n = t.numel() // (heads * dims)
    if t.numel() != n * heads * dims or (t.dim() > 2 and t.shape[-1] != dims) or (t.dim() == 3 and t.shape[0] != n):
        raise ValueError(f"{name} must be [tokens][{heads}][{dims}]")
    return n


def write_kv(p: Plan, k_new, v_new, kv_cache, num_cache_blocks: int, block_table, token_starts, positions, centroids=None,
             err_word=None, stream=None) -> None:
    """pda_write_kv: K and V of any number of new tokens per sequence, in the cache's format (see include/pda.h).
    k_new, v_new: bf16 [N][Hk][128], rows of any stride that is a multiple of 8 elements; token_starts: int32 [B + 1];
    positions: int32 [B]; centroids: fp32 [16], for a TQ4 plan."""
    c = _Call(kv_cache, "kv_cache")
    B = p.num_seqs
    (k, ks), (v, vs) = _rows(c, k_new, "k_new", p), _rows(c, v_new, "v_new", p)
    N = k_new.shape[0]
    if v_new.shape[0] != N:
        raise ValueError("k_new and v_new must hold the same tokens")
    args = (k, v, ks, vs, N, c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.opt(centroids, "centroids", _F32, 64), c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4),
            c.ptr(token_starts, "token_starts", _I32, (B + 1) * 4), c.ptr(positions, "positions", _I32, B * 4))
    c.run("pda_write_kv", lib().pda_write_kv, p, args, err_word, stream)


def read_kv(p: Plan, kv_cache, num_cache_blocks: int, block_table, token_starts, positions, k_out, v_out, centroids=None,
            err_word=None, stream=None) -> None:
    """pda_read_kv: tokens of the cache, gathered and dequantised into k_out, v_out [N][Hk][128], bf16 or fp32 (see
    include/pda.h).  One of the two may be None."""
    c = _Call(kv_cache, "kv_cache")
    B, row = p.num_seqs, p.num_kv_heads * p.head_dim
    given = [(t, n) for t, n in ((k_out, "k_out"), (v_out, "v_out")) if t is not None]
    if not given:
        raise ValueError("k_out or v_out must be given")
    dtype = given[0][0].dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"k_out and v_out have dtype {dtype}")
    N = [_tokens(t, n, p.num_kv_heads, p.head_dim) for t, n in given][0]
    outs = tuple(c.opt(t, n, (dtype,), N * row * dtype.itemsize) for t, n in ((k_out, "k_out"), (v_out, "v_out")))
    args = (c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.opt(centroids, "centroids", _F32, 64), c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4),
            c.ptr(token_starts, "token_starts", _I32, (B + 1) * 4), c.ptr(positions, "positions", _I32, B * 4), N, *outs,
            OUT_F32 if dtype is torch.float32 else OUT_BF16)
    c.run("pda_read_kv", lib().pda_read_kv, p, args, err_word, stream)


def tree_workspace(p: Plan, num_tokens: int, device):
    """The workspace of decode_tree with up to num_tokens drafted tokens in all."""
    n = lib().pda_tree_workspace_size(p, num_tokens)
    if n < 0:
        raise PdaError(-1, "pda_tree_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def decode_tree(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, token_starts, tree_masks=None,
                window: int = 0, num_first: int = 0, centroids=None, ws=None, out=None, out_dtype=torch.bfloat16,
                err_word=None, stream=None):
    """pda_decode_tree: a step for drafted tokens in chains (tree_masks None) or trees (see include/pda.h); query: bf16
    [N][Hk*QG][128], tree_masks: int64 [N][words]; returns out [N][Hk*QG][128]."""
    c = _Call(kv_cache, "kv_cache")
    B, rows, D = p.num_seqs, p.num_kv_heads * p.query_group_size, p.head_dim
    N = _tokens(query, "query", rows, D)
    words = 0
    if tree_masks is not None:
        if tree_masks.dim() != 2 or tree_masks.shape[0] < N or tree_masks.shape[1] < 1:
            raise ValueError("tree_masks must be [tokens][words]")
        words = tree_masks.shape[1]
    if ws is None:
        ws = _made(lambda: tree_workspace(p, N, kv_cache.device), c.index, stream)
    if out is None:
        out = _made(lambda: torch.zeros((N, rows, D), dtype=out_dtype, device=kv_cache.device), c.index, stream)
    n = N * rows * D
    f32 = out.dtype is torch.float32
    args = (c.ptr(query, "query", _BF16, n * 2, host_ok=True), N,
            c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.opt(centroids, "centroids", _F32, 64), c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4),
            c.ptr(context_lens, "context_lens", _I32, B * 4), c.ptr(token_starts, "token_starts", _I32, (B + 1) * 4),
            c.opt(tree_masks, "tree_masks", (torch.int64, torch.uint64), N * words * 8), words,
            _int32(window, "window"), _int32(num_first, "num_first"),
            c.ptr(ws, "ws", _U8, 0), ws.nbytes, c.ptr(out, "out", (torch.float32, torch.bfloat16), n * (4 if f32 else 2), host_ok=True),
            OUT_F32 if f32 else OUT_BF16)
    c.run("pda_decode_tree", lib().pda_decode_tree, p, args, err_word, stream)
    return out


def accept_tokens(p: Plan, kv_cache, num_cache_blocks: int, block_table, context_lens, path, path_lens, out_lens,
                  err_word=None, stream=None) -> None:
    """pda_accept_tokens: the accepted drafted tokens move to consecutive positions (see include/pda.h).
    path: int32 [B][max_path], ascending, rows past the B sequences' not looked at; path_lens, out_lens: int32 [B]."""
    c = _Call(kv_cache, "kv_cache")
    B = p.num_seqs
    if path.dim() != 2 or path.shape[0] < B:
        raise ValueError("path must be [sequences][max_path]")
    A = path.shape[1]
    args = (c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4),
            c.ptr(context_lens, "context_lens", _I32, B * 4), c.ptr(path, "path", _I32, B * A * 4),
            c.ptr(path_lens, "path_lens", _I32, B * 4), A, c.ptr(out_lens, "out_lens", _I32, B * 4))
    c.run("pda_accept_tokens", lib().pda_accept_tokens, p, args, err_word, stream)


def decode_window(p: Plan, query, kv_cache, num_cache_blocks: int, block_table, context_lens, window: int,
                  num_first: int = 0, centroids=None, out=None, out_dtype=torch.bfloat16, err_word=None, stream=None):
    """pda_decode_window: a decode step over the last `window` tokens and the first num_first (see include/pda.h);
    returns out [B][Hk*QG][D]."""
    c = _Call(kv_cache, "kv_cache")
    B, rows, D = p.num_seqs, p.num_kv_heads * p.query_group_size, p.head_dim
    if out is None:
        out = _made(lambda: torch.empty((B, rows, D), dtype=out_dtype, device=kv_cache.device), c.index, stream)
    n = B * rows * D
    f32 = out.dtype is torch.float32
    args = (c.ptr(query, "query", _BF16, n * 2, host_ok=True),
            c.ptr(kv_cache, "kv_cache", None, num_cache_blocks * p.cache_block_bytes), num_cache_blocks,
            c.opt(centroids, "centroids", _F32, 64),
            c.ptr(block_table, "block_table", _I32, B * p.max_blocks_per_seq * 4, host_ok=True),
            c.ptr(context_lens, "context_lens", _I32, B * 4, host_ok=True), _int32(window, "window"),
            _int32(num_first, "num_first"),
            c.ptr(out, "out", (torch.float32, torch.bfloat16), n * (4 if f32 else 2), host_ok=True),
            OUT_F32 if f32 else OUT_BF16)
    c.run("pda_decode_window", lib().pda_decode_window, p, args, err_word, stream)
    return out
