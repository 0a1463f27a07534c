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
