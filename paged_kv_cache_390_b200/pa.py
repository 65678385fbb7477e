"""Python binding of ``libpa.so`` (the C ABI in ``include/pa.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors must be CUDA tensors, contiguous, in the layouts of
``pa.h``; work is enqueued on the current torch stream (or ``stream``).  There
is no fallback: if the library is missing this module raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_F32, PA_F16, PA_BF16, PA_INT8, PA_FP8E4M3 = 0, 1, 2, 3, 4
PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_NO_SPACE = 0, 1, 2, 3, 4
DEVERR_BLOCK_ID, DEVERR_SEQ_LEN, DEVERR_SLOT, DEVERR_TIMEOUT = 1, 2, 4, 8

_FLOAT_CODES = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}
CACHE_CODES = {"f32": PA_F32, "f16": PA_F16, "bf16": PA_BF16, "int8": PA_INT8, "fp8": PA_FP8E4M3}

_lock = threading.Lock()
_lib = None


class PAError(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {status_name(status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libpa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_390_b200.build`"
                " (there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        LL = ctypes.c_int64
        sigs = {
            "pa_reshape_and_cache": (I, [P, P, I, P, P, I, P, P, P, I, I, I, I, I, P, P]),
            "pa_decode_v1": (I, [P, P, I, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F, P, P]),
            "pa_decode_v2_partition": (I, [P, P, P, P, I, P, P, I, P, P, P, I, P, I, I, I, I,
                                           I, I, F, I, I, P, P]),
            "pa_decode_v2_merge": (I, [P, I, P, P, P, P, I, I, I, I, I, P]),
            "pa_decode_v2_workspace_bytes": (S, [I, I, I, I]),
            "pa_decode_fused": (I, [P, P, I, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F, P, S,
                                    P, P]),
            "pa_decode_fused_workspace_bytes": (S, [I, I, I, I]),
            "pa_decode_fused_noalloc": (I, [P, P, I, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F,
                                            P, P]),
            "pa_decode_fused_noalloc_scratch_bytes": (S, []),
            "pa_choose_partition_size": (I, [I, I, I, I, I]),
            "pa_kv_bytes_per_token": (ctypes.c_double, [I, I, I, I]),
            "pa_status_string": (ctypes.c_char_p, [I]),
            "pa_last_cuda_error_string": (ctypes.c_char_p, []),
            "pa_get_device_error": (I, [ctypes.POINTER(ctypes.c_int), I]),
            "pa_set_decode_config": (I, [I, I]),
            "pa_set_wait_limit_ns": (I, [ctypes.c_ulonglong]),
            "pa_set_fault_injection": (I, [I]),
            "pa_set_pdl": (I, [I]),
            "pa_copy_blocks": (I, [P, P, P, P, I, P, P, P, P, I, I, P, I, I, I, I, P, P]),
            "pa_append_decode_v1": (I, [P, P, I, P, P, P, P, P, I, P, P, P, I, P, I, I, I, I, I,
                                        I, F, P, P]),
            "pa_set_prefetch_tiles": (I, [I]),
            "pa_decode_cascade": (I, [P, P, I, P, P, I, P, I, P, I, I, I, I, I, I, F, I, P, S, P,
                                      P]),
            "pa_decode_cascade_workspace_bytes": (S, [I, I, I]),
            "pa_set_cascade_config": (I, [I, I]),
            "pa_prefill": (I, [P, P, I, P, I, I, P, P, I, P, I, P, I, I, I, I, I, I, F, P, P]),
            "pa_rope_and_cache": (I, [P, P, P, P, I, LL, LL, LL, P, I, P, P, I, I, P, P, I, P, P,
                                      P, I, I, I, I, I, I, P, P]),
            "pa_decode_masked": (I, [P, P, I, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F, F, P, P,
                                     I, P, P, I, P, S, P, P]),
            "pa_decode_masked_workspace_bytes": (S, [I, I, I, I, I]),
            "pa_prefill_masked": (I, [P, P, I, P, I, I, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F,
                                      F, P, P, P, I, P, P]),
            "pa_evict": (I, [P, P, I, P, P, P, I, P, P, I, P, I, I, I, P, I, P, I, P, I, I, I, I, I,
                             P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


def status_name(status: int) -> str:
    try:
        return lib().pa_status_string(int(status)).decode()
    except Exception:                                   # library not loadable
        return f"status {status}"


def _check(rc: int, what: str) -> None:
    if rc == PA_ERR_CUDA:
        raise PAError(f"{what} ({lib().pa_last_cuda_error_string().decode()})", rc)
    if rc != PA_OK:
        raise PAError(what, rc)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _same_device(dense, rows=()) -> int:
    """Index of the CUDA device that all the tensors are on; those of `dense` contiguous."""
    first = dense[0]
    if not first.is_cuda:
        raise ValueError("tensors passed to libpa must be CUDA tensors")
    index = first.get_device()
    for t in dense:
        if t is not None:
            if t.get_device() != index:
                raise ValueError("tensors of one call must be on one CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensors passed to libpa must be contiguous")
    for t in rows:
        if t.get_device() != index:
            raise ValueError("tensors of one call must be on one CUDA device")
    return index


def _enter(index, stream):
    """Make device `index` current, and `stream` (if given) torch's stream there, so that
    what the call allocates belongs to the stream that uses it.  Returns the context to
    leave again, None in the usual case (the current device and stream)."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("the stream and the tensors must be on one CUDA device")
        ctx = torch.cuda.stream(stream)
    elif index != torch.cuda.current_device():
        ctx = torch.cuda.device(index)
    else:
        return None
    ctx.__enter__()
    return ctx


def _leave(ctx) -> None:
    if ctx is not None:
        ctx.__exit__(None, None, None)


def _addr(t):
    return None if t is None else t.data_ptr()


def _row_stride(t, T, heads, D) -> int:
    """Token stride of [T, heads, D] rows whose last two dimensions are dense."""
    token, head, elem = t.stride()
    if T and (elem != 1 or (heads > 1 and head != D)):
        raise ValueError("a token's rows must be dense")
    return token if T > 1 else heads * D


def _batch_checks(block_tables, seq_lens, num_seqs) -> None:
    if (block_tables.dtype != torch.int32 or block_tables.dim() != 2
            or block_tables.shape[0] != num_seqs or seq_lens.dtype != torch.int32
            or seq_lens.shape != (num_seqs,)):
        raise ValueError("block tables are int32 [num_seqs, width], lengths int32 [num_seqs]")


def _pool_checks(k_cache, v_cache, k_scale, v_scale, cache_dtype) -> int:
    """Shapes and dtypes of the paged pool and its scales; the cache dtype's code."""
    code = cache_code(k_cache, cache_dtype)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same shape and dtype")
    if k_cache.element_size() != (4, 2, 2, 1, 1)[code]:
        raise ValueError("the cache tensor's element size does not fit cache_dtype")
    if code in (PA_INT8, PA_FP8E4M3):
        num_blocks, block_size, num_kv_heads, _ = k_cache.shape
        for t in (k_scale, v_scale):
            if t is None or t.dtype != torch.float32 or t.shape != (num_blocks, num_kv_heads,
                                                                    block_size):
                raise ValueError("scales must be float32 [num_blocks, num_kv_heads, block_size]")
    return code


def cache_code(cache: torch.Tensor, cache_dtype: str | None = None) -> int:
    if cache_dtype is not None:
        return CACHE_CODES[cache_dtype]
    if cache.dtype in _FLOAT_CODES:
        return _FLOAT_CODES[cache.dtype]
    if cache.dtype == torch.int8:
        return PA_INT8
    if cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        return PA_FP8E4M3
    raise TypeError(f"unsupported cache dtype {cache.dtype}")


# ----------------------------------------------------------------------------------

def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, *, cache_dtype=None,
                      k_scale=None, v_scale=None, err_flag=None, stream=None) -> None:
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    rc = lib().pa_reshape_and_cache(
        _ptr(key), _ptr(value), _FLOAT_CODES[key.dtype], _ptr(k_cache), _ptr(v_cache),
        cache_code(k_cache, cache_dtype), _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping),
        key.shape[0], num_kv_heads, head_dim, block_size, num_blocks, _ptr(err_flag),
        _stream(stream))
    _check(rc, "pa_reshape_and_cache")


def rope_inv_freq(rotary_dim, base=10000.0, device="cuda") -> torch.Tensor:
    """inv_freq of pa_rope_and_cache: base ** (-2 i / rotary_dim), in 64 bits."""
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return (float(base) ** (-i / rotary_dim)).to(device)


def rope_pair_axis(sections, spread=False, device="cuda") -> torch.Tensor:
    """pair_axis of pa_rope_and_cache for axes that own sections[a] pairs each: whole
    runs in the axes' order, or (spread) the axes in turn until each has its share."""
    if spread:
        left, axis = [int(n) for n in sections], []
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(int(n))]
    return torch.tensor(axis, dtype=torch.int32, device=device)


def rope_and_cache(q, key, value, positions, inv_freq, pair_axis, k_cache, v_cache, slot_mapping,
                   *, interleaved=False, out=None, cache_dtype=None, k_scale=None, v_scale=None,
                   err_flag=None, stream=None) -> torch.Tensor:
    """Turn the query and key rows of new tokens by their rotary positions (several axes:
    positions int64 [axes, T], or [T] for one) and write the turned keys and the values
    to the paged cache, in one launch; returns the turned queries.  q [T, H, D] and key,
    value [T, H_kv, D] may be slices of a fused projection (rows dense, any token
    stride); out=q turns dense queries in place."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_tokens, num_heads, q_dim = q.shape
    num_axes = positions.shape[0] if positions.dim() == 2 else 1
    rows, pairs, dtype = (num_tokens, num_kv_heads, head_dim), inv_freq.shape, q.dtype
    if (q_dim != head_dim or key.shape != rows or value.shape != rows
            or positions.shape[-1] != num_tokens or positions.dim() > 2
            or slot_mapping.shape != (num_tokens,) or pair_axis.shape != pairs or len(pairs) != 1):
        raise ValueError("shapes of q, key, value, positions, slots, frequencies and caches differ")
    if key.dtype != dtype or value.dtype != dtype:
        raise ValueError("key and value must have q's dtype")
    if (positions.dtype != torch.int64 or slot_mapping.dtype != torch.int64
            or inv_freq.dtype != torch.float64 or pair_axis.dtype != torch.int32):
        raise ValueError("positions and slots are int64, inv_freq float64, pair_axis int32")
    code = _pool_checks(k_cache, v_cache, k_scale, v_scale, cache_dtype)
    index = _same_device((k_cache, v_cache, positions, inv_freq, pair_axis, slot_mapping, k_scale,
                          v_scale, err_flag, out), (q, key, value))
    strides = (_row_stride(q, num_tokens, num_heads, head_dim),
               _row_stride(key, num_tokens, num_kv_heads, head_dim),
               _row_stride(value, num_tokens, num_kv_heads, head_dim))
    if out is not None and (out.shape != q.shape or out.dtype != dtype):
        raise ValueError("out must have q's shape and dtype")
    ctx = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        rc = (_lib or lib()).pa_rope_and_cache(
            out.data_ptr(), q.data_ptr(), key.data_ptr(), value.data_ptr(), _FLOAT_CODES[dtype],
            *strides, positions.data_ptr(), num_axes, inv_freq.data_ptr(), pair_axis.data_ptr(),
            2 * pairs[0], 1 if interleaved else 0, k_cache.data_ptr(), v_cache.data_ptr(), code,
            _addr(k_scale), _addr(v_scale), slot_mapping.data_ptr(), num_tokens, num_heads,
            num_kv_heads, head_dim, block_size, num_blocks, _addr(err_flag),
            torch._C._cuda_getCurrentRawStream(index))
    finally:
        _leave(ctx)
    if rc:
        _check(rc, "pa_rope_and_cache")
    return out


def copy_blocks(src_k, src_v, dst_k, dst_v, block_mapping, *, cache_dtype=None,
                src_k_scale=None, src_v_scale=None, dst_k_scale=None, dst_v_scale=None,
                err_flag=None, stream=None) -> None:
    """Copy whole blocks: row p of block_mapping (int64 [num_pairs, 2], on the device)
    makes destination block [p, 1] a copy of source block [p, 0].  Source and
    destination pools may be the same tensors (copy-on-write) or a device pool and a
    pinned host pool (swap out / swap in)."""
    nb_src, block_size, num_kv_heads, head_dim = src_k.shape
    if dst_k.shape[1:] != src_k.shape[1:] or dst_k.dtype != src_k.dtype:
        raise ValueError("source and destination pools must have the same block shape and dtype")
    for t in (src_k, src_v, dst_k, dst_v, src_k_scale, src_v_scale, dst_k_scale, dst_v_scale):
        if t is not None and not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools must be CUDA tensors or pinned host tensors")
    if not block_mapping.is_cuda or block_mapping.dtype != torch.int64:
        raise ValueError("block_mapping must be an int64 CUDA tensor [num_pairs, 2]")
    rc = lib().pa_copy_blocks(
        _ptr(src_k), _ptr(src_v), _ptr(src_k_scale), _ptr(src_v_scale), nb_src,
        _ptr(dst_k), _ptr(dst_v), _ptr(dst_k_scale), _ptr(dst_v_scale), dst_k.shape[0],
        cache_code(src_k, cache_dtype), _ptr(block_mapping),
        block_mapping.shape[0] if block_mapping.numel() else 0, num_kv_heads, head_dim,
        block_size, _ptr(err_flag), _stream(stream))
    _check(rc, "pa_copy_blocks")


class MaskedWorkspace:
    """Workspace of pa_decode_masked; score_width is the scores' last dimension (0: calls
    without scores)."""

    def __init__(self, num_seqs, num_heads, num_kv_heads, head_dim, score_width=0, device="cuda"):
        dev = torch.device(device)
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(dev):
            self.nbytes = int(lib().pa_decode_masked_workspace_bytes(
                num_seqs, num_heads, num_kv_heads, head_dim, score_width))
            self.buf = torch.empty(max(self.nbytes, 256), dtype=torch.uint8, device=dev)
        self.address = self.buf.data_ptr()


def _row_ints(t, n, what):
    if t is not None and (t.dtype != torch.int32 or t.shape != (n,)):
        raise ValueError(f"{what} must be int32 [{n}]")


def _mask_checks(q, head_dim, num_kv_heads, slopes):
    num_heads = q.shape[1]
    if q.dim() != 3 or q.shape[2] != head_dim or num_heads % num_kv_heads:
        raise ValueError("q must be [rows, num_heads, head_dim], whole groups of heads")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (num_heads,)):
        raise ValueError("alibi_slopes must be float32 [num_heads]")


def decode_masked(q, k_cache, v_cache, block_tables, seq_lens, scale, *, softcap=0.0,
                  alibi_slopes=None, kv_start=None, window=0, scores_in=None, scores_out=None,
                  out=None, workspace: MaskedWorkspace | None = None, cache_dtype=None,
                  k_scale=None, v_scale=None, err_flag=None, stream=None) -> torch.Tensor:
    """Paged decode attention with scores capped by a tanh (softcap), a bias by distance
    (alibi_slopes float32 [H]), the start of the token's document (kv_start int32 [S]) and
    a sliding window; with scores_out (float32 [S, H_kv, width]) every cached token's
    weight, summed over its kv head's query heads, is added to scores_in."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    code = _pool_checks(k_cache, v_cache, k_scale, v_scale, cache_dtype)
    _mask_checks(q, head_dim, num_kv_heads, alibi_slopes)
    _batch_checks(block_tables, seq_lens, num_seqs)
    _row_ints(kv_start, num_seqs, "kv_start")
    width = 0
    if scores_out is not None:
        width = scores_out.shape[-1]
        for t in (scores_in, scores_out):
            if t is not None and (t.dtype != torch.float32
                                  or t.shape != (num_seqs, num_kv_heads, width)):
                raise ValueError("scores must be float32 [num_seqs, num_kv_heads, width]")
    elif scores_in is not None:
        raise ValueError("scores_in needs scores_out")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype):
        raise ValueError("out must have q's shape and dtype")
    index = _same_device((q, k_cache, v_cache, block_tables, seq_lens, alibi_slopes, kv_start,
                          scores_in, scores_out, out, k_scale, v_scale, err_flag,
                          workspace.buf if workspace is not None else None))
    ctx = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty_like(q)
        if num_seqs == 0:
            return out
        if workspace is None:
            workspace = MaskedWorkspace(num_seqs, num_heads, num_kv_heads, head_dim, width, q.device)
        rc = (_lib or lib()).pa_decode_masked(
            out.data_ptr(), q.data_ptr(), _FLOAT_CODES[q.dtype], k_cache.data_ptr(),
            v_cache.data_ptr(), code, _addr(k_scale), _addr(v_scale), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), num_seqs, num_heads, num_kv_heads, head_dim,
            block_size, num_blocks, scale, softcap, _addr(alibi_slopes), _addr(kv_start), window,
            _addr(scores_in), _addr(scores_out), width, workspace.address, workspace.nbytes,
            _addr(err_flag), torch._C._cuda_getCurrentRawStream(index))
    finally:
        _leave(ctx)
    if rc:
        _check(rc, "pa_decode_masked")
    return out


def prefill_masked(q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, *,
                   softcap=0.0, alibi_slopes=None, kv_start=None, prefix_lens=None, window=0,
                   max_query_len=None, out=None, cache_dtype=None, k_scale=None, v_scale=None,
                   err_flag=None, stream=None) -> torch.Tensor:
    """pa_prefill with changed scores: as decode_masked, with a document start per query
    row (kv_start int32 [total_q]) and a prefix that every row of its sequence sees
    (prefix_lens int32 [S])."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    total_q, num_heads, _ = q.shape
    num_seqs = seq_lens.shape[0]
    code = _pool_checks(k_cache, v_cache, k_scale, v_scale, cache_dtype)
    _mask_checks(q, head_dim, num_kv_heads, alibi_slopes)
    _batch_checks(block_tables, seq_lens, num_seqs)
    _row_ints(query_start, num_seqs + 1, "query_start")
    _row_ints(kv_start, total_q, "kv_start")
    _row_ints(prefix_lens, num_seqs, "prefix_lens")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype):
        raise ValueError("out must have q's shape and dtype")
    index = _same_device((q, k_cache, v_cache, block_tables, seq_lens, query_start, alibi_slopes,
                          kv_start, prefix_lens, out, k_scale, v_scale, err_flag))
    ctx = _enter(index, stream)
    try:
        if out is None:
            out = torch.empty_like(q)
        if num_seqs == 0 or total_q == 0:
            return out
        if max_query_len is None:
            max_query_len = int((query_start[1:] - query_start[:-1]).max())
        rc = (_lib or lib()).pa_prefill_masked(
            out.data_ptr(), q.data_ptr(), _FLOAT_CODES[q.dtype], query_start.data_ptr(), total_q,
            max_query_len, k_cache.data_ptr(), v_cache.data_ptr(), code, _addr(k_scale),
            _addr(v_scale), block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(),
            num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, softcap,
            _addr(alibi_slopes), _addr(kv_start), _addr(prefix_lens), window, _addr(err_flag),
            torch._C._cuda_getCurrentRawStream(index))
    finally:
        _leave(ctx)
    if rc:
        _check(rc, "pa_prefill_masked")
    return out


def evict(k_cache, v_cache, block_tables, seq_lens, new_block_tables, scores, num_keep, num_recent,
          *, kept=None, new_scores=None, new_lens=None, cache_dtype=None, k_scale=None,
          v_scale=None, err_flag=None, stream=None):
    """Cut sequences down to num_keep tokens per kv head: the num_recent newest and the
    highest-scored others, moved in their order to the blocks of new_block_tables (see
    BlockManager.evict).  scores float32 [S, H_kv, width].  Returns (kept int32
    [S, H_kv, num_keep], padded with -1; new_lens int32 [S]; new_scores)."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs = seq_lens.shape[0]
    code = _pool_checks(k_cache, v_cache, k_scale, v_scale, cache_dtype)
    _batch_checks(block_tables, seq_lens, num_seqs)
    _batch_checks(new_block_tables, seq_lens, num_seqs)
    if (scores.dtype != torch.float32 or scores.dim() != 3
            or scores.shape[:2] != (num_seqs, num_kv_heads)):
        raise ValueError("scores must be float32 [num_seqs, num_kv_heads, width]")
    index = _same_device((k_cache, v_cache, block_tables, seq_lens, new_block_tables, scores, kept,
                          new_scores, new_lens, k_scale, v_scale, err_flag))
    unit = (num_seqs, num_kv_heads)
    for t, dt in ((kept, torch.int32), (new_scores, torch.float32)):
        if t is not None and (t.dtype != dt or t.dim() != 3 or t.shape[:2] != unit):
            raise ValueError("kept (int32) and new_scores (float32) are "
                             "[num_seqs, num_kv_heads, width]")
    if new_lens is not None and (new_lens.dtype != torch.int32 or new_lens.shape != (num_seqs,)):
        raise ValueError("new_lens must be int32 [num_seqs]")
    ctx = _enter(index, stream)
    try:
        if kept is None:
            kept = torch.empty((*unit, num_keep), dtype=torch.int32, device=k_cache.device)
        if new_scores is None:
            new_scores = torch.zeros((*unit, num_keep), device=k_cache.device)
        if new_lens is None:
            new_lens = torch.empty(num_seqs, dtype=torch.int32, device=k_cache.device)
        if num_seqs == 0:
            return kept, new_lens, new_scores
        rc = (_lib or lib()).pa_evict(
            k_cache.data_ptr(), v_cache.data_ptr(), code, _addr(k_scale), _addr(v_scale),
            block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(),
            new_block_tables.data_ptr(), new_block_tables.shape[1], scores.data_ptr(),
            scores.shape[2], num_keep, num_recent, kept.data_ptr(), kept.shape[2],
            new_scores.data_ptr(), new_scores.shape[2], new_lens.data_ptr(), num_seqs, num_kv_heads,
            head_dim, block_size, num_blocks, _addr(err_flag),
            torch._C._cuda_getCurrentRawStream(index))
    finally:
        _leave(ctx)
    if rc:
        _check(rc, "pa_evict")
    return kept, new_lens, new_scores


def decode_v1(q, k_cache, v_cache, block_tables, seq_lens, scale, *, out=None, cache_dtype=None,
              k_scale=None, v_scale=None, err_flag=None, stream=None) -> torch.Tensor:
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    rc = lib().pa_decode_v1(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(k_cache), _ptr(v_cache),
        cache_code(k_cache, cache_dtype), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, num_heads, num_kv_heads, head_dim,
        block_size, num_blocks, float(scale), _ptr(err_flag), _stream(stream))
    _check(rc, "pa_decode_v1")
    return out


def append_decode_v1(q, key, value, slot_mapping, k_cache, v_cache, block_tables, seq_lens,
                     scale, *, out=None, cache_dtype=None, k_scale=None, v_scale=None,
                     err_flag=None, stream=None) -> torch.Tensor:
    """One decode step in one launch: writes each sequence's new token (key, value
    [num_seqs, num_kv_heads, head_dim] at slot_mapping [num_seqs]) into the cache and
    decodes over every cached token, the new one included."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    if key.dtype != q.dtype or value.dtype != q.dtype:
        raise ValueError("key and value must have q's dtype")
    rc = lib().pa_append_decode_v1(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(key), _ptr(value), _ptr(slot_mapping),
        _ptr(k_cache), _ptr(v_cache), cache_code(k_cache, cache_dtype), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        num_heads, num_kv_heads, head_dim, block_size, num_blocks, float(scale), _ptr(err_flag),
        _stream(stream))
    _check(rc, "pa_append_decode_v1")
    return out


def prefill(q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, *,
            max_query_len=None, out=None, err_flag=None, stream=None) -> torch.Tensor:
    """Causal multi-token query: rows [query_start[s], query_start[s+1]) of q are the last
    tokens of sequence s, already in the cache; returns out [total_q, H, D]."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    total_q, num_heads, _ = q.shape
    if max_query_len is None:
        max_query_len = int((query_start[1:] - query_start[:-1]).max()) if query_start.numel() > 1 else 0
    if out is None:
        out = torch.empty_like(q)
    rc = lib().pa_prefill(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(query_start), total_q, int(max_query_len),
        _ptr(k_cache), _ptr(v_cache), cache_code(k_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), seq_lens.shape[0], num_heads, num_kv_heads,
        head_dim, block_size, num_blocks, float(scale), _ptr(err_flag), _stream(stream))
    _check(rc, "pa_prefill")
    return out


def decode_cascade(q, k_cache, v_cache, block_tables, seq_lens, scale, prefix_len, *,
                   out=None, workspace=None, err_flag=None, stream=None) -> torch.Tensor:
    """pa_decode_v1 for sequences that share their first prefix_len tokens (the same
    blocks): the prefix on the tensor cores once per kv head, each sequence's own tokens
    on the persistent decode, the partials merged.  A caller-provided workspace must be
    zero-filled before its first use."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    need = lib().pa_decode_cascade_workspace_bytes(num_seqs, num_heads, head_dim)
    if workspace is None:       # zero-filled once; every complete call leaves it that way
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib().pa_decode_cascade(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(k_cache), _ptr(v_cache),
        cache_code(k_cache), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        num_heads, num_kv_heads, head_dim, block_size, num_blocks, float(scale), int(prefix_len),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err_flag),
        _stream(stream))
    _check(rc, "pa_decode_cascade")
    return out


def decode_v2_partition(q, k_cache, v_cache, block_tables, seq_lens, scale, partition_size,
                        tmp_out, max_logits, exp_sums, *, cache_dtype=None, k_scale=None,
                        v_scale=None, err_flag=None, stream=None) -> None:
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    max_parts = tmp_out.shape[2]
    rc = lib().pa_decode_v2_partition(
        _ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums), _ptr(q), _FLOAT_CODES[q.dtype],
        _ptr(k_cache), _ptr(v_cache), cache_code(k_cache, cache_dtype), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), num_seqs,
        num_heads, num_kv_heads, head_dim, block_size, num_blocks, float(scale),
        int(partition_size), max_parts, _ptr(err_flag), _stream(stream))
    _check(rc, "pa_decode_v2_partition")


def decode_v2_merge(out, tmp_out, max_logits, exp_sums, seq_lens, partition_size, *,
                    stream=None) -> None:
    num_seqs, num_heads, max_parts, head_dim = tmp_out.shape
    rc = lib().pa_decode_v2_merge(
        _ptr(out), _FLOAT_CODES[out.dtype], _ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums),
        _ptr(seq_lens), num_seqs, num_heads, head_dim, int(partition_size), max_parts,
        _stream(stream))
    _check(rc, "pa_decode_v2_merge")


class V2Workspace:
    """tmp_out / max_logits / exp_sums for pa_decode_v2_partition, allocated by torch."""

    def __init__(self, num_seqs, num_heads, head_dim, max_parts, device="cuda"):
        self.tmp_out = torch.empty((num_seqs, num_heads, max_parts, head_dim),
                                   dtype=torch.float32, device=device)
        self.max_logits = torch.empty((num_seqs, num_heads, max_parts), dtype=torch.float32,
                                      device=device)
        self.exp_sums = torch.empty_like(self.max_logits)
        self.max_parts = max_parts


def decode_v2(q, k_cache, v_cache, block_tables, seq_lens, scale, *, max_seq_len=None,
              partition_size=None, out=None, workspace: V2Workspace | None = None,
              cache_dtype=None, k_scale=None, v_scale=None, err_flag=None,
              stream=None) -> torch.Tensor:
    """Partition step then merge.  ``max_seq_len`` (if not given) is read from
    ``block_tables``' capacity, which never needs a device->host copy."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    if max_seq_len is None:
        max_seq_len = block_tables.shape[1] * block_size
    if partition_size is None:
        partition_size = choose_partition_size(max_seq_len, num_seqs, num_kv_heads,
                                               block_size=block_size)
    max_parts = max(1, -(-max_seq_len // partition_size))
    if workspace is None or workspace.max_parts < max_parts:
        workspace = V2Workspace(num_seqs, num_heads, head_dim, max_parts, q.device)
    if out is None:
        out = torch.empty_like(q)
    decode_v2_partition(q, k_cache, v_cache, block_tables, seq_lens, scale, partition_size,
                        workspace.tmp_out, workspace.max_logits, workspace.exp_sums,
                        cache_dtype=cache_dtype, k_scale=k_scale, v_scale=v_scale,
                        err_flag=err_flag, stream=stream)
    decode_v2_merge(out, workspace.tmp_out, workspace.max_logits, workspace.exp_sums, seq_lens,
                    partition_size, stream=stream)
    return out


class FusedWorkspace:
    """Workspace of pa_decode_fused (arrival counters + partial records), zeroed once;
    the kernel leaves the counters at zero after every complete call."""

    def __init__(self, num_seqs, num_kv_heads, head_dim, device="cuda"):
        dev = torch.device(device)
        sms = torch.cuda.get_device_properties(dev).multi_processor_count
        self.nbytes = int(lib().pa_decode_fused_workspace_bytes(num_seqs, num_kv_heads,
                                                               head_dim, sms))
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=dev)
        self.num_seqs, self.num_kv_heads, self.head_dim = num_seqs, num_kv_heads, head_dim

    def fits(self, num_seqs, num_kv_heads, head_dim) -> bool:
        return (num_seqs <= self.num_seqs and num_kv_heads == self.num_kv_heads
                and head_dim == self.head_dim)

    def counters(self) -> torch.Tensor:
        return self.buf[: self.num_seqs * self.num_kv_heads * 4].view(torch.int32)


def decode_fused(q, k_cache, v_cache, block_tables, seq_lens, scale, *, out=None,
                 workspace: FusedWorkspace | None = None, cache_dtype=None, k_scale=None,
                 v_scale=None, err_flag=None, stream=None) -> torch.Tensor:
    """Single-launch persistent decode (pa_decode_fused)."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    if workspace is None or not workspace.fits(num_seqs, num_kv_heads, head_dim):
        workspace = FusedWorkspace(num_seqs, num_kv_heads, head_dim, q.device)
    if out is None:
        out = torch.empty_like(q)
    rc = lib().pa_decode_fused(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(k_cache), _ptr(v_cache),
        cache_code(k_cache, cache_dtype), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, num_heads, num_kv_heads, head_dim,
        block_size, num_blocks, float(scale), _ptr(workspace.buf), workspace.nbytes,
        _ptr(err_flag), _stream(stream))
    _check(rc, "pa_decode_fused")
    return out


def decode_fused_noalloc(q, k_cache, v_cache, block_tables, seq_lens, scale, out, *,
                         cache_dtype=None, k_scale=None, v_scale=None, err_flag=None,
                         stream=None) -> torch.Tensor:
    """pa_decode_fused on the library's fixed scratch array: the caller passes only
    inputs and the output, nothing is allocated.  Calls must not overlap on the GPU."""
    num_blocks, block_size, num_kv_heads, head_dim = k_cache.shape
    num_seqs, num_heads, _ = q.shape
    rc = lib().pa_decode_fused_noalloc(
        _ptr(out), _ptr(q), _FLOAT_CODES[q.dtype], _ptr(k_cache), _ptr(v_cache),
        cache_code(k_cache, cache_dtype), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), num_seqs, num_heads, num_kv_heads, head_dim,
        block_size, num_blocks, float(scale), _ptr(err_flag), _stream(stream))
    _check(rc, "pa_decode_fused_noalloc")
    return out


def pick_decode_variant(num_seqs, num_kv_heads, max_seq_len, num_sms=None) -> str:
    """'v1' when one CTA per (sequence, kv head) already fills the GPU with short units
    (it needs no merge), else 'fused' (balances long or few sequences over every SM)."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    units = num_seqs * num_kv_heads
    tiles_per_unit = -(-int(max_seq_len) // 16)
    return "v1" if units >= num_sms and tiles_per_unit <= 256 else "fused"


def choose_partition_size(max_seq_len, num_seqs, num_kv_heads, num_sms=None, block_size=16) -> int:
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(lib().pa_choose_partition_size(int(max_seq_len), int(num_seqs), int(num_kv_heads),
                                              int(num_sms), int(block_size)))


def workspace_bytes(num_seqs, num_heads, head_dim, max_parts) -> int:
    return int(lib().pa_decode_v2_workspace_bytes(num_seqs, num_heads, head_dim, max_parts))


def kv_bytes_per_token(num_layers, num_kv_heads, head_dim, dtype_bytes) -> float:
    return float(lib().pa_kv_bytes_per_token(num_layers, num_kv_heads, head_dim, dtype_bytes))


def get_device_error(clear: bool = True) -> int:
    v = ctypes.c_int(0)
    _check(lib().pa_get_device_error(ctypes.byref(v), int(clear)), "pa_get_device_error")
    return v.value


def set_decode_config(warps: int = 0, stages: int = 0) -> None:
    _check(lib().pa_set_decode_config(int(warps), int(stages)), "pa_set_decode_config")


def set_prefetch_tiles(tiles_per_warp: int = -1) -> None:
    """L2 prefetch depth per decode warp before the PDL wait (PDL mode 2); -1 = default."""
    _check(lib().pa_set_prefetch_tiles(int(tiles_per_warp)), "pa_set_prefetch_tiles")


def set_wait_limit_ns(limit_ns: int = 0) -> None:
    """Per-wait time limit inside the decode kernels (0: the default, 2 s)."""
    _check(lib().pa_set_wait_limit_ns(int(limit_ns)), "pa_set_wait_limit_ns")


def set_cascade_config(prefix_splits: int = 0, suffix_form: int = 0) -> None:
    """pa_decode_cascade knobs: KV splits of the prefix launch (1..4; 0 = automatic
    placement; -1 = side by side with the suffix whenever it fits) and the suffix form
    (0 persistent decode + merge, 1 v1 decode merging in its epilogue)."""
    _check(lib().pa_set_cascade_config(int(prefix_splits), int(suffix_form)),
           "pa_set_cascade_config")


def set_pdl(mode: int = 1) -> None:
    """Programmatic dependent launch mode (0 off, 1 default, 2 early table reads)."""
    _check(lib().pa_set_pdl(int(mode)), "pa_set_pdl")


def set_fault_injection(mode: int = 0) -> None:
    """Test hook: mode 1 withholds each decode warp's first stage so its bounded
    wait runs out (reported as DEVERR_TIMEOUT), mode 3 each masked decode warp's last
    one, where it has more than two; 0 turns it off."""
    _check(lib().pa_set_fault_injection(int(mode)), "pa_set_fault_injection")
