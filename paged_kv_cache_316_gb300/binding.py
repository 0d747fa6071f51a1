"""Thin Python binding of libpagedkv.so (``include/pagedkv.h``).

Argument marshalling only: every function derives sizes and strides from
torch tensor shapes, passes device pointers and the current CUDA stream to
the C entry point of the same name, and raises on a non-zero status.  No
step of the computation happens here, and there is no CPU fallback: when the
library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

NHD, HND = 0, 1
F16, BF16, E4M3, F16_E4M3, BF16_E4M3 = 0, 1, 2, 3, 4

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libpagedkv.so"
_lib = None

_c_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_sz = ctypes.c_size_t

_SIGNATURES = {
    "pkv_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "pkv_kernel_launches": ([], ctypes.c_ulonglong),
    "pkv_debug_bounds": ([], ctypes.c_int),
    "pkv_set_wait_limit_ns": ([ctypes.c_ulonglong], ctypes.c_ulonglong),
    "paged_seq_lens": ([_c_p, _c_p, _i32, _i32, _c_p, _c_p], ctypes.c_int),
    "paged_batch_indices_positions": ([_c_p, _c_p, _i32, _i64, _c_p, _c_p, _c_p],
                                      ctypes.c_int),
    "paged_append": ([_c_p, _c_p, _i64, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _c_p,
                      _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32, _c_p, _c_p],
                     ctypes.c_int),
    "paged_decode_workspace_size": ([_i32] * 8, _sz),
    "paged_decode": ([_c_p, _c_p, _c_p, _i64, _i64, _c_p, _sz, _c_p, _i32, _c_p,
                      _i32, _i32, _f32, _f32, _i32, _c_p, _i32, _i32, _i32, _i32,
                      _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_decode_varlen": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _sz, _c_p, _i32, _c_p,
                             _i32, _i32, _f32, _f32, _i32, _c_p, _i32, _c_p, _i32, _i32, _i32,
                             _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_decode_ex": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _sz, _c_p, _i32, _c_p,
                         _i32, _i32, _f32, _f32, _c_p, _c_p, _i32, _c_p, _i32, _c_p, _i32, _i32,
                         _i32, _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_decode_noalloc": ([_c_p, _c_p, _c_p, _i64, _i64, _c_p, _i32, _c_p, _i32, _i32,
                              _f32, _f32, _i32, _c_p, _i32, _i32, _i32, _i32, _i32, _i32,
                              _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_append_scaled": ([_c_p, _c_p, _i64, _c_p, _c_p, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i64, _i32,
                             _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32, _c_p, _c_p], ctypes.c_int),
    "paged_decode_window_workspace_size": ([_i32] * 9, _sz),
    "paged_decode_window": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _c_p, _c_p, _i64, _i32, _c_p, _sz, _c_p, _i32,
                             _c_p, _i32, _i32, _f32, _f32, _c_p, _c_p, _i32, _i32, _c_p, _i32, _c_p, _i32, _i32,
                             _i32, _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_prefill_workspace_size": ([_i32] * 4, _sz),
    "paged_prefill": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _i64, _f32, _c_p, _sz, _i32,
                       _i32, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32,
                       _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_prefill_ex": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _i64, _f32, _c_p, _sz, _i32,
                          _i32, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32,
                          _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                          _c_p], ctypes.c_int),
    "paged_prefill_scaled_workspace_size": ([_i32] * 7, _sz),
    "paged_prefill_window": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _i64, _c_p, _c_p, _i64, _i32, _f32, _c_p, _sz,
                              _i32, _i32, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                              _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "paged_prefill_fp8_workspace_size": ([_i32] * 5 + [_i64] + [_i32] * 4, _sz),
    "paged_prefill_fp8": ([_c_p, _i64, _c_p, _c_p, _i64, _i64, _i64, _f32, _c_p, _c_p, _c_p, _c_p,
                           _sz, _i32, _i32, _c_p, _c_p, _c_p, _i32, _i32, _i32, _i32, _i32, _i32,
                           _i32, _i32, _i32, _i32, _i32, _i32, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
}


class PagedKVError(RuntimeError):
    pass


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library(path: str | None = None):
    """Load libpagedkv.so from the package directory (raises if missing).
    With `path`, load that build of the library instead and route every later
    call to it (e.g. the range-checking libpagedkv_debug.so; passing
    library_path() switches back)."""
    global _lib
    if _lib is None or path is not None:
        path = path or library_path()
        if not os.path.exists(path):
            raise PagedKVError(
                f"{path} is not built: run `python -m paged_kv_cache_316_gb300.build` "
                "(nvcc, sm_103a) first; there is no fallback implementation")
        lib = ctypes.CDLL(path)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def debug_bounds() -> bool:
    """True when the loaded library is the range-checking debug build."""
    return bool(load_library().pkv_debug_bounds())


def kernel_launches() -> int:
    return int(load_library().pkv_kernel_launches())


def set_wait_limit_ns(ns: int) -> int:
    """Limit of the bounded pipeline waits of later append / prefill
    launches (0: the default, one second); returns the previous limit."""
    return int(load_library().pkv_set_wait_limit_ns(int(ns)))


def _check(status: int):
    if status != 0:
        msg = load_library().pkv_status_string(status).decode()
        raise PagedKVError(f"libpagedkv status {status}: {msg}")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise PagedKVError("tensor arguments must live on a CUDA device")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (no Stream object per call)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise PagedKVError(f"unsupported element type {t.dtype}")
    return code


def _decode_dtype(query: torch.Tensor, cache: torch.Tensor) -> int:
    """Decode's dtype code: the query/output type, with an E4M3 cache when
    the cache holds 8-bit floats."""
    q = _dtype_code(query)
    if q not in (F16, BF16):
        raise PagedKVError(f"query must be fp16 or bf16, not {query.dtype}")
    if cache.dtype == torch.float8_e4m3fn:
        return F16_E4M3 if q == F16 else BF16_E4M3
    if cache.dtype != query.dtype:
        raise PagedKVError("the cache holds the query's type or e4m3")
    return q


def _layout_code(kv_layout) -> int:
    if kv_layout in (NHD, "NHD"):
        return NHD
    if kv_layout in (HND, "HND"):
        return HND
    raise PagedKVError(f"kv_layout must be NHD or HND, got {kv_layout!r}")


def _rows_contiguous(t) -> bool:
    """t[0].is_contiguous(), from the shape and strides."""
    if t.is_contiguous():
        return True
    n = 1
    shape, stride = t.shape, t.stride()
    if len(shape) == 4:  # (a view of K or V in a [pages, 2, ..] pool)
        a, b = shape[3], shape[2] * shape[3]
        if stride[3] == 1 and stride[2] == a and stride[1] == b:
            return True
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] != 1 and stride[i] != n:
            return t.numel() == 0
        n *= shape[i]
    return True


def split_cache(kv_cache, layout: int):
    """(k_ptr, v_ptr, page_stride, num_pages, num_heads, page_size, head_dim)
    for a 5-D [P, 2, ...] tensor or a (k, v) tuple of 4-D tensors."""
    if isinstance(kv_cache, (tuple, list)):
        base, v = kv_cache
        shape, stride = base.shape, base.stride(0)
        if v.shape != shape or v.stride(0) != stride:
            raise PagedKVError("K and V caches must have the same shape and page stride")
        if v.dtype != base.dtype or v.get_device() != base.get_device():
            raise PagedKVError("K and V caches hold the same type on the same device")
        if not (_rows_contiguous(base) and _rows_contiguous(v)):
            raise PagedKVError("each page must be contiguous")
        kp, vp = base.data_ptr(), v.data_ptr()
        P, H, S, D = shape
    else:
        base = kv_cache
        shape = base.shape
        if len(shape) != 5 or shape[1] != 2:
            raise PagedKVError("a single kv_cache tensor must be [pages, 2, ...]")
        if not _rows_contiguous(base):
            raise PagedKVError("each page must be contiguous")
        strides = base.stride()
        stride = strides[0]
        kp = base.data_ptr()
        vp = kp + strides[1] * base.element_size()
        P, _, H, S, D = shape
    if not base.is_cuda:
        raise PagedKVError("tensor arguments must live on a CUDA device")
    if layout != HND:
        H, S = S, H
    return kp, vp, stride, P, H, S, D, base


def base_dtype(kv_cache) -> torch.dtype:
    return (kv_cache[0] if isinstance(kv_cache, (tuple, list)) else kv_cache).dtype


def split_scales(kv_scales, num_pages: int, num_heads: int, page_size: int, device: int):
    """(k_ptr, v_ptr, page stride, block) of the block scales of an E4M3
    cache: one float32 tensor [pages, 2, heads, page_size // block] or a
    (k, v) tuple of [pages, heads, page_size // block]."""
    if isinstance(kv_scales, (tuple, list)):
        k, v = kv_scales
        shape, stride = k.shape, k.stride()
        if len(shape) != 3 or v.shape != shape or v.stride() != stride:
            raise PagedKVError("K and V scales must be [pages, heads, blocks] of the same shape and strides")
        same = v.dtype == torch.float32 and v.get_device() == k.get_device()
        vp = v.data_ptr()
    else:
        k = kv_scales
        shape, stride = k.shape, k.stride()
        if len(shape) != 4 or shape[1] != 2:
            raise PagedKVError("a single kv_scales tensor must be [pages, 2, heads, blocks]")
        vp = k.data_ptr() + 4 * stride[1]
        shape, stride, same = (shape[0], shape[2], shape[3]), (stride[0], stride[2], stride[3]), True
    P, H, blocks = shape
    if P != num_pages or H != num_heads or blocks < 1 or page_size % blocks:
        raise PagedKVError(f"scales must be [{num_pages}, {num_heads}, page_size // block] for each of K and V")
    if not same or k.dtype != torch.float32 or k.get_device() != device:
        raise PagedKVError("scales are float32 on the cache's device")
    if (blocks > 1 and stride[2] != 1) or (H > 1 and stride[1] != blocks):
        raise PagedKVError("the scales of a page must be contiguous")
    return k.data_ptr(), vp, stride[0] if P > 1 else max(H * blocks, stride[0]), page_size // blocks


def _same_device(*tensors):
    """All given tensors live on the current CUDA device: the library
    launches there.  Returns that device's index."""
    here = torch.cuda.current_device() if tensors[0].is_cuda else -2
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise PagedKVError("tensor arguments must live on the current CUDA device")
    return here


def _stream_on(stream, device: int) -> int:
    """_stream when the current device's index is known."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


_addr = torch.Tensor.data_ptr


# ---- index helpers ------------------------------------------------------------------

def paged_seq_lens(kv_indptr, kv_last_page_len, page_size: int, seq_lens=None,
                   stream=None):
    B = kv_last_page_len.shape[0]
    if seq_lens is None:
        seq_lens = torch.empty(B, dtype=torch.int32, device=kv_indptr.device)
    _check(load_library().paged_seq_lens(_ptr(kv_indptr), _ptr(kv_last_page_len), B,
                                         page_size, _ptr(seq_lens), _stream(stream)))
    return seq_lens


def paged_batch_indices_positions(append_indptr, seq_lens, nnz: int,
                                  batch_indices=None, positions=None, stream=None):
    B = seq_lens.shape[0]
    dev = append_indptr.device
    if batch_indices is None:
        batch_indices = torch.empty(nnz, dtype=torch.int32, device=dev)
    if positions is None:
        positions = torch.empty(nnz, dtype=torch.int32, device=dev)
    _check(load_library().paged_batch_indices_positions(
        _ptr(append_indptr), _ptr(seq_lens), B, nnz, _ptr(batch_indices),
        _ptr(positions), _stream(stream)))
    return batch_indices, positions


# ---- append -----------------------------------------------------------------------------

def paged_append(append_key, append_value, batch_indices, positions, paged_kv_cache,
                 kv_indices, kv_indptr, kv_last_page_len, kv_layout="NHD",
                 err_word=None, stream=None) -> None:
    layout = _layout_code(kv_layout)
    kp, vp, stride, P, H, S, D, _ = split_cache(paged_kv_cache, layout)
    nnz = append_key.shape[0]
    if not (append_key.is_contiguous() and append_value.is_contiguous()):
        raise PagedKVError("append_key/append_value must be contiguous")
    if append_value.shape != append_key.shape or tuple(append_key.shape[1:]) != (H, D):
        raise PagedKVError(f"append_key/append_value must both be [nnz, {H}, {D}]")
    if append_key.dtype != base_dtype(paged_kv_cache) or append_value.dtype != append_key.dtype:
        raise PagedKVError("append_key/append_value hold the cache's element type")
    for t in (batch_indices, positions):
        if t.dtype != torch.int32 or t.numel() < nnz:
            raise PagedKVError(f"batch_indices/positions must be int32 with >= {nnz} entries")
    _check(load_library().paged_append(
        _ptr(append_key), _ptr(append_value), nnz, _ptr(batch_indices),
        _ptr(positions), kp, vp, stride, P, _ptr(kv_indices), _ptr(kv_indptr),
        _ptr(kv_last_page_len), kv_last_page_len.shape[0], H, D, S, layout,
        _dtype_code(append_key), _ptr(err_word), _stream(stream)))


def paged_append_scaled(append_key, append_value, batch_indices, positions, paged_kv_cache, kv_scales,
                        kv_indices, kv_indptr, kv_last_page_len, kv_layout="NHD", err_word=None,
                        stream=None) -> None:
    """Append 16-bit tokens to an E4M3 cache with one power-of-two scale for
    each block of tokens and head.  kv_scales (float32, updated in place):
    [pages, 2, heads, page_size // block] or a (K, V) tuple of [pages, heads,
    page_size // block]; an element stands for its E4M3 value times its
    block's scale.  A block that gets tokens takes the larger of its scale
    (if it holds earlier tokens) and the smallest power of two under which the
    new values fit; earlier values of a block whose scale grew are rounded
    again.  The entries of one request and block have consecutive positions
    and follow one another, as paged_batch_indices_positions gives them."""
    layout = _layout_code(kv_layout)
    kp, vp, stride, P, H, S, D, base = split_cache(paged_kv_cache, layout)
    nnz = append_key.shape[0]
    if not (append_key.is_contiguous() and append_value.is_contiguous()):
        raise PagedKVError("append_key/append_value must be contiguous")
    if append_value.shape != append_key.shape or tuple(append_key.shape[1:]) != (H, D):
        raise PagedKVError(f"append_key/append_value must both be [nnz, {H}, {D}]")
    if base_dtype(paged_kv_cache) != torch.float8_e4m3fn:
        raise PagedKVError("the cache holds float8_e4m3fn")
    dtype = _dtype_code(append_key)
    if dtype not in (F16, BF16) or append_value.dtype != append_key.dtype:
        raise PagedKVError("append_key/append_value are both fp16 or both bf16")
    for t in (batch_indices, positions):
        if t.dtype != torch.int32 or t.numel() < nnz or not t.is_contiguous():
            raise PagedKVError(f"batch_indices/positions must be contiguous int32 with >= {nnz} entries")
    B = kv_last_page_len.shape[0]
    for t in (kv_indices, kv_indptr, kv_last_page_len):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise PagedKVError("kv_indices/kv_indptr/kv_last_page_len must be contiguous int32")
    if kv_indptr.numel() != B + 1:
        raise PagedKVError(f"kv_indptr must have {B + 1} entries")
    ks, vs, ss, block = split_scales(kv_scales, P, H, S, base.get_device())
    if ks == vs and P > 0:
        raise PagedKVError("K and V take scales of their own")
    device = _same_device(base, append_key, append_value, batch_indices, positions, kv_indices, kv_indptr,
                          kv_last_page_len, err_word)
    status = load_library().paged_append_scaled(
        _addr(append_key), _addr(append_value), nnz, _addr(batch_indices), _addr(positions), kp, vp, stride, P, ks, vs,
        ss, block, _addr(kv_indices), _addr(kv_indptr), _addr(kv_last_page_len), B, H, D, S, layout, dtype,
        None if err_word is None else _addr(err_word), _stream_on(stream, device))
    if status:
        _check(status)


# ---- decode -------------------------------------------------------------------------------

def _scale_arg(scale, device):
    """A host float -> (value, NULL); a one-element float32 tensor on the
    query's device -> (1.0, its address)."""
    if isinstance(scale, torch.Tensor):
        if scale.dtype != torch.float32 or scale.numel() != 1 or scale.device != device:
            raise PagedKVError("a tensor scale is one float32 value on the query's device")
        return 1.0, _ptr(scale)
    return float(scale), None


def paged_decode_workspace_size(batch_size, q_len_per_req, num_qo_heads, num_kv_heads,
                                head_dim, max_seq_len, page_size, window_left=-1, first_tokens=None) -> int:
    """Workspace of paged_decode; with first_tokens given (0 too), of one with
    first_tokens or kv_scales."""
    if first_tokens is not None:
        return int(load_library().paged_decode_window_workspace_size(
            batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim,
            max_seq_len, page_size, window_left, first_tokens))
    return int(load_library().paged_decode_workspace_size(
        batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim,
        max_seq_len, page_size, window_left))


def _check_decode_args(query, out, lse, block_tables, seq_lens, rows_needed: int):
    """The C ABI of the uniform decode takes no row count: the shapes it
    trusts are checked here, so that no kernel reads or writes past the end
    of query, out or lse."""
    rows, Hqo, _ = query.shape
    if not query.is_contiguous():
        raise PagedKVError("query must be contiguous [rows, num_qo_heads, head_dim]")
    if rows < rows_needed:
        raise PagedKVError(f"query has {rows} rows; the requests need {rows_needed}")
    if out.shape != query.shape or out.dtype != query.dtype or not out.is_contiguous():
        raise PagedKVError("out must be a contiguous tensor of the query's shape and dtype")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (rows, Hqo)
                            or not lse.is_contiguous()):
        raise PagedKVError(f"lse must be a contiguous float32 [{rows}, {Hqo}] tensor")
    B = seq_lens.shape[0]
    if seq_lens.dim() != 1 or seq_lens.element_size() != 4:
        raise PagedKVError("seq_lens must be a 1-D tensor of 32-bit lengths")
    if block_tables.dim() != 2 or block_tables.shape[0] < B or block_tables.dtype != torch.int32 \
            or block_tables.stride(1) != 1:
        raise PagedKVError("block_tables must be int32 [>= batch_size, pages] with unit column stride")


def paged_decode(query, kv_cache, workspace, block_tables, seq_lens, max_seq_len: int,
                 bmm1_scale: float = 1.0, bmm2_scale: float = 1.0, window_left: int = -1,
                 sinks=None, kv_layout="HND", q_len_per_req: int = 1, out=None,
                 lse=None, err_word=None, stream=None, max_q_len=None, cum_seq_lens_q=None,
                 enable_pdl=None, first_tokens: int = 0, kv_scales=None):
    """seq_lens: int32 (or uint32) tensor holding the unsigned kv lengths.
    With cum_seq_lens_q ([B+1] int32 on the device) and max_q_len, request b
    has the query rows cum[b] .. cum[b+1]-1 (variable-length queries) and
    q_len_per_req is ignored.  bmm1_scale / bmm2_scale may be one-element
    float32 device tensors, read when the kernels run; enable_pdl launches
    the call's first kernel as a programmatic dependent of the stream's
    previous kernel (None / False: an ordinary launch).  first_tokens: keys
    at the start of each request that stay visible under window_left; the
    pages between them and the window are not read.  kv_scales: block scales
    of a float8_e4m3fn cache (see paged_append_scaled); each element stands
    for its value times its block's scale."""
    if first_tokens or kv_scales is not None:
        return _decode_window(query, kv_cache, workspace, block_tables, seq_lens, max_seq_len, bmm1_scale, bmm2_scale,
                              window_left, sinks, kv_layout, q_len_per_req, out, lse, err_word, stream, max_q_len,
                              cum_seq_lens_q, enable_pdl, first_tokens, kv_scales)
    layout = _layout_code(kv_layout)
    kp, vp, stride, P, Hkv, S, D, base = split_cache(kv_cache, layout)
    rows, Hqo, Dq = query.shape
    if Dq != D:
        raise PagedKVError("query head_dim differs from the cache's")
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(query)
    if (cum_seq_lens_q is None) != (max_q_len is None):
        raise PagedKVError("cum_seq_lens_q and max_q_len go together")
    if cum_seq_lens_q is not None:
        if cum_seq_lens_q.dtype != torch.int32 or tuple(cum_seq_lens_q.shape) != (B + 1,):
            raise PagedKVError(f"cum_seq_lens_q must be int32 [{B + 1}]")
        _check_decode_args(query, out, lse, block_tables, seq_lens, 0)
    else:
        _check_decode_args(query, out, lse, block_tables, seq_lens, B * q_len_per_req)
    s1, s1_dev = _scale_arg(bmm1_scale, query.device)
    s2, s2_dev = _scale_arg(bmm2_scale, query.device)
    if s1_dev or s2_dev or enable_pdl:
        mq = int(max_q_len) if cum_seq_lens_q is not None else q_len_per_req
        _check(load_library().paged_decode_ex(
            _ptr(query), rows, kp, vp, stride, P, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(block_tables),
            block_tables.stride(0), _ptr(seq_lens), B, max_seq_len, s1, s2, s1_dev, s2_dev,
            window_left, _ptr(sinks), mq, _ptr(cum_seq_lens_q), Hqo, Hkv, D, S, layout,
            _decode_dtype(query, base), 1 if enable_pdl else 0, _ptr(out), _ptr(lse),
            _ptr(err_word), _stream(stream)))
        return out
    if cum_seq_lens_q is not None:
        _check(load_library().paged_decode_varlen(
            _ptr(query), rows, kp, vp, stride, P, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(block_tables),
            block_tables.stride(0), _ptr(seq_lens), B, max_seq_len, bmm1_scale,
            bmm2_scale, window_left, _ptr(sinks), int(max_q_len), _ptr(cum_seq_lens_q), Hqo,
            Hkv, D, S, layout, _decode_dtype(query, base), _ptr(out), _ptr(lse), _ptr(err_word),
            _stream(stream)))
        return out
    _check(load_library().paged_decode(
        _ptr(query), kp, vp, stride, P, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(block_tables),
        block_tables.stride(0), _ptr(seq_lens), B, max_seq_len, bmm1_scale,
        bmm2_scale, window_left, _ptr(sinks), q_len_per_req, Hqo, Hkv, D, S,
        layout, _decode_dtype(query, base), _ptr(out), _ptr(lse), _ptr(err_word),
        _stream(stream)))
    return out


def _decode_window(query, kv_cache, workspace, block_tables, seq_lens, max_seq_len, bmm1_scale, bmm2_scale, window_left,
                   sinks, kv_layout, q_len_per_req, out, lse, err_word, stream, max_q_len, cum_seq_lens_q, enable_pdl,
                   first_tokens, kv_scales):
    """paged_decode under a window with first tokens and / or over a cache with
    block scales."""
    layout = _layout_code(kv_layout)
    kp, vp, stride, P, Hkv, S, D, base = split_cache(kv_cache, layout)
    shape = query.shape
    rows, Hqo, Dq = shape
    if Dq != D:
        raise PagedKVError("query head_dim differs from the cache's")
    if seq_lens.dim() != 1 or seq_lens.element_size() != 4 or not seq_lens.is_contiguous():
        raise PagedKVError("seq_lens must be a contiguous 1-D tensor of 32-bit lengths")
    B = seq_lens.shape[0]
    dtype = _decode_dtype(query, base)
    ks = vs = cum = sink_ptr = lse_ptr = err_ptr = None
    ss = block = 0
    if kv_scales is not None:
        if dtype not in (F16_E4M3, BF16_E4M3):
            raise PagedKVError("kv_scales belong to a float8_e4m3fn cache")
        ks, vs, ss, block = split_scales(kv_scales, P, Hkv, S, base.get_device())
    if (cum_seq_lens_q is None) != (max_q_len is None):
        raise PagedKVError("cum_seq_lens_q and max_q_len go together")
    if cum_seq_lens_q is None:
        max_q = q_len_per_req
        if rows < B * max_q:
            raise PagedKVError(f"query has {rows} rows; the requests need {B * max_q}")
    else:
        max_q = int(max_q_len)
        if cum_seq_lens_q.dtype != torch.int32 or tuple(cum_seq_lens_q.shape) != (B + 1,) \
                or not cum_seq_lens_q.is_contiguous():
            raise PagedKVError(f"cum_seq_lens_q must be contiguous int32 [{B + 1}]")
        cum = _ptr(cum_seq_lens_q)
    if not query.is_contiguous():
        raise PagedKVError("query must be contiguous [rows, num_qo_heads, head_dim]")
    if out is None:
        out = torch.empty_like(query)
    elif out.shape != shape or out.dtype != query.dtype or not out.is_contiguous():
        raise PagedKVError("out must be a contiguous tensor of the query's shape and dtype")
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != shape[:2] or not lse.is_contiguous():
            raise PagedKVError(f"lse must be a contiguous float32 [{rows}, {Hqo}] tensor")
        lse_ptr = _addr(lse)
    bt_shape, bt_stride = block_tables.shape, block_tables.stride()
    if len(bt_shape) != 2 or bt_stride[1] != 1 or block_tables.dtype != torch.int32 or bt_shape[0] < B:
        raise PagedKVError("block_tables must be int32 [>= batch_size, pages] with unit column stride")
    if bt_shape[1] * S < max_seq_len:  # (a view's row stride may be wider than its columns)
        raise PagedKVError("block_tables has fewer columns than max_seq_len needs")
    if sinks is not None:
        if sinks.dtype != torch.float32 or sinks.numel() != Hqo or not sinks.is_contiguous():
            raise PagedKVError(f"sinks must be contiguous float32 [{Hqo}]")
        sink_ptr = _addr(sinks)
    s1, s2, s1_dev, s2_dev = bmm1_scale, bmm2_scale, None, None
    if type(s1) is not float:
        s1, s1_dev = _scale_arg(s1, query.device)
    if type(s2) is not float:
        s2, s2_dev = _scale_arg(s2, query.device)
    if err_word is not None:
        err_ptr = _ptr(err_word)
    device = _same_device(query, base, workspace, block_tables, seq_lens, cum_seq_lens_q, sinks, out, lse, err_word)
    status = load_library().paged_decode_window(
        _addr(query), rows, kp, vp, stride, P, ks, vs, ss, block, _addr(workspace), workspace.nbytes,
        _addr(block_tables), bt_stride[0], _addr(seq_lens), B, max_seq_len, s1, s2, s1_dev, s2_dev, window_left,
        first_tokens, sink_ptr, max_q, cum, Hqo, Hkv, D, S, layout, dtype, 1 if enable_pdl else 0, _addr(out), lse_ptr,
        err_ptr, _stream_on(stream, device))
    if status:
        _check(status)
    return out


def paged_decode_noalloc(query, kv_cache, block_tables, seq_lens, max_seq_len: int,
                         bmm1_scale: float = 1.0, bmm2_scale: float = 1.0,
                         window_left: int = -1, sinks=None, kv_layout="HND",
                         q_len_per_req: int = 1, out=None, lse=None, err_word=None,
                         stream=None):
    """paged_decode for callers that cannot allocate device memory at the
    call: the split partials use the library's fixed device scratch array
    (PKV_NOALLOC_SCRATCH_BYTES) instead of a workspace tensor.  Calls that
    overlap on the GPU share that array and race."""
    layout = _layout_code(kv_layout)
    kp, vp, stride, P, Hkv, S, D, base = split_cache(kv_cache, layout)
    rows, Hqo, Dq = query.shape
    if Dq != D:
        raise PagedKVError("query head_dim differs from the cache's")
    B = seq_lens.shape[0]
    if out is None:
        out = torch.empty_like(query)
    _check_decode_args(query, out, lse, block_tables, seq_lens, B * q_len_per_req)
    _check(load_library().paged_decode_noalloc(
        _ptr(query), kp, vp, stride, P, _ptr(block_tables), block_tables.stride(0),
        _ptr(seq_lens), B, max_seq_len, bmm1_scale, bmm2_scale, window_left, _ptr(sinks),
        q_len_per_req, Hqo, Hkv, D, S, layout, _decode_dtype(query, base), _ptr(out), _ptr(lse),
        _ptr(err_word), _stream(stream)))
    return out


# ---- prefill ---------------------------------------------------------------------------------

def paged_prefill_workspace_size(batch_size, num_qo_heads, max_token_per_sequence,
                                 max_sequence_kv) -> int:
    return int(load_library().paged_prefill_workspace_size(
        batch_size, num_qo_heads, max_token_per_sequence, max_sequence_kv))


def paged_prefill_fp8_workspace_size(batch_size, num_qo_heads, num_kv_heads,
                                     max_token_per_sequence, max_sequence_kv, total_q, d_qk, d_vo,
                                     q_dtype, kv_dtype) -> int:
    """Workspace of paged_prefill with an E4M3 query and/or caches (dtypes
    as torch dtypes)."""
    return int(load_library().paged_prefill_fp8_workspace_size(
        batch_size, num_qo_heads, num_kv_heads, max_token_per_sequence, max_sequence_kv, total_q,
        d_qk, d_vo, E4M3 if q_dtype == torch.float8_e4m3fn else BF16,
        E4M3 if kv_dtype == torch.float8_e4m3fn else BF16))


def paged_prefill_scaled_workspace_size(batch_size, num_qo_heads, num_kv_heads, max_token_per_sequence,
                                        max_sequence_kv, d_qk, d_vo) -> int:
    """Workspace of paged_prefill over E4M3 caches with block scales (kv_scales)."""
    return int(load_library().paged_prefill_scaled_workspace_size(
        batch_size, num_qo_heads, num_kv_heads, max_token_per_sequence, max_sequence_kv, d_qk, d_vo))


def _scale_ptr(t, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != 1 or t.device != device:
        raise PagedKVError("q_scale / k_scale / v_scale: one float32 value on the query's device")
    return _ptr(t)


def paged_prefill(q, k_cache, v_cache, scale: float, workspace,
                  max_token_per_sequence: int, max_sequence_kv: int,
                  actual_seq_lens_q, actual_seq_lens_kv, block_tables,
                  causal: bool = True, out=None, lse=None, kv_layout="HND",
                  err_word=None, stream=None, batch_offsets_q=None, batch_offsets_o=None,
                  batch_offsets_k=None, batch_offsets_v=None, q_scale=None, k_scale=None,
                  v_scale=None, o_data_type=None, window_left: int = -1, first_tokens: int = 0,
                  kv_scales=None):
    """block_tables=None: k_cache / v_cache are contiguous [rows, Hkv, d]
    tensors (the page's non-paged case; kv_layout is then NHD).  The
    batch_offsets_* tensors ([B] int32 on the device, token rows) place each
    request's queries, outputs / LSEs and (contiguous K/V) keys / values.
    q and/or the (paged) caches may be float8_e4m3fn: q_scale, k_scale and
    v_scale (one float32 each on the device, or None for 1) dequantise them,
    and the output is o_data_type (bf16 when q is E4M3 and none is given);
    the workspace then needs paged_prefill_fp8_workspace_size bytes.
    window_left, first_tokens: the query at position p sees key j if also
    j >= p - window_left or j < first_tokens (-1: no window); the pages between
    a request's first tokens and its first query's window are not read.
    kv_scales: block scales of float8_e4m3fn caches under a 16-bit query (see
    paged_append_scaled); the workspace then needs
    paged_prefill_scaled_workspace_size bytes."""
    if block_tables is None:
        kv_layout = "NHD"
    layout = _layout_code(kv_layout)
    total_q, Hqo, d_qk = q.shape
    if block_tables is None:
        P, Hkv, dk = k_cache.shape
        S, dv = 1, v_cache.shape[2]
    elif layout == HND:
        P, Hkv, S, dk = k_cache.shape
        dv = v_cache.shape[3]
    else:
        P, S, Hkv, dk = k_cache.shape
        dv = v_cache.shape[3]
    if dk != d_qk:
        raise PagedKVError("q head_dim differs from the key cache's")
    e4 = torch.float8_e4m3fn
    if kv_scales is not None or window_left != -1 or first_tokens:
        return _prefill_window(q, k_cache, v_cache, scale, workspace, max_token_per_sequence, max_sequence_kv,
                               actual_seq_lens_q, actual_seq_lens_kv, block_tables, causal, out, lse, layout,
                               (P, Hkv, S, dv), err_word, stream,
                               (batch_offsets_q, batch_offsets_o, batch_offsets_k, batch_offsets_v),
                               (q_scale, k_scale, v_scale), o_data_type, window_left, first_tokens, kv_scales)
    fp8 = q.dtype == e4 or k_cache.dtype == e4 or any(x is not None for x in (q_scale, k_scale, v_scale))
    odt = o_data_type or (torch.bfloat16 if q.dtype == e4 else q.dtype)
    if out is None:
        out = torch.empty((total_q, Hqo, dv), dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty((total_q, Hqo), dtype=torch.float32, device=q.device)
    if tuple(out.shape) != (total_q, Hqo, dv) or out.dtype != odt or not out.is_contiguous():
        raise PagedKVError(f"out must be a contiguous {odt} [{total_q}, {Hqo}, {dv}] tensor")
    if tuple(lse.shape) != (total_q, Hqo) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise PagedKVError(f"lse must be a contiguous float32 [{total_q}, {Hqo}] tensor")
    if not q.is_contiguous():
        raise PagedKVError("q must be contiguous [total_q, num_qo_heads, d_qk]")
    B = actual_seq_lens_q.shape[0]
    bt_stride = 0 if block_tables is None else block_tables.stride(0)
    offsets = (batch_offsets_q, batch_offsets_o, batch_offsets_k, batch_offsets_v)
    if fp8:
        if block_tables is None or any(o is not None for o in offsets):
            raise PagedKVError("the E4M3 prefill takes paged caches and packed rows")
        if v_cache.dtype != k_cache.dtype:
            raise PagedKVError("k_cache and v_cache hold the same element type")
        _check(load_library().paged_prefill_fp8(
            _ptr(q), total_q, _ptr(k_cache), _ptr(v_cache), k_cache.stride(0), v_cache.stride(0),
            P, scale, _scale_ptr(q_scale, q.device), _scale_ptr(k_scale, q.device),
            _scale_ptr(v_scale, q.device), _ptr(workspace), workspace.numel() * workspace.element_size(),
            max_token_per_sequence, max_sequence_kv, _ptr(actual_seq_lens_q),
            _ptr(actual_seq_lens_kv), _ptr(block_tables), bt_stride, B, int(causal), Hqo, Hkv, d_qk,
            dv, S, layout, _dtype_code(q), _dtype_code(k_cache), _dtype_code(out), _ptr(out),
            _ptr(lse), _ptr(err_word), _stream(stream)))
    elif all(o is None for o in offsets):
        _check(load_library().paged_prefill(
            _ptr(q), total_q, _ptr(k_cache), _ptr(v_cache), k_cache.stride(0), v_cache.stride(0),
            P, scale, _ptr(workspace), workspace.numel() * workspace.element_size(),
            max_token_per_sequence, max_sequence_kv, _ptr(actual_seq_lens_q),
            _ptr(actual_seq_lens_kv), _ptr(block_tables), bt_stride, B,
            int(causal), Hqo, Hkv, d_qk, dv, S, layout, _dtype_code(q), _ptr(out),
            _ptr(lse), _ptr(err_word), _stream(stream)))
    else:
        _check(load_library().paged_prefill_ex(
            _ptr(q), total_q, _ptr(k_cache), _ptr(v_cache), k_cache.stride(0), v_cache.stride(0),
            P, scale, _ptr(workspace), workspace.numel() * workspace.element_size(),
            max_token_per_sequence, max_sequence_kv, _ptr(actual_seq_lens_q),
            _ptr(actual_seq_lens_kv), _ptr(block_tables), bt_stride, B,
            int(causal), Hqo, Hkv, d_qk, dv, S, layout, _dtype_code(q), _ptr(out),
            _ptr(lse), *(_ptr(o) for o in offsets), _ptr(err_word), _stream(stream)))
    return out, lse


def _prefill_window(q, k_cache, v_cache, scale, workspace, max_q, max_kv, lens_q, lens_kv, block_tables, causal, out,
                    lse, layout, dims, err_word, stream, offsets, scalar_scales, o_data_type, window_left, first_tokens,
                    kv_scales):
    """paged_prefill under a window and / or over caches with block scales."""
    P, Hkv, S, dv = dims
    total_q, Hqo, d_qk = q.shape
    qdt = q.dtype
    dtype = _dtype_code(q)
    sq, sk, sv = scalar_scales
    if dtype > BF16 or sq is not None or sk is not None or sv is not None or (o_data_type is not None and
                                                                              o_data_type != qdt):
        raise PagedKVError("window_left, first_tokens and kv_scales take a 16-bit query and output and no "
                           "q_scale / k_scale / v_scale")
    if not q.is_contiguous():
        raise PagedKVError("q must be contiguous [total_q, num_qo_heads, d_qk]")
    ks = vs = None
    ss = block = 0
    kdt = k_cache.dtype
    if kv_scales is not None:
        if kdt != torch.float8_e4m3fn or block_tables is None:
            raise PagedKVError("kv_scales belong to paged float8_e4m3fn caches")
        ks, vs, ss, block = split_scales(kv_scales, P, Hkv, S, k_cache.get_device())
        dtype = F16_E4M3 if dtype == F16 else BF16_E4M3
    elif kdt != qdt:
        raise PagedKVError("the caches hold the query's type, or float8_e4m3fn with kv_scales")
    if v_cache.dtype != kdt or v_cache.shape[:-1] != k_cache.shape[:-1]:
        raise PagedKVError("K and V caches must have the same type, pages, heads and page size")
    if not (_rows_contiguous(k_cache) and _rows_contiguous(v_cache)):
        raise PagedKVError("each page must be contiguous")
    if out is None:
        out = torch.empty((total_q, Hqo, dv), dtype=qdt, device=q.device)
    elif tuple(out.shape) != (total_q, Hqo, dv) or out.dtype != qdt or not out.is_contiguous():
        raise PagedKVError(f"out must be a contiguous {qdt} [{total_q}, {Hqo}, {dv}] tensor")
    if lse is None:
        lse = torch.empty((total_q, Hqo), dtype=torch.float32, device=q.device)
    elif tuple(lse.shape) != (total_q, Hqo) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise PagedKVError(f"lse must be a contiguous float32 [{total_q}, {Hqo}] tensor")
    B = lens_q.shape[0]
    off_ptrs = (None, None, None, None)
    lens = (lens_q, lens_kv)
    oq, oo, ok, ov = offsets
    if oq is not None or oo is not None or ok is not None or ov is not None:
        lens += tuple(o for o in offsets if o is not None)
        off_ptrs = tuple(_ptr(o) for o in offsets)
    for t in lens:
        if t.dtype != torch.int32 or t.dim() != 1 or t.numel() != B or not t.is_contiguous():
            raise PagedKVError(f"lengths and batch offsets must be contiguous int32 [{B}]")
    bt_ptr, bt_stride = None, 0
    if block_tables is not None:
        bt = block_tables.stride()
        if len(bt) != 2 or bt[1] != 1 or block_tables.shape[0] < B or block_tables.dtype != torch.int32:
            raise PagedKVError("block_tables must be int32 [>= batch_size, pages] with unit column stride")
        if block_tables.shape[1] * S < max_kv:  # (a view's row stride may be wider than its columns)
            raise PagedKVError("block_tables has fewer columns than max_sequence_kv needs")
        bt_ptr, bt_stride = _addr(block_tables), bt[0]
    device = _same_device(q, k_cache, v_cache, workspace, block_tables, out, lse, err_word, *lens)
    status = load_library().paged_prefill_window(
        _addr(q), total_q, _addr(k_cache), _addr(v_cache), k_cache.stride(0), v_cache.stride(0), P, ks, vs, ss, block,
        scale, _addr(workspace), workspace.nbytes, max_q, max_kv, _addr(lens_q), _addr(lens_kv), bt_ptr, bt_stride, B,
        1 if causal else 0, window_left, first_tokens, Hqo, Hkv, d_qk, dv, S, layout, dtype, _addr(out), _addr(lse),
        *off_ptrs, None if err_word is None else _addr(err_word), _stream_on(stream, device))
    if status:
        _check(status)
    return out, lse
