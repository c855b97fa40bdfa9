"""Python binding of ``libpa.so``: the C-ABI calls of ``include/pa.h`` with the
same names, taking torch CUDA tensors.

Argument marshalling only: shapes and dtypes are read off the tensors into a
``pa_dims`` struct, pointers come from ``data_ptr()``, the stream from
``torch.cuda.current_stream()`` unless one is given.  Every operation runs in
the library's CUDA kernels; there is no fallback.  Importing this module
loads the library and raises :class:`LibraryMissing` if it is not built.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK = 0
STATUS = {0: "PA_OK", -1: "PA_ERR_NULL", -2: "PA_ERR_DTYPE", -3: "PA_ERR_SHAPE", -4: "PA_ERR_UNSUPPORTED",
          -5: "PA_ERR_WORKSPACE", -6: "PA_ERR_CUDA", -7: "PA_ERR_ALIGN", -8: "PA_ERR_MEMORY"}
PA_F16, PA_BF16, PA_FP8_E4M3, PA_INT4 = 0, 1, 2, 3
DEVERR = {1: "BLOCK_ID", 2: "CONTEXT", 4: "SLOT", 8: "COPY_PAIR", 16: "TIMEOUT", 32: "LAYOUT"}
# torch dtypes accepted for an FP8 E4M3 cache (the codes as bytes, or torch's own e4m3fn type)
FP8_CACHE_DTYPES = (torch.uint8, torch.float8_e4m3fn)

# The C entry points declared in include/pa.h, in declaration order.
EXPORTS = ["pa_decode_workspace_size", "pa_decode_num_partitions", "pa_decode", "pa_decode_noalloc",
           "pa_decode_fp8", "pa_reshape_and_cache_fp8", "pa_decode_ext_workspace_size", "pa_decode_ext",
           "pa_decode_int4", "pa_reshape_and_cache_int4", "pa_gather_cache", "pa_rope_frequencies", "pa_rope",
           "pa_rope_and_cache",
           "pa_prefix_cache_create", "pa_prefix_cache_destroy", "pa_prefix_cache_match", "pa_prefix_cache_insert",
           "pa_prefix_cache_release", "pa_prefix_cache_evict", "pa_prefix_cache_stats", "pa_prefix_order",
           "pa_reshape_and_cache", "pa_copy_blocks", "pa_swap_blocks", "pa_check_wait_timeout", "pa_last_error",
           "pa_device_error", "pa_version"]


class LibraryMissing(RuntimeError):
    pass


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class pa_dims(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


class pa_decode_opts(ctypes.Structure):
    _fields_ = [("q_len", ctypes.c_int32), ("window", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("seq_order", ctypes.c_void_p)]


class pa_rope_opts(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("magnitude", ctypes.c_double)]


class pa_rope_config(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise LibraryMissing(f"{path} is not built; run `python -m paged_kv_cache_424_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    dp = ctypes.POINTER(pa_dims)
    lib.pa_decode_workspace_size.argtypes = [dp, i32, i32]
    lib.pa_decode_workspace_size.restype = u64
    lib.pa_decode_num_partitions.argtypes = [dp, i32, i32]
    lib.pa_decode_num_partitions.restype = i32
    lib.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, dp, i32, i32, vp, u64, vp]
    lib.pa_decode.restype = ctypes.c_int
    lib.pa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, dp, i32, i32, vp]
    lib.pa_decode_noalloc.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.pa_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, f32, f32, f32, i32, dp, i32, i32, vp, u64, vp]
    lib.pa_decode_fp8.restype = ctypes.c_int
    lib.pa_reshape_and_cache_fp8.argtypes = [vp, vp, vp, vp, vp, i32, dp, f32, f32, vp]
    lib.pa_reshape_and_cache_fp8.restype = ctypes.c_int
    op = ctypes.POINTER(pa_decode_opts)
    lib.pa_decode_ext_workspace_size.argtypes = [dp, op, i32, i32]
    lib.pa_decode_ext_workspace_size.restype = u64
    lib.pa_decode_ext.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, dp, op, i32, i32, vp, u64, vp]
    lib.pa_decode_ext.restype = ctypes.c_int
    rp = ctypes.POINTER(pa_rope_opts)
    f64p = ctypes.POINTER(ctypes.c_double)
    lib.pa_decode_int4.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, dp, i32, i32, vp, u64, vp]
    lib.pa_decode_int4.restype = ctypes.c_int
    lib.pa_reshape_and_cache_int4.argtypes = [vp, vp, vp, vp, vp, i32, dp, vp]
    lib.pa_reshape_and_cache_int4.restype = ctypes.c_int
    lib.pa_gather_cache.argtypes = [vp, vp, vp, vp, vp, i32, dp, f32, f32, vp]
    lib.pa_gather_cache.restype = ctypes.c_int
    lib.pa_rope_frequencies.argtypes = [ctypes.POINTER(pa_rope_config), f64p, f64p]
    lib.pa_rope_frequencies.restype = ctypes.c_int
    lib.pa_rope.argtypes = [vp, vp, vp, vp, vp, i32, dp, rp, i64, i64, vp]
    lib.pa_rope.restype = ctypes.c_int
    lib.pa_rope_and_cache.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, dp, rp, i64, i64, i64, f32, f32, vp]
    lib.pa_rope_and_cache.restype = ctypes.c_int
    ip = ctypes.POINTER(ctypes.c_int32)
    lp = ctypes.POINTER(ctypes.c_int64)
    lib.pa_prefix_cache_create.argtypes = [i64]
    lib.pa_prefix_cache_create.restype = vp
    lib.pa_prefix_cache_destroy.argtypes = [vp]
    lib.pa_prefix_cache_destroy.restype = None
    lib.pa_prefix_cache_match.argtypes = [vp, ip, i32, ip, i32]
    lib.pa_prefix_cache_match.restype = i32
    lib.pa_prefix_cache_insert.argtypes = [vp, ip, i32, ip, i32]
    lib.pa_prefix_cache_insert.restype = ctypes.c_int
    lib.pa_prefix_cache_release.argtypes = [vp, ip, i32]
    lib.pa_prefix_cache_release.restype = i32
    lib.pa_prefix_cache_evict.argtypes = [vp, i32, ip]
    lib.pa_prefix_cache_evict.restype = i32
    lib.pa_prefix_cache_stats.argtypes = [vp, lp, lp, lp, lp]
    lib.pa_prefix_cache_stats.restype = ctypes.c_int
    lib.pa_prefix_order.argtypes = [ip, ip, i32, i32, ip]
    lib.pa_prefix_order.restype = ctypes.c_int
    lib.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i32, dp, vp]
    lib.pa_reshape_and_cache.restype = ctypes.c_int
    lib.pa_copy_blocks.argtypes = [vp, vp, i32, vp, i32, dp, vp]
    lib.pa_copy_blocks.restype = ctypes.c_int
    lib.pa_swap_blocks.argtypes = [vp, vp, i64, vp, vp, i64, vp, i32, dp, vp]
    lib.pa_swap_blocks.restype = ctypes.c_int
    lib.pa_last_error.argtypes = []
    lib.pa_last_error.restype = ctypes.c_char_p
    lib.pa_check_wait_timeout.argtypes = [i32, vp]
    lib.pa_check_wait_timeout.restype = ctypes.c_int
    lib.pa_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.pa_device_error.restype = ctypes.c_int
    lib.pa_version.argtypes = []
    lib.pa_version.restype = i32
    return lib


LIB = _load()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return PA_F16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (3 us of a 13 us call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int) -> None:
    if status != PA_OK:
        raise PagedAttentionError(status, LIB.pa_last_error().decode(errors="replace"))


def _need_cuda(*ts: Optional[torch.Tensor]) -> None:
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def int4_cache_shape(num_blocks: int, num_kv_heads: int, head_dim: int) -> tuple:
    """Shape of a 4-bit K or V pool (a uint8 tensor): per (block, KV head) the
    16 rows' codes and then their (scale, low) pairs."""
    return (num_blocks, num_kv_heads, 8 * head_dim + 64)


def _is_int4(cache: torch.Tensor) -> bool:
    return cache.dim() == 3 and cache.dtype == torch.uint8


def _on_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    """All on one CUDA device, the current one (whose streams the calls use)."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            dev = -1
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device")


def _dense(*ts: Optional[torch.Tensor]) -> None:
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("outputs, caches and index tensors must be contiguous")


@functools.lru_cache(maxsize=512)
def _dims_ref(*fields: int):
    """A pa_dims by reference; the calls only read it."""
    return ctypes.byref(pa_dims(*fields))


def _kv_code(cache: torch.Tensor) -> int:
    if _is_int4(cache):
        return PA_INT4
    return PA_FP8_E4M3 if cache.dtype in FP8_CACHE_DTYPES else _dtype_code(cache)


def make_dims(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
              max_blocks_per_seq: int, num_blocks: int, dtype: int, kv_dtype: int = 0) -> pa_dims:
    return pa_dims(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, dtype,
                   kv_dtype)


def _pool_shape(cache: torch.Tensor) -> tuple:
    """(blocks, KV heads, block size, head_dim) of a pool."""
    if _is_int4(cache):
        NB, Hk, nbytes = cache.shape
        if nbytes < 72 or (nbytes - 64) % 8:
            raise ValueError("a 4-bit pool is uint8 [num_blocks, num_kv_heads, 8 * head_dim + 64]")
        return NB, Hk, 16, (nbytes - 64) // 8
    return tuple(cache.shape)


def dims_of(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor) -> pa_dims:
    S, H, D = q.shape
    NB, Hk, B, D2 = _pool_shape(k_cache)
    if D2 != D:
        raise ValueError("q and k_cache disagree on head_dim")
    MB = block_tables.shape[1] if block_tables.dim() == 2 else 0
    return make_dims(S, H, Hk, D, B, MB, NB, _dtype_code(q), _kv_code(k_cache))


def cache_dims(k_cache: torch.Tensor, dtype: Optional[torch.dtype] = None) -> pa_dims:
    """Block geometry of a cache; `dtype` is the 16-bit type of the tokens
    written into it (taken from the cache itself unless it is FP8 or 4-bit)."""
    NB, Hk, B, D = _pool_shape(k_cache)
    kv = _kv_code(k_cache)
    if dtype is not None:
        code = _dtype_code(torch.empty(0, dtype=dtype))
    else:
        code = PA_F16 if kv in (PA_FP8_E4M3, PA_INT4) else kv
    return make_dims(0, Hk, Hk, D, B, 0, NB, code, kv)


# ---------------------------------------------------------------------------
# the C-ABI calls
# ---------------------------------------------------------------------------
def pa_version() -> int:
    return int(LIB.pa_version())


def pa_last_error() -> str:
    return LIB.pa_last_error().decode(errors="replace")


def pa_decode_workspace_size(dims: pa_dims, max_context_len: int, partition_tokens: int = 0) -> int:
    n = LIB.pa_decode_workspace_size(ctypes.byref(dims), int(max_context_len), int(partition_tokens))
    if n == ctypes.c_size_t(-1).value:
        raise PagedAttentionError(-3, pa_last_error())
    return int(n)


def pa_decode_num_partitions(dims: pa_dims, max_context_len: int, partition_tokens: int = 0) -> int:
    n = int(LIB.pa_decode_num_partitions(ctypes.byref(dims), int(max_context_len), int(partition_tokens)))
    if n < 0:
        raise PagedAttentionError(n, pa_last_error())
    return n


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, num_kv_heads: int,
              max_context_len: int, partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """out[s, h] = softmax(scale * q[s, h] . K_s^T) V_s over the paged cache."""
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    dims = dims_of(q, k_cache, block_tables)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = LIB.pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
                       float(scale), int(num_kv_heads), ctypes.byref(dims), int(max_context_len),
                       int(partition_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st)
    return out


def pa_decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, num_kv_heads: int,
                      max_context_len: int, partition_tokens: int = 0, stream=None) -> torch.Tensor:
    """pa_decode without a workspace argument: the split-KV scratch is the
    library's own 64 MiB device array, for callers that cannot allocate.
    Calls that overlap on the GPU race on that shared scratch."""
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    dims = dims_of(q, k_cache, block_tables)
    st = LIB.pa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), float(scale), int(num_kv_heads), ctypes.byref(dims),
                               int(max_context_len), int(partition_tokens), _stream(stream))
    _check(st)
    return out


def pa_decode_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, k_scale: float,
                  v_scale: float, num_kv_heads: int, max_context_len: int, partition_tokens: int = 0,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_decode over FP8 E4M3 caches (uint8 or float8_e4m3fn tensors):
    K = code * k_scale, V = code * v_scale."""
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if k_cache.dtype not in FP8_CACHE_DTYPES or v_cache.dtype not in FP8_CACHE_DTYPES:
        raise TypeError("FP8 caches must be uint8 or float8_e4m3fn tensors")
    dims = dims_of(q, k_cache, block_tables)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = LIB.pa_decode_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
                           float(scale), float(k_scale), float(v_scale), int(num_kv_heads), ctypes.byref(dims),
                           int(max_context_len), int(partition_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st)
    return out


def _int4_arguments(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, context_lens: torch.Tensor) -> None:
    """What has to go together in an attention call over a 4-bit cache."""
    if out.shape != q.shape or out.dtype != q.dtype or v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or \
            block_tables.dim() != 2 or block_tables.shape[0] != q.shape[0] or context_lens.numel() != q.shape[0]:
        raise ValueError("out must be as q, v_cache as k_cache, block_tables [num_seqs, blocks], context_lens [num_seqs]")


def pa_decode_int4(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, num_kv_heads: int,
                   max_context_len: int, partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """pa_decode over 4-bit caches (uint8 tensors of int4_cache_shape): an
    element is code * scale + low of its row."""
    if not _is_int4(k_cache) or not _is_int4(v_cache):
        raise TypeError("4-bit caches must be uint8 tensors of int4_cache_shape")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    S, H, D = q.shape
    NB, Hk, nbytes = k_cache.shape
    if nbytes != 8 * D + 64:
        raise ValueError("q and k_cache disagree on head_dim")
    _int4_arguments(out, q, k_cache, v_cache, block_tables, context_lens)
    _on_device(q, out, k_cache, v_cache, block_tables, context_lens, workspace)
    _dense(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    dims = _dims_ref(S, H, Hk, D, 16, block_tables.shape[1], NB, _dtype_code(q), PA_INT4)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = LIB.pa_decode_int4(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                            block_tables.data_ptr(), context_lens.data_ptr(), scale, num_kv_heads, dims,
                            max_context_len, partition_tokens, _ptr(workspace), ws_bytes, _stream(stream))
    if st != PA_OK:
        _check(st)
    return out


def pa_decode_ext_workspace_size(dims: pa_dims, opts: pa_decode_opts, max_context_len: int,
                                 partition_tokens: int = 0) -> int:
    n = LIB.pa_decode_ext_workspace_size(ctypes.byref(dims), ctypes.byref(opts), int(max_context_len),
                                         int(partition_tokens))
    if n == ctypes.c_size_t(-1).value:
        raise PagedAttentionError(-3, pa_last_error())
    return int(n)


def ext_dims(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor) -> pa_dims:
    """dims of a [S, q_len, H, D] query batch."""
    S, QL, H, D = q.shape
    return dims_of(q.view(S, QL * H, D)[:, :H], k_cache, block_tables)


def pa_decode_ext(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, num_kv_heads: int,
                  max_context_len: int, q_len: int = 1, window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                  partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                  seq_order: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Multi-token / sliding-window decode: q and out are [S, q_len, H, D];
    query i of sequence s sits at position context_lens[s] - q_len + i and
    attends to its `window` most recent positions (all when 0).  The caches
    may be 16-bit, FP8 E4M3 (uint8 / float8_e4m3fn) or 4-bit."""
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if q.dim() != 4 or q.shape[1] != q_len or tuple(out.shape) != tuple(q.shape):
        raise ValueError("q and out must be [num_seqs, q_len, num_heads, head_dim]")
    if _is_int4(k_cache):
        _int4_arguments(out, q, k_cache, v_cache, block_tables, context_lens)
    dims = ext_dims(q, k_cache, block_tables)
    if seq_order is not None:
        _need_cuda(seq_order)
        if seq_order.dtype != torch.int32 or seq_order.numel() != q.shape[0]:
            raise TypeError("seq_order must be int32 [num_seqs]")
    opts = pa_decode_opts(int(q_len), int(window), float(k_scale), float(v_scale),
                          None if seq_order is None else seq_order.data_ptr())
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = LIB.pa_decode_ext(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
                           float(scale), int(num_kv_heads), ctypes.byref(dims), ctypes.byref(opts),
                           int(max_context_len), int(partition_tokens), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st)
    return out


# ---------------------------------------------------------------------------
# prefix caching (host)
# ---------------------------------------------------------------------------
def _i32p(a):
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


class PrefixCache:
    """The library's host prefix cache (pa_prefix_cache_*): token ids of
    full 16-token blocks -> the physical blocks holding their K/V."""

    def __init__(self, num_blocks: int):
        self._h = LIB.pa_prefix_cache_create(int(num_blocks))
        if not self._h:
            raise PagedAttentionError(-3, pa_last_error())

    def close(self) -> None:
        if self._h:
            LIB.pa_prefix_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def match(self, tokens) -> list:
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        out = np.zeros(max(1, t.size // 16), dtype=np.int32)
        n = LIB.pa_prefix_cache_match(self._h, _i32p(t), int(t.size), _i32p(out), int(t.size // 16))
        if n < 0:
            raise PagedAttentionError(n, pa_last_error())
        return out[:n].tolist()

    def insert(self, tokens, blocks) -> None:
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        b = np.ascontiguousarray(blocks, dtype=np.int32)
        _check(LIB.pa_prefix_cache_insert(self._h, _i32p(t), int(t.size), _i32p(b), int(b.size)))

    def release(self, blocks) -> int:
        import numpy as np
        b = np.ascontiguousarray(blocks, dtype=np.int32)
        n = LIB.pa_prefix_cache_release(self._h, _i32p(b), int(b.size))
        if n < 0:
            raise PagedAttentionError(n, pa_last_error())
        return int(n)

    def evict(self, max_blocks: int) -> list:
        import numpy as np
        out = np.zeros(max(1, max_blocks), dtype=np.int32)
        n = LIB.pa_prefix_cache_evict(self._h, int(max_blocks), _i32p(out))
        if n < 0:
            raise PagedAttentionError(n, pa_last_error())
        return out[:n].tolist()

    def stats(self) -> dict:
        v = [ctypes.c_int64(0) for _ in range(4)]
        _check(LIB.pa_prefix_cache_stats(self._h, *[ctypes.byref(x) for x in v]))
        return dict(zip(("cached", "evictable", "hits", "lookups"), (x.value for x in v)))


def pa_prefix_order(block_tables, context_lens):
    """Host: the shared-prefix-aware order of the batch (numpy int32 [S])."""
    import numpy as np
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    cl = np.ascontiguousarray(context_lens, dtype=np.int32)
    S = cl.shape[0]
    MB = bt.shape[1] if bt.ndim == 2 else 0
    order = np.zeros(max(1, S), dtype=np.int32)
    _check(LIB.pa_prefix_order(_i32p(bt), _i32p(cl), int(S), int(MB), _i32p(order)))
    return order[:S]


def pa_reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                             slot_mapping: torch.Tensor, k_scale: float, v_scale: float, stream=None) -> None:
    """k_cache[slot // 16, :, slot % 16] = e4m3(key[t] / k_scale) (and V) for slot >= 0."""
    _need_cuda(key, value, k_cache, v_cache, slot_mapping)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if k_cache.dtype not in FP8_CACHE_DTYPES or v_cache.dtype not in FP8_CACHE_DTYPES:
        raise TypeError("FP8 caches must be uint8 or float8_e4m3fn tensors")
    dims = cache_dims(k_cache, key.dtype)
    st = LIB.pa_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                      int(slot_mapping.numel()), ctypes.byref(dims), float(k_scale), float(v_scale),
                                      _stream(stream))
    _check(st)


def pa_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         slot_mapping: torch.Tensor, stream=None) -> None:
    """k_cache[slot // 16, :, slot % 16] = key[t] (and V) for slot >= 0."""
    _need_cuda(key, value, k_cache, v_cache, slot_mapping)
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    dims = cache_dims(k_cache)
    st = LIB.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                  int(slot_mapping.numel()), ctypes.byref(dims), _stream(stream))
    _check(st)


def _rows_dims(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               slots: torch.Tensor, num_heads: int):
    """dims (by reference) of [tokens, KV heads, head_dim] rows that go with
    `slots` and a pair of pools, after checking that they do."""
    NB, Hk, B, D = _pool_shape(k_cache)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must have one shape and dtype")
    if slots.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    shape = (slots.numel(), Hk, D)
    if key.shape != shape or value.shape != shape:
        raise ValueError(f"key and value must be {list(shape)}, got {list(key.shape)} and {list(value.shape)}")
    kv = _kv_code(k_cache)
    if value.dtype != key.dtype or (kv < PA_FP8_E4M3 and k_cache.dtype != key.dtype):
        raise TypeError("key, value and a 16-bit cache must have one dtype")
    return _dims_ref(0, num_heads, Hk, D, B, 0, NB, _dtype_code(key), kv)


def pa_reshape_and_cache_int4(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              slot_mapping: torch.Tensor, stream=None) -> None:
    """The 4-bit row of slot_mapping[t] = the codes, scale and low of key[t] (and value[t]) for slot >= 0."""
    if not _is_int4(k_cache):
        raise TypeError("4-bit caches must be uint8 tensors of int4_cache_shape")
    dims = _rows_dims(key, value, k_cache, v_cache, slot_mapping, 0)
    _on_device(key, value, k_cache, v_cache, slot_mapping)
    _dense(key, value, k_cache, v_cache, slot_mapping)
    st = LIB.pa_reshape_and_cache_int4(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                       slot_mapping.data_ptr(), key.shape[0], dims, _stream(stream))
    if st != PA_OK:
        _check(st)


def pa_gather_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    slot_mapping: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """key[t] (and value[t]) = the cached row of slot_mapping[t] in key's 16-bit
    dtype, for slot >= 0; other rows stay as they are."""
    dims = _rows_dims(key, value, k_cache, v_cache, slot_mapping, 0)
    _on_device(key, value, k_cache, v_cache, slot_mapping)
    _dense(key, value, k_cache, v_cache, slot_mapping)
    st = LIB.pa_gather_cache(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             slot_mapping.data_ptr(), key.shape[0], dims, k_scale, v_scale, _stream(stream))
    if st != PA_OK:
        _check(st)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def pa_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                        original_context: float = 0.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                        beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, magnitude) of a rotation of the first `rotary_dim` dims: a
    float64 CPU tensor [rotary_dim / 2] (copy it to the device once) and a
    float, both for pa_rope and pa_rope_and_cache.  `scaling` is one of
    ROPE_SCALING: "plain", "linear", "ntk", "bands" or "yarn"."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling {scaling!r}: one of {sorted(ROPE_SCALING)}")
    cfg = pa_rope_config(int(rotary_dim), ROPE_SCALING[scaling], float(base), float(factor), float(original_context),
                         float(low_freq_factor), float(high_freq_factor), float(beta_fast), float(beta_slow))
    inv_freq = torch.zeros(max(1, int(rotary_dim) // 2), dtype=torch.float64)
    magnitude = ctypes.c_double(1.0)
    _check(LIB.pa_rope_frequencies(ctypes.byref(cfg),
                                   ctypes.cast(inv_freq.data_ptr(), ctypes.POINTER(ctypes.c_double)),
                                   ctypes.byref(magnitude)))
    return inv_freq, magnitude.value


def _token_stride(t: torch.Tensor, what: str) -> int:
    """Elements between the tokens of a [tokens, heads, head_dim] tensor whose
    heads are contiguous (a view of a fused projection may have gaps between tokens)."""
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if sd != 1 or (sh != D and H > 1):
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with contiguous heads")
    return st if T > 1 else H * D


def _rope_opts(inv_freq: torch.Tensor, positions: torch.Tensor, tokens: int, interleaved: bool, inverse: bool,
               magnitude: float):
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise TypeError("inv_freq must be float64 [rotary_dim / 2] (pa_rope_frequencies)")
    if positions.dtype != torch.int64 or positions.numel() != tokens:
        raise TypeError("positions must be int64, one per token")
    return ctypes.byref(pa_rope_opts(inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0,
                                     1 if inverse else 0, magnitude))


def _same(a: Optional[torch.Tensor], b: Optional[torch.Tensor], what: str) -> None:
    if a is None or b is None:
        if a is not b:
            raise ValueError(f"{what} and its output go together")
    elif a.shape != b.shape or a.dtype != b.dtype:
        raise ValueError(f"{what} and its output must have one shape and dtype")


def pa_rope(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], k_out: Optional[torch.Tensor],
            k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
            magnitude: float = 1.0, inverse: bool = False, stream=None) -> None:
    """q_out = rotate(q), k_out = rotate(k) for [tokens, heads, head_dim]
    queries and keys (either pair may be None).  Inputs may be views with a
    gap between tokens; outputs are contiguous, or the contiguous input
    itself.  `inverse` turns back: the gradient of the rotation."""
    _same(q, q_out, "q")
    _same(k, k_out, "k")
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    _on_device(x, q, q_out, k, k_out, positions, inv_freq)
    _dense(q_out, k_out, positions, inv_freq)
    T, H, D = x.shape
    if q is not None and k is not None and (k.shape[0] != T or k.shape[2] != D or q.dtype != k.dtype):
        raise ValueError("q and k must have the same tokens, head_dim and dtype")
    opts = _rope_opts(inv_freq, positions, T, interleaved, inverse, magnitude)
    dims = _dims_ref(0, 0 if q is None else H, 0 if k is None else k.shape[1], D, 16, 0, 1, _dtype_code(x), 0)
    st = LIB.pa_rope(_ptr(q_out), _ptr(q), _ptr(k_out), _ptr(k), positions.data_ptr(), T, dims, opts,
                     0 if q is None else _token_stride(q, "q"), 0 if k is None else _token_stride(k, "k"),
                     _stream(stream))
    if st != PA_OK:
        _check(st)


def pa_rope_and_cache(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor], key: torch.Tensor,
                      value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
                      magnitude: float = 1.0, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """q_out = rotate(q); the cache rows of slot_mapping[t] = rotate(key[t])
    and value[t] in the pools' type (16-bit, FP8 E4M3 or 4-bit).  Tokens with a
    negative slot are left out entirely.  q, key and value may be views of a
    fused projection; q may be None."""
    _same(q, q_out, "q")
    T, _, D = key.shape
    if q is not None and (q.shape[0] != T or q.shape[2] != D or q.dtype != key.dtype):
        raise ValueError("q and key must have the same tokens, head_dim and dtype")
    dims = _rows_dims(key, value, k_cache, v_cache, slot_mapping, 0 if q is None else q.shape[1])
    _on_device(key, q, q_out, value, k_cache, v_cache, slot_mapping, positions, inv_freq)
    _dense(q_out, k_cache, v_cache, slot_mapping, positions, inv_freq)
    opts = _rope_opts(inv_freq, positions, T, interleaved, False, magnitude)
    st = LIB.pa_rope_and_cache(_ptr(q_out), _ptr(q), key.data_ptr(), value.data_ptr(), k_cache.data_ptr(),
                               v_cache.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), T, dims, opts,
                               0 if q is None else _token_stride(q, "q"), _token_stride(key, "key"),
                               _token_stride(value, "value"), k_scale, v_scale, _stream(stream))
    if st != PA_OK:
        _check(st)


def pa_copy_blocks(k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor],
                   block_mapping: torch.Tensor, stream=None) -> None:
    """Per layer: block dst of K and V becomes a copy of block src."""
    if len(k_caches) != len(v_caches) or not k_caches:
        raise ValueError("need matching, non-empty lists of K and V caches")
    _need_cuda(*k_caches, *v_caches, block_mapping)
    if block_mapping.dtype != torch.int64:
        raise TypeError("block_mapping must be int64")
    L = len(k_caches)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_caches])
    vp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_caches])
    dims = cache_dims(k_caches[0])
    pairs = block_mapping.numel() // 2
    st = LIB.pa_copy_blocks(ctypes.cast(kp, ctypes.c_void_p), ctypes.cast(vp, ctypes.c_void_p), L,
                            _ptr(block_mapping), int(pairs), ctypes.byref(dims), _stream(stream))
    _check(st)


def pa_swap_blocks(src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor, dst_v: torch.Tensor,
                   block_mapping: torch.Tensor, stream=None) -> None:
    """Block dst of the destination pools becomes a copy of block src of the
    source pools; each pool a CUDA tensor or a pinned CPU tensor."""
    for t in (src_k, src_v, dst_k, dst_v, block_mapping):
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools and mapping must be contiguous CUDA tensors or pinned CPU tensors")
    if block_mapping.dtype != torch.int64:
        raise TypeError("block_mapping must be int64")
    if src_k.shape[1:] != dst_k.shape[1:] or src_v.shape != src_k.shape or dst_v.shape != dst_k.shape:
        raise ValueError("pools disagree on the block shape")
    dims = cache_dims(src_k)
    st = LIB.pa_swap_blocks(_ptr(src_k), _ptr(src_v), int(src_k.shape[0]), _ptr(dst_k), _ptr(dst_v),
                            int(dst_k.shape[0]), _ptr(block_mapping), int(block_mapping.numel() // 2),
                            ctypes.byref(dims), _stream(stream))
    _check(st)


def pa_check_wait_timeout(milliseconds: int = 50, stream=None) -> None:
    """Enqueue the bounded-wait diagnostic (a wait that can never complete
    gives up after about `milliseconds` and flags PA_DEVERR_TIMEOUT)."""
    _check(LIB.pa_check_wait_timeout(int(milliseconds), _stream(stream)))


def pa_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    w = ctypes.c_uint32(0)
    _check(LIB.pa_device_error(_stream(stream), ctypes.byref(w)))
    return int(w.value)
