"""Python binding of libpa.so, the GB300 paged KV-cache library.

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels (or, for the block pool, its C++ host code).  Names follow the
C ABI in include/pa.h.  Tensors are torch tensors; PyTorch provides device
memory and streams.  If libpa.so is missing this module raises on import:
there is no fallback path.

Cache layout (one layer): a contiguous tensor [2, num_blocks, block_size,
num_kv_heads, head_size] of bf16 or fp32, index 0 = keys, 1 = values; or a
4-bit pool, a contiguous uint8 tensor [num_blocks, num_kv_heads,
block_size / 8, 9 * head_size] (alloc_fp4_cache) for the pa_*_fp4 calls and
the block copies; or an 8-bit pool, a contiguous int8 tensor [num_blocks,
num_kv_heads, block_size / 8, 16 * (head_size + 1)] (alloc_int8_cache) for the
pa_*_int8 calls and the block copies.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_CUDA = 3
PA_ERR_OUT_OF_BLOCKS = 4
PA_ERR_BAD_STATE = 5
PA_ERR_DEVICE_CHECK = 6
PA_ERR_TIMEOUT = 7
PA_BF16 = 0
PA_FP32 = 1
PA_FP4 = 2
PA_INT8 = 3
PA_KERNEL_AUTO = 0
PA_KERNEL_SIMT = 1
PA_KERNEL_TENSOR = 2
PA_DEVERR_SLOT = 0x1
PA_DEVERR_BLOCK_ID = 0x2
PA_DEVERR_SEQ_LEN = 0x4
PA_DEVERR_TIMEOUT = 0x8
PA_DEVERR_BLOCKS = 0x10
PA_DEVERR_POSITION = 0x20
PA_PARTITION_BALANCED = -2

# Every function include/pa.h declares.
EXPORTS = (
    "pa_reshape_and_cache", "pa_copy_blocks", "pa_decode", "pa_decode_ex", "pa_decode_no_alloc",
    "pa_decode_partition_size", "pa_decode_select_kernel",
    "pa_decode_workspace_size", "pa_slot_mapping", "pa_pool_create", "pa_pool_destroy",
    "pa_pool_add_seq", "pa_pool_fork", "pa_pool_append_token", "pa_pool_append_tokens",
    "pa_pool_free_seq", "pa_pool_block_table", "pa_pool_fill_tables", "pa_pool_slot",
    "pa_pool_ref_count", "pa_pool_num_free", "pa_get_device_error", "pa_status_string",
    "pa_version", "pa_set_decode_trace", "pa_pool_add_seq_tokens", "pa_pool_append_token_id",
    "pa_pool_is_cached", "pa_pool_free_queue", "pa_pool_reset_prefix_cache", "pa_pool_usage",
    "pa_swap_blocks", "pa_pool_set_cpu_blocks", "pa_pool_swap_out", "pa_pool_swap_in",
    "pa_pool_is_swapped", "pa_pool_num_free_cpu", "pa_decode_append", "pa_copy_bytes",
    "pa_set_decode_wait_limit", "pa_decode_shared_plan", "pa_decode_shared_workspace_size",
    "pa_decode_shared", "pa_reshape_and_cache_fp4", "pa_gather_cache_fp4", "pa_decode_fp4",
    "pa_decode_fp4_workspace_size", "pa_extend_tables", "pa_reshape_and_cache_int8",
    "pa_gather_cache_int8", "pa_decode_int8", "pa_decode_int8_workspace_size", "pa_evict_blocks",
    "pa_norm_rope",
)


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, _status_string(status), status))


class OutOfBlocks(PAError):
    pass


class SharedPlanInfo(ctypes.Structure):
    _fields_ = [("num_chunks", ctypes.c_int32), ("num_members", ctypes.c_int32),
                ("min_shared_tokens", ctypes.c_int32), ("min_chunk_stages", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("plan_ints", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("query_out", "key_out", "query", "key")]
                + [(n, ctypes.c_int64) for n in ("query_out_stride", "key_out_stride", "query_stride",
                                                 "key_stride")]
                + [(n, ctypes.c_void_p) for n in ("query_weight", "key_weight", "cos_sin", "positions",
                                                  "position_offsets")]
                + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_int32) for n in ("dtype", "num_tokens", "num_heads", "num_kv_heads",
                                                 "head_size", "rotary_dim", "max_position",
                                                 "interleaved")])


# The same, packed at once (attributes of a Structure, one by one, take 3 us a call).
_norm_rope_bytes = struct.Struct("@4P4q5Pf8i4x").pack
assert struct.calcsize("@4P4q5Pf8i4x") == ctypes.sizeof(NormRopeArgs)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError("libpa.so is not built (%s); run python paged_kv_cache_78_gb300/_build.py"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    sz = ctypes.c_size_t
    desc = ctypes.POINTER(CacheDesc)
    p_i32, p_i64, p_sz = ctypes.POINTER(i32), ctypes.POINTER(i64), ctypes.POINTER(sz)
    sig = {
        "pa_reshape_and_cache": [vp, desc, vp, vp, vp, i32, vp],
        "pa_copy_blocks": [vp, desc, vp, i32, vp],
        "pa_decode": [vp, vp, vp, desc, vp, i32, vp, i32, i32, f32, i32, i32, vp, sz, vp],
        "pa_decode_ex": [vp, vp, vp, desc, vp, i32, vp, i32, i32, f32, i32, i32, vp, sz, i32, vp],
        "pa_decode_no_alloc": [vp, vp, vp, desc, vp, i32, vp, i32, i32, f32, i32, i32, vp],
        "pa_decode_append": [vp, vp, vp, desc, vp, i32, vp, i32, i32, f32, i32, i32, vp, vp, vp,
                             sz, i32, vp],
        "pa_decode_partition_size": [desc, i32, i32, i32, i32, p_i32],
        "pa_decode_select_kernel": [desc, i32, i32, vp, i32, p_i32],
        "pa_decode_workspace_size": [desc, i32, i32, i32, i32, p_sz],
        "pa_slot_mapping": [vp, i32, i32, i32, i32, vp, vp, i32, vp],
        "pa_pool_create": [i32, i32, vp, ctypes.POINTER(vp)],
        "pa_pool_add_seq": [vp, i64, p_i64],
        "pa_pool_fork": [vp, i64, p_i64],
        "pa_pool_append_token": [vp, i64, p_i64, vp],
        "pa_pool_append_tokens": [vp, vp, i32, vp, vp, p_i32],
        "pa_pool_free_seq": [vp, i64],
        "pa_pool_block_table": [vp, i64, vp, i32, p_i32, p_i64],
        "pa_pool_fill_tables": [vp, vp, i32, vp, i32, vp],
        "pa_pool_slot": [vp, i64, i64, p_i64],
        "pa_pool_ref_count": [vp, i32, p_i32],
        "pa_get_device_error": [ctypes.POINTER(ctypes.c_uint32), vp],
        "pa_set_decode_trace": [vp, sz, i32],
        "pa_set_decode_wait_limit": [i64],
        "pa_decode_shared_plan": [vp, i32, vp, i32, i32, i32, i32, i32, vp, sz,
                                  ctypes.POINTER(SharedPlanInfo)],
        "pa_decode_shared_workspace_size": [desc, i32, i32, i32, ctypes.POINTER(SharedPlanInfo),
                                            p_sz],
        "pa_decode_shared": [vp, vp, vp, desc, vp, i32, vp, i32, i32, f32, i32, vp,
                             ctypes.POINTER(SharedPlanInfo), vp, vp, vp, sz, vp],
        "pa_reshape_and_cache_fp4": [vp, desc, vp, vp, i32, i64, i64, vp, i32, f32, f32, vp],
        "pa_gather_cache_fp4": [vp, vp, i32, vp, desc, vp, i32, f32, f32, vp],
        "pa_decode_fp4_workspace_size": [desc, i32, p_sz],
        "pa_decode_fp4": [vp, vp, i32, i64, vp, desc, f32, f32, vp, i32, vp, i32, i32, f32, vp, sz,
                          vp],
        "pa_extend_tables": [vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32,
                             vp],
        "pa_reshape_and_cache_int8": [vp, desc, vp, vp, i32, i64, i64, vp, i32, vp],
        "pa_gather_cache_int8": [vp, vp, i32, vp, desc, vp, i32, vp],
        "pa_decode_int8_workspace_size": [desc, i32, i32, i32, p_sz],
        "pa_decode_int8": [vp, vp, i32, i64, vp, desc, vp, i32, vp, i32, i32, f32, vp, vp, f32, vp, sz,
                           vp],
        "pa_evict_blocks": [vp, vp, i32, vp, i32, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp,
                            vp, vp],
        "pa_norm_rope": [vp, vp],  # a NormRopeArgs, or its bytes
        "pa_pool_add_seq_tokens": [vp, vp, i64, p_i64, p_i64],
        "pa_pool_append_token_id": [vp, i64, i32, p_i64, vp],
        "pa_pool_is_cached": [vp, i32, p_i32],
        "pa_pool_free_queue": [vp, vp, i32, p_i32],
        "pa_pool_reset_prefix_cache": [vp],
        "pa_pool_usage": [vp, p_i64, p_i64],
        "pa_swap_blocks": [vp, desc, vp, desc, vp, i32, vp],
        "pa_copy_bytes": [vp, vp, sz, vp],
        "pa_pool_set_cpu_blocks": [vp, i32],
        "pa_pool_swap_out": [vp, vp, i32, vp, p_i32],
        "pa_pool_swap_in": [vp, vp, i32, vp, p_i32],
        "pa_pool_is_swapped": [vp, i64, p_i32],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.pa_pool_destroy.argtypes = [vp]
    lib.pa_pool_destroy.restype = None
    lib.pa_pool_num_free.argtypes = [vp]
    lib.pa_pool_num_free.restype = i32
    lib.pa_status_string.argtypes = [ctypes.c_int]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_version.argtypes = []
    lib.pa_version.restype = ctypes.c_char_p
    return lib


lib = _load()


def _status_string(status: int) -> str:
    return lib.pa_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status == PA_OK:
        return
    if status == PA_ERR_OUT_OF_BLOCKS:
        raise OutOfBlocks(status, where)
    raise PAError(status, where)


def version() -> str:
    return lib.pa_version().decode()


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.float32:
        return PA_FP32
    raise TypeError("tensors must be bfloat16 or float32, got %s" % t.dtype)


def cache_desc(cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a [2, num_blocks, block_size, num_kv_heads, head_size] pool."""
    if cache.dim() != 5 or cache.shape[0] != 2:
        raise ValueError("cache must be [2, num_blocks, block_size, num_kv_heads, head_size]")
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    _, nb, bs, hkv, d = cache.shape
    return CacheDesc(nb, bs, hkv, d, _dtype_code(cache))


@functools.lru_cache(maxsize=64)
def _fp4_geometry(shape):
    """(descriptor, a reference to it, KV heads, head size) of a 4-bit pool's shape."""
    if len(shape) != 4 or shape[3] % 9:
        raise ValueError("a 4-bit cache must be [num_blocks, num_kv_heads, block_size / 8, "
                         "9 * head_size]")
    nb, hkv, tiles, size = shape
    desc = CacheDesc(nb, 8 * tiles, hkv, size // 9, PA_FP4)
    return desc, ctypes.byref(desc), hkv, size // 9


def _fp4_pool(cache: torch.Tensor):
    if cache.dtype is not torch.uint8:
        raise TypeError("a 4-bit cache must be uint8, got %s" % cache.dtype)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return _fp4_geometry(cache.shape)


def fp4_cache_desc(cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a 4-bit pool [num_blocks, num_kv_heads, block_size / 8, 9 * head_size]."""
    d = _fp4_pool(cache)[0]
    return CacheDesc(d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype)


def alloc_fp4_cache(num_blocks: int, block_size: int, num_kv_heads: int, head_size: int,
                    device="cuda") -> torch.Tensor:
    """A zeroed 4-bit pool (every key and value zero)."""
    if not 8 <= block_size <= 256 or block_size & (block_size - 1):
        raise ValueError("a 4-bit cache's block_size is a power of two in [8, 256]")
    return torch.zeros((num_blocks, num_kv_heads, block_size // 8, 9 * head_size),
                       dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=64)
def _int8_geometry(shape):
    """(descriptor, a reference to it, KV heads, head size) of an 8-bit pool's shape."""
    if len(shape) != 4 or shape[3] % 16 or shape[3] < 32:
        raise ValueError("an 8-bit cache must be [num_blocks, num_kv_heads, block_size / 8, "
                         "16 * (head_size + 1)]")
    nb, hkv, tiles, size = shape
    desc = CacheDesc(nb, 8 * tiles, hkv, size // 16 - 1, PA_INT8)
    return desc, ctypes.byref(desc), hkv, size // 16 - 1


def _int8_pool(cache: torch.Tensor):
    if cache.dtype is not torch.int8:
        raise TypeError("an 8-bit cache must be int8, got %s" % cache.dtype)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    return _int8_geometry(cache.shape)


def int8_cache_desc(cache: torch.Tensor) -> CacheDesc:
    """Descriptor of an 8-bit pool [num_blocks, num_kv_heads, block_size / 8, 16 * (head_size + 1)]."""
    d = _int8_pool(cache)[0]
    return CacheDesc(d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype)


def alloc_int8_cache(num_blocks: int, block_size: int, num_kv_heads: int, head_size: int,
                     device="cuda") -> torch.Tensor:
    """A zeroed 8-bit pool (every key and value zero)."""
    if not 8 <= block_size <= 256 or block_size & (block_size - 1):
        raise ValueError("an 8-bit cache's block_size is a power of two in [8, 256]")
    return torch.zeros((num_blocks, num_kv_heads, block_size // 8, 16 * (head_size + 1)),
                       dtype=torch.int8, device=device)


def _pool_desc(cache: torch.Tensor) -> CacheDesc:
    if cache.dtype == torch.uint8:
        return fp4_cache_desc(cache)
    return int8_cache_desc(cache) if cache.dtype == torch.int8 else cache_desc(cache)


def _dev_ptr(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return _cuda_raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ---------------------------------------------------------------------------
# kernels
# ---------------------------------------------------------------------------

def pa_reshape_and_cache(cache: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                         slot_mapping: torch.Tensor, stream=None) -> None:
    """cache[0/1, slot // bs, slot % bs] = key/value[t] for every slot >= 0."""
    desc = cache_desc(cache)
    n = key.shape[0]
    if key.shape != value.shape or tuple(key.shape[1:]) != (desc.num_kv_heads, desc.head_size):
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    if key.dtype != cache.dtype or value.dtype != cache.dtype:
        raise TypeError("key/value dtype must match the cache")
    if slot_mapping.shape != (n,):
        raise ValueError("slot_mapping must be [num_tokens]")
    _check(lib.pa_reshape_and_cache(_dev_ptr(cache, "cache"), ctypes.byref(desc),
                                    _dev_ptr(key, "key") if n else None,
                                    _dev_ptr(value, "value") if n else None,
                                    _dev_ptr(slot_mapping, "slot_mapping", torch.int64) if n else None,
                                    n, _stream(stream)), "pa_reshape_and_cache")


def pa_copy_blocks(cache: torch.Tensor, pairs: torch.Tensor, stream=None) -> None:
    """Copy block pairs[i, 0] to block pairs[i, 1] (keys and values)."""
    desc = _pool_desc(cache)
    n = pairs.shape[0] if pairs.numel() else 0
    if n and (pairs.dim() != 2 or pairs.shape[1] != 2):
        raise ValueError("pairs must be [num_pairs, 2]")
    _check(lib.pa_copy_blocks(_dev_ptr(cache, "cache"), ctypes.byref(desc),
                              _dev_ptr(pairs, "pairs", torch.int64) if n else None, n,
                              _stream(stream)), "pa_copy_blocks")


def _dev_or_pinned_ptr(t: torch.Tensor, name: str, dtype=None) -> int:
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("%s must be a CUDA tensor or page-locked host memory" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def pa_copy_bytes(dst: torch.Tensor, src: torch.Tensor, stream=None) -> None:
    """Copy src's bytes into dst with a library kernel; either side may be
    page-locked host memory.  Both contiguous, with the same byte size."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src differ in byte size")
    if nbytes == 0:
        return
    _check(lib.pa_copy_bytes(_dev_or_pinned_ptr(dst, "dst"), _dev_or_pinned_ptr(src, "src"),
                             nbytes, _stream(stream)), "pa_copy_bytes")


def pa_swap_blocks(dst_cache: torch.Tensor, src_cache: torch.Tensor, pairs: torch.Tensor,
                   stream=None) -> None:
    """Copy block pairs[i, 0] of src_cache to block pairs[i, 1] of dst_cache
    (keys and values); either pool may be page-locked host memory."""
    n = pairs.shape[0] if pairs.numel() else 0
    if n and (pairs.dim() != 2 or pairs.shape[1] != 2):
        raise ValueError("pairs must be [num_pairs, 2]")
    dd, sd = _pool_desc(dst_cache), _pool_desc(src_cache)
    _check(lib.pa_swap_blocks(_dev_or_pinned_ptr(dst_cache, "dst_cache"), ctypes.byref(dd),
                              _dev_or_pinned_ptr(src_cache, "src_cache"), ctypes.byref(sd),
                              _dev_or_pinned_ptr(pairs, "pairs", torch.int64) if n else None, n,
                              _stream(stream)), "pa_swap_blocks")


def pa_decode_partition_size(cache_or_desc, num_seqs: int, num_heads: int, max_seq_len: int,
                             partition_size: int = -1) -> int:
    desc = cache_or_desc if isinstance(cache_or_desc, CacheDesc) else cache_desc(cache_or_desc)
    out = ctypes.c_int32()
    _check(lib.pa_decode_partition_size(ctypes.byref(desc), num_seqs, num_heads, max_seq_len,
                                        partition_size, ctypes.byref(out)),
           "pa_decode_partition_size")
    return out.value


def pa_decode_select_kernel(cache_or_desc, num_seqs: int, num_heads: int, query_ptr: int = 0,
                            kernel: int = 0) -> int:
    """The kernel family (PA_KERNEL_SIMT or PA_KERNEL_TENSOR) pa_decode runs
    for these arguments; `query_ptr` is the query's device address (only its
    alignment matters), or 0 to assume a 256-byte aligned buffer."""
    desc = cache_or_desc if isinstance(cache_or_desc, CacheDesc) else cache_desc(cache_or_desc)
    out = ctypes.c_int32()
    _check(lib.pa_decode_select_kernel(ctypes.byref(desc), num_seqs, num_heads,
                                       ctypes.c_void_p(query_ptr or 256), kernel,
                                       ctypes.byref(out)),
           "pa_decode_select_kernel")
    return out.value


def pa_decode_workspace_size(cache_or_desc, num_seqs: int, num_heads: int, max_seq_len: int,
                             partition_size: int = -1) -> int:
    desc = cache_or_desc if isinstance(cache_or_desc, CacheDesc) else cache_desc(cache_or_desc)
    out = ctypes.c_size_t()
    _check(lib.pa_decode_workspace_size(ctypes.byref(desc), num_seqs, num_heads, max_seq_len,
                                        partition_size, ctypes.byref(out)),
           "pa_decode_workspace_size")
    return out.value


def alloc_workspace(nbytes: int, device) -> torch.Tensor | None:
    """Caller-owned decode workspace: zeroed (its header must start at zero),
    256-byte aligned by the caching allocator."""
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def pa_decode(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
              block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
              max_seq_len: int, partition_size: int = -1, workspace: torch.Tensor | None = None,
              stream=None, kernel: int = PA_KERNEL_AUTO) -> None:
    """out[s, hq] = softmax(scale * q[s, hq] . K_s) V_s over the paged tokens.
    kernel: PA_KERNEL_AUTO, PA_KERNEL_SIMT or PA_KERNEL_TENSOR (pa_decode_ex)."""
    desc = cache_desc(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != desc.head_size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    if query.dtype != cache.dtype or out.dtype != cache.dtype:
        raise TypeError("query/out dtype must match the cache")
    if block_tables.dim() != 2 or block_tables.shape[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib.pa_decode_ex(_dev_ptr(out, "out"), _dev_ptr(query, "query"),
                            _dev_ptr(cache, "cache"), ctypes.byref(desc),
                            _dev_ptr(block_tables, "block_tables", torch.int32),
                            block_tables.shape[1], _dev_ptr(seq_lens, "seq_lens", torch.int32), s,
                            hq, float(scale), int(max_seq_len), int(partition_size), ws_ptr,
                            ws_bytes, int(kernel), _stream(stream)), "pa_decode")


def pa_decode_append(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                     max_seq_len: int, key_new: torch.Tensor, value_new: torch.Tensor,
                     partition_size: int = -1, workspace: torch.Tensor | None = None,
                     stream=None, kernel: int = PA_KERNEL_AUTO) -> None:
    """pa_decode that first writes each sequence's newest token (position
    seq_lens[s] - 1; key_new / value_new [num_seqs, num_kv_heads, head_size])
    into its cache slot."""
    desc = cache_desc(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != desc.head_size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    for name, t in (("query", query), ("out", out), ("key_new", key_new), ("value_new", value_new)):
        if t.dtype != cache.dtype:
            raise TypeError("%s dtype must match the cache" % name)
    if key_new.shape != (s, desc.num_kv_heads, d) or value_new.shape != key_new.shape:
        raise ValueError("key_new/value_new must be [num_seqs, num_kv_heads, head_size]")
    if block_tables.dim() != 2 or block_tables.shape[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib.pa_decode_append(_dev_ptr(out, "out"), _dev_ptr(query, "query"),
                                _dev_ptr(cache, "cache"), ctypes.byref(desc),
                                _dev_ptr(block_tables, "block_tables", torch.int32),
                                block_tables.shape[1], _dev_ptr(seq_lens, "seq_lens", torch.int32),
                                s, hq, float(scale), int(max_seq_len), int(partition_size),
                                _dev_ptr(key_new, "key_new"), _dev_ptr(value_new, "value_new"),
                                ws_ptr, ws_bytes, int(kernel), _stream(stream)), "pa_decode_append")


SHARED_TILE_ROWS = 128


class SharedPlan:
    """pa_decode_shared_plan on host block tables and lengths: the plan
    (int32, host) and its sizes; `upload` gives the device copy the decode
    reads."""

    def __init__(self, block_tables, seq_lens, block_size: int, num_heads: int,
                 num_kv_heads: int, min_shared_blocks: int = 8):
        bt = torch.as_tensor(block_tables).to(torch.int32).contiguous().cpu()
        sl = torch.as_tensor(seq_lens).to(torch.int32).contiguous().cpu()
        if bt.dim() != 2 or sl.shape != (bt.shape[0],):
            raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
        n = bt.shape[0]
        self.plan = torch.zeros(4 + 6 * n, dtype=torch.int32)
        self.info = SharedPlanInfo()
        _check(lib.pa_decode_shared_plan(bt.data_ptr(), bt.shape[1], sl.data_ptr(), n, block_size,
                                         num_heads, num_kv_heads, min_shared_blocks,
                                         self.plan.data_ptr(), self.plan.numel(),
                                         ctypes.byref(self.info)), "pa_decode_shared_plan")
        self.plan = self.plan[:self.info.plan_ints].clone()

    @property
    def num_chunks(self) -> int:
        return int(self.info.num_chunks)

    def chunks(self):
        """[(first member index, members, shared tokens, group)] per chunk."""
        nc = self.num_chunks
        return [tuple(int(x) for x in self.plan[4 + 4 * c:8 + 4 * c]) for c in range(nc)]

    def seq_start(self):
        nc, n = self.num_chunks, int(self.plan[1])
        return self.plan[4 + 4 * nc:4 + 4 * nc + n].tolist()

    def members(self):
        nc, n = self.num_chunks, int(self.plan[1])
        return self.plan[4 + 4 * nc + n:].tolist()

    def upload(self, device="cuda") -> torch.Tensor:
        return self.plan.to(device)


def pa_decode_shared_workspace_size(cache_or_desc, num_seqs: int, num_heads: int,
                                    max_seq_len: int, plan: SharedPlan) -> int:
    desc = cache_or_desc if isinstance(cache_or_desc, CacheDesc) else cache_desc(cache_or_desc)
    out = ctypes.c_size_t()
    _check(lib.pa_decode_shared_workspace_size(ctypes.byref(desc), num_seqs, num_heads,
                                               int(max_seq_len), ctypes.byref(plan.info),
                                               ctypes.byref(out)),
           "pa_decode_shared_workspace_size")
    return out.value


def pa_decode_shared(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                     max_seq_len: int, plan: SharedPlan, plan_dev: torch.Tensor,
                     workspace: torch.Tensor | None, key_new: torch.Tensor | None = None,
                     value_new: torch.Tensor | None = None, stream=None) -> None:
    """pa_decode with the blocks the plan's groups share attended once per
    group (plan_dev: the plan's device copy, SharedPlan.upload)."""
    desc = cache_desc(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != desc.head_size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    if query.dtype != cache.dtype or out.dtype != cache.dtype:
        raise TypeError("query/out dtype must match the cache")
    if block_tables.dim() != 2 or block_tables.shape[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    if (key_new is None) != (value_new is None):
        raise ValueError("key_new and value_new go together")
    kn = vn = None
    if key_new is not None:
        if key_new.shape != (s, desc.num_kv_heads, d) or value_new.shape != key_new.shape:
            raise ValueError("key_new/value_new must be [num_seqs, num_kv_heads, head_size]")
        kn, vn = _dev_ptr(key_new, "key_new"), _dev_ptr(value_new, "value_new")
    if plan_dev.numel() < plan.info.plan_ints:
        raise ValueError("plan_dev is shorter than the plan")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check(lib.pa_decode_shared(_dev_ptr(out, "out"), _dev_ptr(query, "query"),
                                _dev_ptr(cache, "cache"), ctypes.byref(desc),
                                _dev_ptr(block_tables, "block_tables", torch.int32),
                                block_tables.shape[1], _dev_ptr(seq_lens, "seq_lens", torch.int32),
                                s, hq, float(scale), int(max_seq_len),
                                _dev_ptr(plan_dev, "plan", torch.int32), ctypes.byref(plan.info),
                                kn, vn, ws_ptr, ws_bytes, _stream(stream)), "pa_decode_shared")


# ---------------------------------------------------------------------------
# 4-bit pool and device-side tables
# ---------------------------------------------------------------------------

# The current device and the raw handle of a device's current stream, without the
# objects around them (2.9 -> 0.2 us a call).
_cuda_get_device = getattr(torch._C, "_cuda_getDevice", None)
_cuda_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_device(t: torch.Tensor, name: str) -> int:
    """The device of t, which has to be the current one (launches go there)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev != _cuda_get_device():
        raise ValueError("%s is on device %d, which is not the current one" % (name, dev))
    return dev


def _arg(t: torch.Tensor, name: str, dtype: torch.dtype, dev: int) -> int:
    """Address of a contiguous tensor of one type on one device."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on CUDA device %d" % (name, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, heads: int, head_size: int, dev: int):
    """Address and row stride (elements) of [n, heads, head_size] rows, which
    may lie apart (a slice of a fused projection's output)."""
    n, h, d = t.shape
    if h != heads or d != head_size:
        raise ValueError("%s must be [n, %d, %d], got %s" % (name, heads, head_size, tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on CUDA device %d" % (name, dev))
    row, inner, one = t.stride()
    if (one != 1 and d > 1) or (inner != d and h > 1):
        raise ValueError("%s: each row's heads must be contiguous" % name)
    return t.data_ptr(), (row if n > 1 else heads * head_size)


def _too_large(n) -> ValueError:
    """For sizes that ctypes would cut to 32 bits."""
    return ValueError("%d is past 2^31 - 1" % n)


def _int32(n) -> int:
    """n, which ctypes would cut to 32 bits (a large or a very negative one could pass for a valid one)."""
    n = int(n)
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        raise ValueError("%d is outside 32 bits" % n)
    return n


def _on(stream, dev: int) -> int:
    return _cuda_raw_stream(dev) if stream is None else _stream(stream)


def pa_reshape_and_cache_fp4(cache: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                             slot_mapping: torch.Tensor, key_scale: float = 1.0,
                             value_scale: float = 1.0, stream=None) -> None:
    """pa_reshape_and_cache into a 4-bit pool: key/value [n, num_kv_heads,
    head_size] (bf16 or fp32, rows may lie apart) are rounded to 4-bit codes
    with a scale per 16 elements; key_scale / value_scale are the pool's
    tensor scales (powers of two)."""
    _, desc, heads, size = _fp4_pool(cache)
    if key.shape != value.shape or key.dim() != 3:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    if key.dtype is not value.dtype:
        raise TypeError("key and value must have the same dtype")
    n = key.shape[0]
    if slot_mapping.shape != (n,):
        raise ValueError("slot_mapping must be [num_tokens]")
    dev = _current_device(cache, "cache")
    kp, ks = _rows(key, "key", heads, size, dev)
    vp, vs = _rows(value, "value", heads, size, dev)
    _check(lib.pa_reshape_and_cache_fp4(cache.data_ptr(), desc, kp, vp,
                                        _dtype_code(key), ks, vs,
                                        _arg(slot_mapping, "slot_mapping", torch.int64, dev), n,
                                        float(key_scale), float(value_scale), _on(stream, dev)),
           "pa_reshape_and_cache_fp4")


def pa_gather_cache_fp4(key: torch.Tensor, value: torch.Tensor, cache: torch.Tensor,
                        slot_mapping: torch.Tensor, key_scale: float = 1.0,
                        value_scale: float = 1.0, stream=None) -> None:
    """Read tokens back from a 4-bit pool: key/value [n, num_kv_heads,
    head_size] (bf16 or fp32, contiguous) receive what the slots hold; rows of
    negative slots stay as they were."""
    _, desc, heads, size = _fp4_pool(cache)
    if key.dim() != 3 or key.shape != value.shape:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    n, h, d = key.shape
    if h != heads or d != size:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    if slot_mapping.shape != (n,):
        raise ValueError("slot_mapping must be [num_tokens]")
    dev = _current_device(cache, "cache")
    _check(lib.pa_gather_cache_fp4(_arg(key, "key", key.dtype, dev),
                                   _arg(value, "value", key.dtype, dev), _dtype_code(key),
                                   cache.data_ptr(), desc,
                                   _arg(slot_mapping, "slot_mapping", torch.int64, dev), n,
                                   float(key_scale), float(value_scale), _on(stream, dev)),
           "pa_gather_cache_fp4")


def pa_decode_fp4_workspace_size(cache_or_desc, num_heads: int) -> int:
    """Workspace bytes of pa_decode_fp4, whatever the batch (alloc_workspace)."""
    desc = (cache_or_desc if isinstance(cache_or_desc, CacheDesc)
            else fp4_cache_desc(cache_or_desc))
    out = ctypes.c_size_t()
    _check(lib.pa_decode_fp4_workspace_size(ctypes.byref(desc), _int32(num_heads), ctypes.byref(out)),
           "pa_decode_fp4_workspace_size")
    return out.value


def pa_decode_fp4(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
                  block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                  workspace: torch.Tensor, key_scale: float = 1.0, value_scale: float = 1.0,
                  stream=None) -> None:
    """pa_decode over a 4-bit pool; query (rows may lie apart) and out are
    bf16 or fp32.  The launch depends on the shapes alone, so that a captured
    call serves sequences as they grow."""
    _, desc, _, size = _fp4_pool(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    if query.dtype is not out.dtype:
        raise TypeError("query and out must have the same dtype")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    if tables[1] > 0x7FFFFFFF:
        raise _too_large(tables[1])
    dev = _current_device(cache, "cache")
    qp, qs = _rows(query, "query", hq, d, dev)
    _check(lib.pa_decode_fp4(_arg(out, "out", query.dtype, dev), qp, _dtype_code(query), qs,
                             cache.data_ptr(), desc, float(key_scale), float(value_scale),
                             _arg(block_tables, "block_tables", torch.int32, dev),
                             tables[1], _arg(seq_lens, "seq_lens", torch.int32, dev), s,
                             hq, float(scale), _arg(workspace, "workspace", workspace.dtype, dev),
                             workspace.nbytes, _on(stream, dev)), "pa_decode_fp4")


def pa_extend_tables(block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     new_tokens: torch.Tensor, block_size: int, num_blocks: int,
                     slot_mapping: torch.Tensor, positions: torch.Tensor | None = None,
                     token_starts: torch.Tensor | None = None,
                     seq_lens_out: torch.Tensor | None = None,
                     free_blocks: torch.Tensor | None = None,
                     free_state: torch.Tensor | None = None,
                     free_state_out: torch.Tensor | None = None, stream=None) -> None:
    """Append new_tokens[r] tokens to every request on the device: block
    tables extended from the ring of free blocks (free_blocks, free_state =
    [front, blocks left]; without them the tables hold every block already),
    slots and positions of the new tokens, -1 behind them, lengths and ring
    state advanced (in place unless *_out are given)."""
    n, = seq_lens.shape
    tables, most = block_tables.shape, slot_mapping.shape
    if len(tables) != 2 or tables[0] != n or new_tokens.shape != (n,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens and new_tokens "
                         "[num_seqs]")
    if len(most) != 1:
        raise ValueError("slot_mapping must be [max_tokens]")
    if positions is not None and positions.shape != most:
        raise ValueError("positions must be [max_tokens]")
    if token_starts is not None and token_starts.shape != (n + 1,):
        raise ValueError("token_starts must be [num_seqs + 1]")
    if (free_blocks is None) != (free_state is None):
        raise ValueError("free_blocks and free_state go together")
    if free_state_out is not None and free_state is None:
        raise ValueError("free_state_out needs free_state")
    largest = max(tables[1], most[0], block_size, num_blocks,
                  0 if free_blocks is None else free_blocks.shape[0])
    if largest > 0x7FFFFFFF:
        raise _too_large(largest)
    block_size, num_blocks = _int32(block_size), _int32(num_blocks)
    dev = _current_device(block_tables, "block_tables")
    i32 = torch.int32
    lens = lens_out = _arg(seq_lens, "seq_lens", i32, dev)
    if seq_lens_out is not None:
        if seq_lens_out.shape != (n,):
            raise ValueError("seq_lens_out must be [num_seqs]")
        lens_out = _arg(seq_lens_out, "seq_lens_out", i32, dev)
    ring = state = state_out = None
    capacity = 0
    if free_state is not None:
        if free_state.shape != (2,) or free_blocks.dim() != 1:
            raise ValueError("free_blocks must be [capacity], free_state [2]")
        ring, capacity = _arg(free_blocks, "free_blocks", i32, dev), free_blocks.shape[0]
        state = state_out = _arg(free_state, "free_state", i32, dev)
        if free_state_out is not None:
            if free_state_out.shape != (2,):
                raise ValueError("free_state_out must be [2]")
            state_out = _arg(free_state_out, "free_state_out", i32, dev)
    _check(lib.pa_extend_tables(
        _arg(block_tables, "block_tables", i32, dev), tables[1], lens,
        _arg(new_tokens, "new_tokens", i32, dev), n, block_size, num_blocks, ring, capacity,
        state, lens_out, state_out, _arg(slot_mapping, "slot_mapping", torch.int64, dev),
        None if positions is None else _arg(positions, "positions", i32, dev),
        None if token_starts is None else _arg(token_starts, "token_starts", i32, dev),
        most[0], _on(stream, dev)), "pa_extend_tables")


# ---------------------------------------------------------------------------
# 8-bit pool, eviction, norms with rotation
# ---------------------------------------------------------------------------

def pa_reshape_and_cache_int8(cache: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                              slot_mapping: torch.Tensor, stream=None) -> None:
    """pa_reshape_and_cache into an 8-bit pool: key/value [n, num_kv_heads,
    head_size] (bf16 or fp32, rows may lie apart) are rounded to 8-bit codes with a
    scale per block and head.  A block's tokens are neighbours in the call."""
    _, desc, heads, size = _int8_pool(cache)
    if key.shape != value.shape or key.dim() != 3:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    if key.dtype is not value.dtype:
        raise TypeError("key and value must have the same dtype")
    n = key.shape[0]
    if slot_mapping.shape != (n,):
        raise ValueError("slot_mapping must be [num_tokens]")
    if n > 0x7FFFFFFF:
        raise _too_large(n)
    dev = _current_device(cache, "cache")
    kp, ks = _rows(key, "key", heads, size, dev)
    vp, vs = _rows(value, "value", heads, size, dev)
    _check(lib.pa_reshape_and_cache_int8(cache.data_ptr(), desc, kp, vp, _dtype_code(key), ks, vs,
                                         _arg(slot_mapping, "slot_mapping", torch.int64, dev), n,
                                         _on(stream, dev)), "pa_reshape_and_cache_int8")


def pa_gather_cache_int8(key: torch.Tensor, value: torch.Tensor, cache: torch.Tensor,
                         slot_mapping: torch.Tensor, stream=None) -> None:
    """Read tokens back from an 8-bit pool: key/value [n, num_kv_heads,
    head_size] (bf16 or fp32, contiguous) receive what the slots hold; rows of
    negative slots stay as they were."""
    _, desc, heads, size = _int8_pool(cache)
    if key.dim() != 3 or key.shape != value.shape:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    n, h, d = key.shape
    if h != heads or d != size:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_size]")
    if slot_mapping.shape != (n,):
        raise ValueError("slot_mapping must be [num_tokens]")
    if n > 0x7FFFFFFF:
        raise _too_large(n)
    dev = _current_device(cache, "cache")
    _check(lib.pa_gather_cache_int8(_arg(key, "key", key.dtype, dev),
                                    _arg(value, "value", key.dtype, dev), _dtype_code(key),
                                    cache.data_ptr(), desc,
                                    _arg(slot_mapping, "slot_mapping", torch.int64, dev), n,
                                    _on(stream, dev)), "pa_gather_cache_int8")


def pa_decode_int8_workspace_size(cache_or_desc, num_heads: int,
                                  block_tables: torch.Tensor | None = None) -> int:
    """Workspace bytes of pa_decode_int8 (alloc_workspace), whatever the batch;
    with block_tables, of calls over tables of that shape that keep weights."""
    desc = (cache_or_desc if isinstance(cache_or_desc, CacheDesc)
            else int8_cache_desc(cache_or_desc))
    seqs, blocks = (0, 0) if block_tables is None else block_tables.shape
    if max(seqs, blocks) > 0x7FFFFFFF:
        raise _too_large(max(seqs, blocks))
    out = ctypes.c_size_t()
    _check(lib.pa_decode_int8_workspace_size(ctypes.byref(desc), _int32(num_heads), seqs, blocks,
                                             ctypes.byref(out)), "pa_decode_int8_workspace_size")
    return out.value


def pa_decode_int8(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
                   block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                   workspace: torch.Tensor, block_weights: torch.Tensor | None = None,
                   block_weights_out: torch.Tensor | None = None, decay: float = 1.0,
                   stream=None) -> None:
    """pa_decode over an 8-bit pool; query (rows may lie apart) and out are bf16
    or fp32.  With block_weights (fp32, the tables' shape) the attention that
    each block gets is added to decay times what it holds (in place unless
    block_weights_out is given; that alone starts from zeros); whoever gives a row to
    a new sequence sets its weights to zero.  The launches depend on the shapes
    alone, so that a captured call serves sequences as they grow."""
    _, desc, _, size = _int8_pool(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    if query.dtype is not out.dtype:
        raise TypeError("query and out must have the same dtype")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    if tables[1] > 0x7FFFFFFF:
        raise _too_large(tables[1])
    dev = _current_device(cache, "cache")
    qp, qs = _rows(query, "query", hq, d, dev)
    before = after = None
    if block_weights is not None:
        if block_weights.shape != tables:
            raise ValueError("block_weights must have the shape of block_tables")
        before = after = _arg(block_weights, "block_weights", torch.float32, dev)
    if block_weights_out is not None:
        if block_weights_out.shape != tables:
            raise ValueError("block_weights_out must have the shape of block_tables")
        after = _arg(block_weights_out, "block_weights_out", torch.float32, dev)
    _check(lib.pa_decode_int8(_arg(out, "out", query.dtype, dev), qp, _dtype_code(query), qs,
                              cache.data_ptr(), desc,
                              _arg(block_tables, "block_tables", torch.int32, dev), tables[1],
                              _arg(seq_lens, "seq_lens", torch.int32, dev), s, hq, float(scale),
                              before, after, float(decay),
                              _arg(workspace, "workspace", workspace.dtype, dev), workspace.nbytes,
                              _on(stream, dev)), "pa_decode_int8")


def pa_evict_blocks(block_tables: torch.Tensor, block_weights: torch.Tensor,
                    seq_lens: torch.Tensor, block_size: int, max_blocks: int, keep_first: int = 1,
                    keep_last: int = 1, free_blocks: torch.Tensor | None = None,
                    free_state: torch.Tensor | None = None,
                    evicted_tokens: torch.Tensor | None = None,
                    block_tables_out: torch.Tensor | None = None,
                    block_weights_out: torch.Tensor | None = None,
                    seq_lens_out: torch.Tensor | None = None,
                    free_state_out: torch.Tensor | None = None,
                    evicted_tokens_out: torch.Tensor | None = None, stream=None) -> None:
    """Sequences of more than max_blocks blocks give up those of the least
    block_weights, the first keep_first and the last keep_last aside: rows of the
    tables and weights close up (what left follows in the table, zeros in the
    weights), lengths shrink, the ring of free blocks (free_blocks, free_state = [front, blocks
    left], as for pa_extend_tables) takes what left, evicted_tokens counts it.  All in place unless
    *_out are given."""
    n, = seq_lens.shape
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != n or block_weights.shape != tables:
        raise ValueError("block_tables and block_weights must be [num_seqs, max_blocks], seq_lens "
                         "[num_seqs]")
    if (free_blocks is None) != (free_state is None):
        raise ValueError("free_blocks and free_state go together")
    if free_state is None and free_state_out is not None:
        raise ValueError("free_state_out needs free_state")
    if evicted_tokens is None and evicted_tokens_out is not None:
        raise ValueError("evicted_tokens_out needs evicted_tokens")
    largest = max(tables[1], block_size, max_blocks, keep_first, keep_last,
                  0 if free_blocks is None else free_blocks.shape[0])
    if largest > 0x7FFFFFFF:
        raise _too_large(largest)
    block_size, max_blocks = _int32(block_size), _int32(max_blocks)
    keep_first, keep_last = _int32(keep_first), _int32(keep_last)
    dev = _current_device(block_tables, "block_tables")
    i32 = torch.int32

    def pair(before, after, name, dtype, shape):
        if before is None:
            return None, None
        if before.shape != shape or (after is not None and after.shape != shape):
            raise ValueError("%s must be %s" % (name, list(shape)))
        at = _arg(before, name, dtype, dev)
        return at, at if after is None else _arg(after, name + "_out", dtype, dev)

    t, t_out = pair(block_tables, block_tables_out, "block_tables", i32, tables)
    w, w_out = pair(block_weights, block_weights_out, "block_weights", torch.float32, tables)
    lens, lens_out = pair(seq_lens, seq_lens_out, "seq_lens", i32, (n,))
    state, state_out = pair(free_state, free_state_out, "free_state", i32, (2,))
    gone, gone_out = pair(evicted_tokens, evicted_tokens_out, "evicted_tokens", i32, (n,))
    ring, capacity = None, 0
    if free_blocks is not None:
        if free_blocks.dim() != 1:
            raise ValueError("free_blocks must be [capacity]")
        ring, capacity = _arg(free_blocks, "free_blocks", i32, dev), free_blocks.shape[0]
    _check(lib.pa_evict_blocks(t, w, tables[1], lens, n, block_size, max_blocks, keep_first,
                               keep_last, ring, capacity, state, gone, t_out, w_out, lens_out,
                               state_out, gone_out, _on(stream, dev)), "pa_evict_blocks")


def pa_norm_rope(query_out: torch.Tensor, key_out: torch.Tensor, query: torch.Tensor,
                 key: torch.Tensor, query_weight: torch.Tensor | None,
                 key_weight: torch.Tensor | None, cos_sin: torch.Tensor | None,
                 positions: torch.Tensor, eps: float = 1e-6, interleaved: bool = False,
                 position_offsets: torch.Tensor | None = None, stream=None) -> None:
    """RMS norm of every head of query [n, num_heads, head_size] and key [n,
    num_kv_heads, head_size] (bf16 or fp32, rows may lie apart; the outputs may
    be the inputs), its weight, and the rotation of the pairs (i, i + rotary / 2),
    or (2 i, 2 i + 1) if interleaved, by cos_sin [max_position, rotary] (cosines,
    then sines; fp32; None: no rotation) at positions (+ position_offsets).
    Rows of negative positions stay as they were."""
    n, heads, size = query.shape
    if query_out.shape != query.shape or key_out.shape != key.shape or key.dim() != 3 \
            or key.shape[0] != n or key.shape[2] != size:
        raise ValueError("query/query_out must be [n, num_heads, head_size], key/key_out [n, "
                         "num_kv_heads, head_size]")
    dtype = query.dtype
    for name, x in (("query_out", query_out), ("key", key), ("key_out", key_out)):
        if x.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, x.dtype))
    if positions.shape != (n,) or (position_offsets is not None and position_offsets.shape != (n,)):
        raise ValueError("positions and position_offsets must be [num_tokens]")
    kv_heads = key.shape[1]
    if max(n, heads, kv_heads) > 0x7FFFFFFF:
        raise _too_large(max(n, heads, kv_heads))
    dev = _current_device(query, "query")
    qo, qos = _rows(query_out, "query_out", heads, size, dev)
    ko, kos = _rows(key_out, "key_out", kv_heads, size, dev)
    q, qs = _rows(query, "query", heads, size, dev)
    k, ks = _rows(key, "key", kv_heads, size, dev)
    weights = []
    for name, w in (("query_weight", query_weight), ("key_weight", key_weight)):
        if w is not None and w.shape != (size,):
            raise ValueError("%s must be [head_size]" % name)
        weights.append(0 if w is None else _arg(w, name, dtype, dev))
    table = most = rotary = 0
    if cos_sin is not None:
        most, rotary = cos_sin.shape
        if most > 0x7FFFFFFF:
            raise _too_large(most)
        if rotary == 0:
            raise ValueError("cos_sin has no columns")
        table = _arg(cos_sin, "cos_sin", torch.float32, dev)
    at = _arg(positions, "positions", torch.int32, dev)
    off = 0 if position_offsets is None else _arg(position_offsets, "position_offsets", torch.int32, dev)
    _check(lib.pa_norm_rope(_norm_rope_bytes(qo, ko, q, k, qos, kos, qs, ks, weights[0], weights[1], table, at,
                                             off, eps, _dtype_code(query), n, heads, kv_heads, size, rotary,
                                             most, bool(interleaved)), _on(stream, dev)), "pa_norm_rope")


NO_ALLOC_WORKSPACE_BYTES = 16 << 20


def pa_decode_no_alloc(out: torch.Tensor, query: torch.Tensor, cache: torch.Tensor,
                       block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                       max_seq_len: int, partition_size: int = -1, stream=None) -> None:
    """pa_decode with the split-KV scratch in the library's own device array
    (for callers that cannot allocate device memory; see include/pa.h)."""
    desc = cache_desc(cache)
    s, hq, d = query.shape
    if out.shape != query.shape or d != desc.head_size:
        raise ValueError("query/out must be [num_seqs, num_heads, head_size]")
    if block_tables.dim() != 2 or block_tables.shape[0] != s or seq_lens.shape != (s,):
        raise ValueError("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]")
    _check(lib.pa_decode_no_alloc(_dev_ptr(out, "out"), _dev_ptr(query, "query"),
                                  _dev_ptr(cache, "cache"), ctypes.byref(desc),
                                  _dev_ptr(block_tables, "block_tables", torch.int32),
                                  block_tables.shape[1],
                                  _dev_ptr(seq_lens, "seq_lens", torch.int32), s, hq,
                                  float(scale), int(max_seq_len), int(partition_size),
                                  _stream(stream)), "pa_decode_no_alloc")


def pa_slot_mapping(block_tables: torch.Tensor, block_size: int, num_blocks: int,
                    seq_idx: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    """Host: physical slots of (sequence, position) pairs through CPU block tables."""
    bt = block_tables.to(torch.int32).contiguous().cpu()
    si = seq_idx.to(torch.int32).contiguous().cpu()
    po = positions.to(torch.int32).contiguous().cpu()
    n = si.numel()
    out = torch.empty(n, dtype=torch.int64)
    _check(lib.pa_slot_mapping(bt.data_ptr(), bt.shape[0], bt.shape[1], block_size, num_blocks,
                               si.data_ptr(), po.data_ptr(), n, out.data_ptr()), "pa_slot_mapping")
    return out


def pa_get_device_error(stream=None) -> int:
    """Synchronise, return and clear the device error word (PA_DEVERR_* bits)."""
    flags = ctypes.c_uint32()
    st = lib.pa_get_device_error(ctypes.byref(flags), _stream(stream))
    if st not in (PA_OK, PA_ERR_DEVICE_CHECK, PA_ERR_TIMEOUT):
        _check(st, "pa_get_device_error")
    return flags.value


# ---------------------------------------------------------------------------
# host block pool
# ---------------------------------------------------------------------------

class Pool:
    """The C++ block pool (pa_pool_*): block tables, slots, copy-on-write pairs."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None):
        self._h = ctypes.c_void_p()
        order = None
        if free_order is not None:
            self._order = (ctypes.c_int32 * num_blocks)(*[int(b) for b in free_order])
            order = ctypes.cast(self._order, ctypes.c_void_p)
        _check(lib.pa_pool_create(num_blocks, block_size, order, ctypes.byref(self._h)),
               "pa_pool_create")
        self.num_blocks = num_blocks
        self.block_size = block_size

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            lib.pa_pool_destroy(h)
            self._h = None

    def add_seq(self, num_tokens: int) -> int:
        out = ctypes.c_int64()
        _check(lib.pa_pool_add_seq(self._h, num_tokens, ctypes.byref(out)), "pa_pool_add_seq")
        return out.value

    def fork(self, parent: int) -> int:
        out = ctypes.c_int64()
        _check(lib.pa_pool_fork(self._h, parent, ctypes.byref(out)), "pa_pool_fork")
        return out.value

    def append_token(self, seq: int):
        """Returns (slot, pair) with pair = (src, dst) of a copy-on-write, or None."""
        slot = ctypes.c_int64()
        pair = (ctypes.c_int64 * 2)()
        _check(lib.pa_pool_append_token(self._h, seq, ctypes.byref(slot), pair),
               "pa_pool_append_token")
        return slot.value, (None if pair[0] < 0 else (pair[0], pair[1]))

    def append_tokens(self, seqs):
        """append_token for each sequence, all or nothing: (slots int64[n], pairs int64[k,2])."""
        n = len(seqs)
        s = torch.tensor(list(seqs), dtype=torch.int64)
        slots = torch.empty(n, dtype=torch.int64)
        pairs = torch.empty((max(n, 1), 2), dtype=torch.int64)
        k = ctypes.c_int32()
        _check(lib.pa_pool_append_tokens(self._h, s.data_ptr(), n, slots.data_ptr(),
                                         pairs.data_ptr(), ctypes.byref(k)),
               "pa_pool_append_tokens")
        return slots, pairs[:k.value].clone()

    def free_seq(self, seq: int) -> None:
        _check(lib.pa_pool_free_seq(self._h, seq), "pa_pool_free_seq")

    # -- prefix caching --------------------------------------------------------
    def add_seq_tokens(self, tokens):
        """New sequence from prompt token ids, sharing cached prefix blocks:
        (seq id, number of leading tokens whose KV is already cached)."""
        t = torch.tensor([int(x) for x in tokens], dtype=torch.int32)
        sid = ctypes.c_int64()
        cached = ctypes.c_int64()
        _check(lib.pa_pool_add_seq_tokens(self._h, t.data_ptr() if t.numel() else None, t.numel(),
                                          ctypes.byref(sid), ctypes.byref(cached)),
               "pa_pool_add_seq_tokens")
        return sid.value, cached.value

    def append_token_id(self, seq: int, token: int):
        """append_token that records the token id: (slot, pair or None)."""
        slot = ctypes.c_int64()
        pair = (ctypes.c_int64 * 2)()
        _check(lib.pa_pool_append_token_id(self._h, seq, int(token), ctypes.byref(slot), pair),
               "pa_pool_append_token_id")
        return slot.value, (None if pair[0] < 0 else (pair[0], pair[1]))

    def is_cached(self, block: int) -> bool:
        out = ctypes.c_int32()
        _check(lib.pa_pool_is_cached(self._h, block, ctypes.byref(out)), "pa_pool_is_cached")
        return bool(out.value)

    def free_queue(self):
        """The free queue, front (next handed out) first."""
        buf = (ctypes.c_int32 * max(self.num_blocks, 1))()
        n = ctypes.c_int32()
        _check(lib.pa_pool_free_queue(self._h, buf, self.num_blocks, ctypes.byref(n)),
               "pa_pool_free_queue")
        return list(buf[:n.value])

    def usage(self):
        """(tokens held by live sequences, physical blocks in use)."""
        t, b = ctypes.c_int64(), ctypes.c_int64()
        _check(lib.pa_pool_usage(self._h, ctypes.byref(t), ctypes.byref(b)), "pa_pool_usage")
        return t.value, b.value

    # -- swapping ---------------------------------------------------------------
    def set_cpu_blocks(self, n: int) -> None:
        _check(lib.pa_pool_set_cpu_blocks(self._h, n), "pa_pool_set_cpu_blocks")
        self.num_cpu_blocks = n

    def _swap(self, fn, name, seqs):
        s = torch.tensor([int(x) for x in seqs], dtype=torch.int64)
        cap = max(1, self.num_blocks)
        pairs = torch.empty((cap, 2), dtype=torch.int64)
        k = ctypes.c_int32()
        _check(fn(self._h, s.data_ptr() if s.numel() else None, s.numel(), pairs.data_ptr(),
                  ctypes.byref(k)), name)
        return pairs[:k.value].clone()

    def swap_out(self, seqs):
        """Move a sequence group to CPU blocks: int64 [k, 2] (GPU block, CPU block) pairs."""
        return self._swap(lib.pa_pool_swap_out, "pa_pool_swap_out", seqs)

    def swap_in(self, seqs):
        """Move a swapped group back: int64 [k, 2] (CPU block, GPU block) pairs."""
        return self._swap(lib.pa_pool_swap_in, "pa_pool_swap_in", seqs)

    def is_swapped(self, seq: int) -> bool:
        out = ctypes.c_int32()
        _check(lib.pa_pool_is_swapped(self._h, seq, ctypes.byref(out)), "pa_pool_is_swapped")
        return bool(out.value)

    def num_free_cpu(self) -> int:
        return int(lib.pa_pool_num_free_cpu(self._h))

    def reset_prefix_cache(self) -> None:
        _check(lib.pa_pool_reset_prefix_cache(self._h), "pa_pool_reset_prefix_cache")

    def table(self, seq: int):
        n = ctypes.c_int32()
        length = ctypes.c_int64()
        cap = 16
        while True:
            buf = (ctypes.c_int32 * cap)()
            st = lib.pa_pool_block_table(self._h, seq, buf, cap, ctypes.byref(n),
                                         ctypes.byref(length))
            if st == PA_OK:
                return list(buf[:n.value]), length.value
            if st == PA_ERR_INVALID_ARG and n.value > cap:
                cap = n.value
                continue
            _check(st, "pa_pool_block_table")

    def fill_tables(self, seqs, max_blocks_per_seq: int):
        """Dense int32 [n, max_blocks_per_seq] tables and int32 [n] lengths (host)."""
        n = len(seqs)
        s = torch.tensor(list(seqs), dtype=torch.int64)
        bt = torch.empty((n, max_blocks_per_seq), dtype=torch.int32)
        sl = torch.empty(n, dtype=torch.int32)
        _check(lib.pa_pool_fill_tables(self._h, s.data_ptr(), n, bt.data_ptr(),
                                       max_blocks_per_seq, sl.data_ptr()), "pa_pool_fill_tables")
        return bt, sl

    def slot(self, seq: int, pos: int) -> int:
        out = ctypes.c_int64()
        _check(lib.pa_pool_slot(self._h, seq, pos, ctypes.byref(out)), "pa_pool_slot")
        return out.value

    def ref_count(self, block: int) -> int:
        out = ctypes.c_int32()
        _check(lib.pa_pool_ref_count(self._h, block, ctypes.byref(out)), "pa_pool_ref_count")
        return out.value

    def num_free(self) -> int:
        return int(lib.pa_pool_num_free(self._h))


def tensor_core_supported(cache: torch.Tensor, num_heads: int) -> bool:
    """Whether PA_KERNEL_TENSOR has a kernel for this cache and head count."""
    try:
        pa_decode_select_kernel(cache, 1, num_heads, kernel=PA_KERNEL_TENSOR)
    except PAError as e:
        if e.status == PA_ERR_UNSUPPORTED:
            return False
        raise
    return True


def pa_set_decode_trace(buffer: torch.Tensor | None, events_per_role: int = 0) -> None:
    """Record the tensor-core decode's timeline into `buffer` (a CUDA tensor;
    see include/pa.h for the record format), or stop recording (None)."""
    if buffer is None:
        _check(lib.pa_set_decode_trace(None, 0, 0), "pa_set_decode_trace")
        return
    _check(lib.pa_set_decode_trace(_dev_ptr(buffer, "buffer"),
                                   buffer.numel() * buffer.element_size(), int(events_per_role)),
           "pa_set_decode_trace")


def pa_set_decode_wait_limit(cycles: int) -> None:
    """Limit (SM clock cycles) of the tensor-core decode's pipeline waits;
    0 restores the default.  A test hook: see include/pa.h."""
    _check(lib.pa_set_decode_wait_limit(int(cycles)), "pa_set_decode_wait_limit")
