"""Python binding of libpagedkv.so: argument marshalling only.

Every function here turns torch tensors into device pointers and sizes and
calls the C ABI declared in ``include/pagedkv.h``; the computation happens in
the library's CUDA kernels. There is no fallback: if the library is missing or
a call fails, a :class:`PagedKVError` is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading

import numpy as np
import torch

KV_FP16, KV_BF16, KV_E5M2, KV_INT8, KV_INT4 = 0, 1, 2, 3, 4
_NAMES = {"fp16": KV_FP16, "bf16": KV_BF16, "e5m2": KV_E5M2, "fp8_e5m2": KV_E5M2, "int8": KV_INT8,
          "int4": KV_INT4}
_TORCH = {torch.float16: KV_FP16, torch.bfloat16: KV_BF16, torch.uint8: KV_E5M2,
          torch.float8_e5m2: KV_E5M2, torch.int8: KV_INT8}
# Types as calls name them, with the tensors' dtypes that hold them (a uint8 tensor without a name is looked at).
_KNOWN = {(name, dt): code for named in (_NAMES.items(), _TORCH.items(), zip(range(5), range(5)))
          for name, code in named
          for dt in ((torch.float16, torch.bfloat16) if code <= KV_BF16 else (torch.uint8, torch.int8, torch.float8_e5m2))}
_KNOWN.update({(None, dt): code for dt, code in _TORCH.items() if dt is not torch.uint8})
BLOCK_SIZE = 16

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class PagedKVError(RuntimeError):
    pass


class _CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_size", ctypes.c_int32)]


def library_path() -> str:
    return os.path.join(_HERE, "libpagedkv.so")


def load_library(path: str | None = None):
    """Load libpagedkv.so (built in-tree by ``__graft_entry__.build()``). A profiling
    tool may pass the path of a variant build of the same library instead; the
    first load wins for the rest of the process."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or library_path()
        if not os.path.exists(path):
            raise PagedKVError(f"{path} is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i32, P = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER
        lib.pkv_kv_cache_write.argtypes = [vp, vp, ctypes.c_int, i32, vp, vp, vp, ctypes.c_int,
                                           P(_CacheDesc), vp, vp]
        lib.pkv_kv_cache_write.restype = ctypes.c_int
        lib.pkv_decode_workspace_bytes.argtypes = [i32, i32, i32, P(_CacheDesc)]
        lib.pkv_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.pkv_paged_attention_decode.argtypes = [
            vp, vp, i32, i32, i32, vp, vp, ctypes.c_int, P(_CacheDesc), vp, i32, vp,
            ctypes.c_float, vp, ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_varlen.argtypes = [
            vp, vp, vp, i32, i32, i32, i32, vp, vp, ctypes.c_int, P(_CacheDesc), vp, i32, vp,
            ctypes.c_float, vp, ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_varlen.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_tree.argtypes = [
            vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, ctypes.c_int, P(_CacheDesc), vp, i32, vp,
            ctypes.c_float, vp, ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_tree.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_noalloc.argtypes = [
            vp, vp, i32, i32, i32, vp, vp, ctypes.c_int, P(_CacheDesc), vp, i32, vp,
            ctypes.c_float, vp, vp]
        lib.pkv_paged_attention_decode_noalloc.restype = ctypes.c_int
        i64 = ctypes.c_int64
        lib.pkv_allocator_create.argtypes = [i32]
        lib.pkv_allocator_create.restype = vp
        lib.pkv_allocator_destroy.argtypes = [vp]
        lib.pkv_allocator_destroy.restype = None
        for fn in ("pkv_allocator_free_blocks", "pkv_allocator_evictable"):
            getattr(lib, fn).argtypes = [vp]
            getattr(lib, fn).restype = i32
        lib.pkv_allocator_refcount.argtypes = [vp, i32]
        lib.pkv_allocator_refcount.restype = i32
        lib.pkv_seq_add.argtypes = [vp, i64]
        lib.pkv_seq_add.restype = ctypes.c_int
        lib.pkv_seq_fork.argtypes = [vp, i64, i64]
        lib.pkv_seq_fork.restype = ctypes.c_int
        lib.pkv_seq_release.argtypes = [vp, i64]
        lib.pkv_seq_release.restype = ctypes.c_int
        lib.pkv_seq_length.argtypes = [vp, i64]
        lib.pkv_seq_length.restype = i32
        lib.pkv_seq_block_table.argtypes = [vp, i64, vp, i32]
        lib.pkv_seq_block_table.restype = i32
        lib.pkv_seq_append.argtypes = [vp, i64, i32, vp, vp, vp, vp]
        lib.pkv_seq_append.restype = ctypes.c_int
        lib.pkv_seq_truncate.argtypes = [vp, i64, i32]
        lib.pkv_seq_truncate.restype = ctypes.c_int
        lib.pkv_prefix_insert.argtypes = [vp, i64, vp, i32]
        lib.pkv_prefix_insert.restype = i32
        lib.pkv_seq_add_cached.argtypes = [vp, i64, vp, i32, vp]
        lib.pkv_seq_add_cached.restype = ctypes.c_int
        lib.pkv_copy_blocks.argtypes = [vp, vp, vp, ctypes.c_int, P(_CacheDesc), vp, vp, i32, vp, vp]
        lib.pkv_copy_blocks.restype = ctypes.c_int
        lib.pkv_kv_cache_write_int8.argtypes = [vp, vp, i32, vp, vp, vp, vp, P(_CacheDesc), vp, vp]
        lib.pkv_kv_cache_write_int8.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_int8.argtypes = [
            vp, vp, i32, i32, i32, vp, vp, vp, P(_CacheDesc), vp, i32, vp, ctypes.c_float, vp,
            ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_int8.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_int8_varlen.argtypes = [
            vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, P(_CacheDesc), vp, i32, vp, ctypes.c_float, vp,
            ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_int8_varlen.restype = ctypes.c_int
        lib.pkv_paged_attention_decode_int8_tree.argtypes = [
            vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, P(_CacheDesc), vp, i32, vp, ctypes.c_float, vp,
            ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_int8_tree.restype = ctypes.c_int
        lib.pkv_decode_chunked_workspace_bytes.argtypes = [vp, i32, i32, i32, P(_CacheDesc)]
        lib.pkv_decode_chunked_workspace_bytes.restype = ctypes.c_size_t
        lib.pkv_paged_attention_decode_chunked.argtypes = [
            vp, vp, vp, vp, i32, i32, vp, vp, vp, ctypes.c_int, P(_CacheDesc), vp, i32, ctypes.c_float, vp,
            ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_chunked.restype = ctypes.c_int
        cint, f32 = ctypes.c_int, ctypes.c_float
        lib.pkv_rotary_embed.argtypes = [vp, i64, vp, i64, cint, i32, i32, i32, vp, i32, vp, i32, i32, ctypes.c_double, i32, vp]
        lib.pkv_rotary_embed.restype = cint
        lib.pkv_rotary_write.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, cint, i32, i32, vp, i32, vp, vp, i32,
                                         i32, ctypes.c_double, vp, vp, vp, cint, P(_CacheDesc), vp, vp]
        lib.pkv_rotary_write.restype = cint
        lib.pkv_prefill_workspace_bytes.argtypes = [i32, i32, i32, P(_CacheDesc)]
        lib.pkv_prefill_workspace_bytes.restype = ctypes.c_size_t
        lib.pkv_paged_attention_prefill.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, cint, P(_CacheDesc), vp,
                                                    i32, vp, f32, vp, ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_prefill.restype = cint
        lib.pkv_kv_cache_accept.argtypes = [vp, vp, vp, cint, P(_CacheDesc), vp, i32, vp, vp, i32, i32, vp, i32, vp,
                                            vp, vp, vp]
        lib.pkv_kv_cache_accept.restype = cint
        lib.pkv_kv_cache_write_int4.argtypes = [vp, vp, cint, i32, vp, vp, vp, vp, P(_CacheDesc), vp, vp]
        lib.pkv_kv_cache_write_int4.restype = cint
        lib.pkv_kv_cache_read.argtypes = [vp, vp, cint, i32, vp, vp, vp, vp, cint, P(_CacheDesc), vp, vp]
        lib.pkv_kv_cache_read.restype = cint
        lib.pkv_paged_attention_decode_int4.argtypes = [vp, vp, cint, vp, vp, i32, i32, i32, i32, vp, vp, vp,
                                                        P(_CacheDesc), vp, i32, vp, f32, vp, ctypes.c_size_t, vp, vp]
        lib.pkv_paged_attention_decode_int4.restype = cint
        lib.pkv_paged_attention_decode_int4_chunked.argtypes = [vp, vp, cint, vp, vp, i32, i32, vp, vp, vp,
                                                                P(_CacheDesc), vp, i32, f32, vp, ctypes.c_size_t, vp,
                                                                vp]
        lib.pkv_paged_attention_decode_int4_chunked.restype = cint
        lib.pkv_decode_counter_bytes.argtypes = [i32, i32, i32, P(_CacheDesc), cint]
        lib.pkv_decode_counter_bytes.restype = ctypes.c_size_t
        lib.pkv_capture_watch.argtypes = [vp, P(ctypes.c_uint64), P(vp)]
        lib.pkv_capture_watch.restype = cint
        lib.pkv_capture_gone.argtypes = [vp]
        lib.pkv_capture_gone.restype = cint
        lib.pkv_selftest_bounded_wait.argtypes = [vp, ctypes.c_uint64, vp, vp]
        lib.pkv_selftest_bounded_wait.restype = ctypes.c_int
        lib.pkv_error_string.argtypes = [ctypes.c_int]
        lib.pkv_error_string.restype = ctypes.c_char_p
        lib.pkv_version.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load_library().pkv_error_string(rc).decode()
        raise PagedKVError(f"{what} failed: {msg} ({rc})")


def _kv_code(kv_dtype, cache: torch.Tensor) -> int:
    """The cache's type: as named, which must have elements of the tensor's size (a wider one would lie
    beyond the tensor), or by the tensor's dtype."""
    code = _KNOWN.get((kv_dtype, cache.dtype))
    if code is not None:
        return code
    if kv_dtype is None:
        if cache.dtype is torch.uint8 and getattr(cache, "_pkv_int4", False):
            raise PagedKVError('calls on an INT4 cache name its type (kv_dtype="int4")')
        return _TORCH[cache.dtype]
    if isinstance(kv_dtype, str):
        code = _NAMES[kv_dtype]
    elif isinstance(kv_dtype, torch.dtype):
        code = _TORCH[kv_dtype]
    else:
        code = int(kv_dtype)
    if 0 <= code <= KV_INT4 and cache.element_size() != (2 if code <= KV_BF16 else 1):
        raise PagedKVError(f"a {cache.dtype} tensor is no cache of type {kv_dtype}" +
                           (" (torch.uint8)" if code == KV_INT4 else ""))
    return code


def _src_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return KV_FP16
    if t.dtype == torch.bfloat16:
        return KV_BF16
    raise PagedKVError(f"unsupported key/value/query dtype {t.dtype}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _desc(cache: torch.Tensor) -> _CacheDesc:
    if cache.dim() != 4 or cache.shape[2] != BLOCK_SIZE:
        raise PagedKVError(f"cache must be [num_blocks, num_kv_heads, 16, head_size], got {tuple(cache.shape)}")
    return _CacheDesc(cache.shape[0], cache.shape[2], cache.shape[1], cache.shape[3])


def _pair(k_cache, v_cache, packed=False) -> _CacheDesc:
    d = _desc(k_cache)
    if tuple(v_cache.shape) != tuple(k_cache.shape) or v_cache.dtype != k_cache.dtype:
        raise PagedKVError("k_cache and v_cache must have the same shape and dtype")
    if packed:   # an INT4 cache, two dimensions a byte
        if k_cache.dtype is not torch.uint8:
            raise PagedKVError("an INT4 cache is a torch.uint8 tensor (alloc_kv_cache)")
        d.head_size *= 2
    return d


def _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens, rows=None, max_rows=None):
    """The library sees only pointers: check here that every tensor is as large as
    the call will read or write. Returns (cache descriptor, num_seqs)."""
    d = _pair(k_cache, v_cache)
    if q.dim() != 3 or tuple(out.shape) != tuple(q.shape):
        raise PagedKVError(f"q and out must both be [rows, num_q_heads, head_size], got "
                           f"{tuple(q.shape)} and {tuple(out.shape)}")
    if int(q.shape[2]) != int(k_cache.shape[3]):
        raise PagedKVError(f"query head size {int(q.shape[2])} != cache head size {int(k_cache.shape[3])}")
    if context_lens.dim() != 1:
        raise PagedKVError("context_lens must be 1-D [num_seqs]")
    S = int(context_lens.shape[0])
    if block_tables.dim() != 2 or int(block_tables.shape[0]) < S:
        raise PagedKVError(f"block_tables must be [num_seqs, max_blocks_per_seq], got {tuple(block_tables.shape)}")
    if rows is not None and int(q.shape[0]) != rows:
        raise PagedKVError(f"q must have num_seqs * q_per_seq = {rows} rows, got {int(q.shape[0])}")
    if max_rows is not None and not (S <= int(q.shape[0]) <= max_rows):
        raise PagedKVError(f"q must have between num_seqs and num_seqs * max_q_per_seq rows, got {int(q.shape[0])}")
    return d, S


def _scales_shape(k_cache, scales, code=KV_INT8):
    if code == KV_INT4:
        nb, hkv, _, half = k_cache.shape
        want = (nb, hkv, 2, BLOCK_SIZE, half // 32, 2)
        if scales.shape != want or scales.dtype is not torch.float16:
            raise PagedKVError(f"scales must be float16 {want} (scale and least value of every 64 dimensions)")
        return
    want = (*k_cache.shape[:2], 2, BLOCK_SIZE)
    if scales.shape != want or scales.dtype != torch.float32:
        raise PagedKVError(f"scales must be float32 {want} (K then V row scales)")


def _write_shapes(key, value, slot_mapping, k_cache, v_cache) -> _CacheDesc:
    d = _pair(k_cache, v_cache)
    want = (int(k_cache.shape[1]), int(k_cache.shape[3]))
    if key.dim() != 3 or tuple(value.shape) != tuple(key.shape) or tuple(key.shape[1:]) != want:
        raise PagedKVError(f"key and value must both be [T, {want[0]}, {want[1]}], got "
                           f"{tuple(key.shape)} and {tuple(value.shape)}")
    if slot_mapping.dim() != 1 or int(slot_mapping.shape[0]) != int(key.shape[0]):
        raise PagedKVError("slot_mapping must be 1-D with one slot per token")
    return d


def _need_cuda_contig(name, t):
    if not t.is_cuda:
        raise PagedKVError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise PagedKVError(f"{name} must be contiguous")


def alloc_kv_cache(num_blocks: int, num_kv_heads: int, head_size: int, kv_dtype,
                   device="cuda", zero: bool = True):
    """Allocate a K/V cache pair [num_blocks, num_kv_heads, 16, head_size]. An INT8
    cache is a torch.int8 tensor whose bytes hold the codes in offset binary
    (byte = code + 128; :func:`int8_codes` reads them back). An INT4 cache is a torch.uint8
    tensor [num_blocks, num_kv_heads, 16, head_size / 2] of packed codes
    (:func:`kv_cache_read` reads them back); calls on it name its type (kv_dtype="int4") and are
    refused if they do not. (The tensors of this call are marked; a view or a copy of one is not,
    and counts as an E5M2 cache in a call that names no type.) ``zero`` fills the caches with the
    value 0 (for INT8: code 0, byte 0x80)."""
    code = _NAMES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype)
    dt = {KV_FP16: torch.float16, KV_BF16: torch.bfloat16, KV_E5M2: torch.uint8, KV_INT8: torch.int8,
          KV_INT4: torch.uint8}[code]
    if code == KV_INT4 and head_size not in (64, 128):
        raise PagedKVError(f"an INT4 cache has head size 64 or 128, got {head_size}")
    shape = (num_blocks, num_kv_heads, BLOCK_SIZE, head_size // 2 if code == KV_INT4 else head_size)
    if zero:
        fill = -128 if code == KV_INT8 else 0   # int8 -128 is the byte 0x80
        pair = torch.full(shape, fill, dtype=dt, device=device), torch.full(shape, fill, dtype=dt, device=device)
    else:
        pair = torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device)
    if code == KV_INT4:
        for t in pair:
            t._pkv_int4 = True   # bytes like an E5M2 cache's
    return pair


def alloc_kv_scales(num_blocks: int, num_kv_heads: int, device="cuda", *, kv_dtype="int8",
                    head_size: int | None = None):
    """Row scales of an INT8 cache pair: one float32 tensor [num_blocks, num_kv_heads, 2, 16],
    [..., 0, t] the K scale and [..., 1, t] the V scale of token t of a block. Of an INT4 cache pair
    (kv_dtype="int4", head_size): float16 [num_blocks, num_kv_heads, 2, 16, head_size / 64, 2], the
    scale and the least value of every 64 dimensions."""
    code = _NAMES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype)
    if code == KV_INT4:
        if head_size not in (64, 128):
            raise PagedKVError(f"an INT4 cache's scales need its head size, 64 or 128, got {head_size}")
        return torch.zeros((num_blocks, num_kv_heads, 2, BLOCK_SIZE, head_size // 64, 2), dtype=torch.float16,
                           device=device)
    if code != KV_INT8:
        raise PagedKVError("only INT8 and INT4 caches have scales")
    return torch.zeros((num_blocks, num_kv_heads, 2, BLOCK_SIZE), dtype=torch.float32, device=device)


def int8_codes(cache: torch.Tensor) -> torch.Tensor:
    """The signed codes of an INT8 cache, whose bytes are stored in offset binary
    (byte = code + 128): a torch.int8 tensor of the same shape and device."""
    if cache.dtype != torch.int8:
        raise PagedKVError("int8_codes reads an INT8 cache (torch.int8)")
    return (cache.view(torch.uint8).to(torch.int16) - 128).to(torch.int8)


def kv_cache_write_int8(key, value, slot_mapping, k_cache, v_cache, scales, *,
                        device_status=None, stream=None):
    """Quantise fp16 key/value [T, Hkv, D] into INT8 caches (codes in offset binary,
    byte = code + 128) and their row scales."""
    for n, t in (("key", key), ("value", value), ("slot_mapping", slot_mapping), ("k_cache", k_cache),
                 ("v_cache", v_cache), ("scales", scales)):
        _need_cuda_contig(n, t)
    if key.dtype != torch.float16 or k_cache.dtype != torch.int8 or scales.dtype != torch.float32:
        raise PagedKVError("INT8 cache write takes fp16 key/value, int8 caches, float32 scales")
    if slot_mapping.dtype != torch.int32:
        raise PagedKVError("slot_mapping must be int32")
    d = _write_shapes(key, value, slot_mapping, k_cache, v_cache)
    _scales_shape(k_cache, scales)
    rc = load_library().pkv_kv_cache_write_int8(
        _ptr(key), _ptr(value), int(key.shape[0]), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
        _ptr(scales), ctypes.byref(d), _ptr(device_status), _stream_handle(stream, key.device))
    _check(rc, "kv_cache_write_int8")


def paged_attention_decode_int8(out, q, k_cache, v_cache, scales, block_tables, context_lens,
                                q_per_seq: int, scale: float, *, workspace=None, device_status=None,
                                stream=None):
    """paged_attention_decode over an INT8 cache with its row scales (q/out fp16)."""
    for n, t in (("out", out), ("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("scales", scales),
                 ("block_tables", block_tables), ("context_lens", context_lens)):
        _need_cuda_contig(n, t)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise PagedKVError("block_tables and context_lens must be int32")
    d, S = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                          rows=int(context_lens.shape[0]) * int(q_per_seq))
    _scales_shape(k_cache, scales)
    Hq = int(q.shape[1])
    lib = load_library()
    with _on_device(q.device):
        if workspace is None:
            workspace = _decode_workspace(lib, q.get_device(), stream, S, Hq, int(q_per_seq), ctypes.byref(d), d.num_kv_heads,
                                          d.head_size, KV_INT8)
        rc = lib.pkv_paged_attention_decode_int8(
            _ptr(out), _ptr(q), S, Hq, int(q_per_seq), _ptr(k_cache), _ptr(v_cache), _ptr(scales),
            ctypes.byref(d), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
            float(scale), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
            _ptr(device_status), _stream_handle(stream, q.device))
    _check(rc, "paged_attention_decode_int8")
    return out


def kv_cache_write(key, value, slot_mapping, k_cache, v_cache, kv_dtype=None, *,
                   device_status=None, stream=None):
    """Scatter key/value [T, Hkv, D] into their cache slots (fp16->E5M2 cast for an E5M2 cache)."""
    for n, t in (("key", key), ("value", value), ("slot_mapping", slot_mapping),
                 ("k_cache", k_cache), ("v_cache", v_cache)):
        _need_cuda_contig(n, t)
    if slot_mapping.dtype != torch.int32:
        raise PagedKVError("slot_mapping must be int32")
    d, hkv, head = _desc_of(k_cache, v_cache)
    shape = key.shape
    if len(shape) != 3 or shape[1] != hkv or shape[2] != head or value.shape != shape or \
            slot_mapping.shape != shape[:1]:
        _write_shapes(key, value, slot_mapping, k_cache, v_cache)
    rc = load_library().pkv_kv_cache_write(
        key.data_ptr(), value.data_ptr(), _src_code(key), shape[0], slot_mapping.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _kv_code(kv_dtype, k_cache), d,
        _addr(device_status), _stream_of(stream, key.get_device()))
    _check(rc, "kv_cache_write")


def decode_workspace_bytes(num_seqs: int, num_q_heads: int, q_per_seq: int, k_cache, kv_dtype=None) -> int:
    """Bytes of workspace a decode call needs for this problem on the cache's device."""
    d = _desc(k_cache)
    if _kv_code(kv_dtype, k_cache) == KV_INT4:   # (two dimensions a byte)
        d.head_size *= 2
    with torch.cuda.device(k_cache.device):
        return int(load_library().pkv_decode_workspace_bytes(num_seqs, num_q_heads, q_per_seq,
                                                             ctypes.byref(d)))


def _on_device(device):
    """The device context for a call, entered only when the tensors are not on the current device."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


class _Scratch:
    """A buffer of calls that follow one another on a stream. Its first ``clean`` bytes hold nothing
    but piece counters, which every launch leaves clear; a call that has more of them clears the
    rest first."""
    __slots__ = ("ws", "size", "clean")

    def __init__(self):
        self.ws, self.size, self.clean = None, 0, -1

    def take(self, nbytes: int, counters: int, dev: int) -> torch.Tensor:
        if self.clean != counters or self.size < nbytes:
            if self.ws is None or self.size < nbytes:
                self.size, self.clean = max(nbytes, 256), 0
                self.ws = torch.empty(self.size, dtype=torch.uint8, device=dev)
            if self.clean < counters:
                self.ws[self.clean:counters].zero_()
            self.clean = counters
        return self.ws


class _Capture:
    """Scratch of the calls captured into one graph, from its memory pool and held until the graph
    and its executables are gone: what a replay writes to is nobody else's, and nothing else
    leaves its numbers where a replay expects clear counters."""
    __slots__ = ("watch", "scratch", "outgrown")

    def __init__(self, watch):
        self.watch, self.scratch, self.outgrown = watch, {}, []


_scratches: dict = {}   # (kind, device, stream): _Scratch
_captures: dict = {}    # capture: _Capture


def _scratch(kind: str, nbytes: int, counters: int, dev: int, stream) -> torch.Tensor:
    """Scratch of a call whose first ``counters`` bytes are its piece counters: one buffer per kind,
    device and stream that calls run on, grown as needed; a graph's own for captured calls."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _scratch_here((kind, dev, stream.cuda_stream), nbytes, counters)
    return _scratch_here((kind, dev, _stream_of(None, dev)), nbytes, counters)


def _scratch_here(key, nbytes: int, counters: int) -> torch.Tensor:
    if torch.cuda.is_current_stream_capturing():
        return _captured_scratch(key, nbytes, counters)
    s = _scratches.get(key)
    if s is None or s.size < nbytes:
        with _lock_captures:
            _let_go(load_library())
        if s is None:
            s = _scratches[key] = _Scratch()
    return s.take(nbytes, counters, key[1])


def _let_go(lib):
    """Gives back the scratch of graphs that are gone (looked at whenever a buffer is about to be made)."""
    for gone in [c for c, h in _captures.items() if lib.pkv_capture_gone(h.watch)]:
        del _captures[gone]


def _captured_scratch(key, nbytes: int, counters: int) -> torch.Tensor:
    lib, capture, watch = load_library(), ctypes.c_uint64(), ctypes.c_void_p()
    with _lock_captures:
        _check(lib.pkv_capture_watch(key[2], ctypes.byref(capture), None), "capture")
        held = _captures.get(capture.value)
        if held is None:
            _let_go(lib)
            _check(lib.pkv_capture_watch(key[2], ctypes.byref(capture), ctypes.byref(watch)), "capture")
            held = _captures[capture.value] = _Capture(watch.value)
        s = held.scratch.get(key)
        if s is None:
            s = held.scratch[key] = _Scratch()
        old = s.ws
        ws = s.take(nbytes, counters, key[1])
        if old is not None and old is not ws:
            held.outgrown.append(old)
        return ws


_lock_captures = threading.Lock()
_decode_sizes: dict = {}


def _decode_workspace(lib, dev: int, stream, S, Hq, n, desc, hkv, head, code) -> torch.Tensor:
    """Scratch of a decode call (sizes kept per device and problem shape)."""
    key = (dev, S, Hq, n, hkv, head, code)
    sizes = _decode_sizes.get(key)
    if sizes is None:
        sizes = (int(lib.pkv_decode_workspace_bytes(S, Hq, n, desc)),
                 int(lib.pkv_decode_counter_bytes(S, Hq, n, desc, code)))
        if sizes[0] and sizes[1]:   # (else refused: the call says why)
            if len(_decode_sizes) > 4096:
                _decode_sizes.clear()
            _decode_sizes[key] = sizes
    return _scratch("decode", *sizes, dev, stream)


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, q_per_seq: int,
                           scale: float, kv_dtype=None, *, workspace=None, device_status=None,
                           stream=None):
    """out[s*n+j, hq] = softmax(scale * q K^T) V over sequence s's blocks (causal among its
    n = q_per_seq query tokens). q/out: [S*n, Hq, D]; caches [NB, Hkv, 16, D]."""
    for n, t in (("out", out), ("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("block_tables", block_tables), ("context_lens", context_lens)):
        _need_cuda_contig(n, t)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise PagedKVError("block_tables and context_lens must be int32")
    if out.dtype != q.dtype:
        raise PagedKVError("out and q must share a dtype")
    d, S = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                          rows=int(context_lens.shape[0]) * int(q_per_seq))
    Hq = int(q.shape[1])
    code = _kv_code(kv_dtype, k_cache)
    lib = load_library()
    with _on_device(q.device):
        if workspace is None:
            workspace = _decode_workspace(lib, q.get_device(), stream, S, Hq, int(q_per_seq), ctypes.byref(d), d.num_kv_heads,
                                          d.head_size, code)
        rc = lib.pkv_paged_attention_decode(
            _ptr(out), _ptr(q), S, Hq, int(q_per_seq), _ptr(k_cache), _ptr(v_cache), code,
            ctypes.byref(d), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens),
            float(scale), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
            _ptr(device_status), _stream_handle(stream, q.device))
    _check(rc, "paged_attention_decode")
    return out


def paged_attention_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens,
                                   q_per_seq: int, scale: float, kv_dtype=None, *,
                                   device_status=None, stream=None):
    """Same as :func:`paged_attention_decode`, but the split-KV scratch comes from a
    fixed buffer inside the library, so neither this call nor the library allocates
    device memory (for callers that cannot allocate at this point). Problems too
    large for that buffer raise PagedKVError ("workspace too small"). Calls that
    overlap on the GPU share the buffer and must be serialised."""
    for n, t in (("out", out), ("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("block_tables", block_tables), ("context_lens", context_lens)):
        _need_cuda_contig(n, t)
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise PagedKVError("block_tables and context_lens must be int32")
    if out.dtype != q.dtype:
        raise PagedKVError("out and q must share a dtype")
    d, _ = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                          rows=int(context_lens.shape[0]) * int(q_per_seq))
    with _on_device(q.device):
        rc = load_library().pkv_paged_attention_decode_noalloc(
            _ptr(out), _ptr(q), int(context_lens.shape[0]), int(q.shape[1]), int(q_per_seq),
            _ptr(k_cache), _ptr(v_cache), _kv_code(kv_dtype, k_cache), ctypes.byref(d),
            _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), float(scale),
            _ptr(device_status), _stream_handle(stream, q.device))
    _check(rc, "paged_attention_decode_noalloc")
    return out


def _int8_scales(code, k_cache, scales):
    """An INT8 or INT4 cache is read with its scales; other caches take none."""
    if (code in (KV_INT8, KV_INT4)) != (scales is not None):
        raise PagedKVError("an INT8 or INT4 cache is read with its scales (alloc_kv_scales); other caches take none")
    if scales is not None:
        _need_cuda_contig("scales", scales)
        _scales_shape(k_cache, scales, code)


def paged_attention_decode_varlen(out, q, cu_q_lens, k_cache, v_cache, block_tables, context_lens,
                                  max_q_per_seq: int, scale: float, kv_dtype=None, *, scales=None,
                                  workspace=None, device_status=None, stream=None):
    """Decode attention for a batch whose sequences carry different numbers of query
    tokens, packed without padding: sequence s owns rows cu_q_lens[s]..cu_q_lens[s+1]-1
    of q/out ([total_rows, Hq, D]), 1 <= n_s <= max_q_per_seq, causal among its tokens.
    An INT8 or INT4 cache takes its scales (``scales``)."""
    if _is_int4(kv_dtype):
        return _decode_int4("paged_attention_decode_varlen", out, q, cu_q_lens, None, k_cache, v_cache, scales,
                            block_tables, context_lens, max_q_per_seq, scale, workspace, device_status, stream)
    for nm, t in (("out", out), ("q", q), ("cu_q_lens", cu_q_lens), ("k_cache", k_cache),
                  ("v_cache", v_cache), ("block_tables", block_tables), ("context_lens", context_lens)):
        _need_cuda_contig(nm, t)
    if (block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32
            or cu_q_lens.dtype != torch.int32):
        raise PagedKVError("block_tables, context_lens and cu_q_lens must be int32")
    if out.dtype != q.dtype:
        raise PagedKVError("out and q must share a dtype")
    d, S = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens,
                          max_rows=int(context_lens.shape[0]) * int(max_q_per_seq))
    if cu_q_lens.dim() != 1 or int(cu_q_lens.shape[0]) != S + 1:
        raise PagedKVError("cu_q_lens must have num_seqs + 1 entries")
    code = _kv_code(kv_dtype, k_cache)
    _int8_scales(code, k_cache, scales)
    Hq = int(q.shape[1])
    lib = load_library()
    with _on_device(q.device):
        if workspace is None:
            workspace = _decode_workspace(lib, q.get_device(), stream, S, Hq, int(max_q_per_seq), ctypes.byref(d), d.num_kv_heads,
                                          d.head_size, code)
        ws = (_ptr(workspace), int(workspace.numel() * workspace.element_size()))
        if code == KV_INT8:
            rc = lib.pkv_paged_attention_decode_int8_varlen(
                _ptr(out), _ptr(q), _ptr(cu_q_lens), int(q.shape[0]), S, Hq, int(max_q_per_seq),
                _ptr(k_cache), _ptr(v_cache), _ptr(scales), ctypes.byref(d), _ptr(block_tables),
                int(block_tables.shape[1]), _ptr(context_lens), float(scale), *ws, _ptr(device_status),
                _stream_handle(stream, q.device))
        else:
            rc = lib.pkv_paged_attention_decode_varlen(
                _ptr(out), _ptr(q), _ptr(cu_q_lens), int(q.shape[0]), S, Hq, int(max_q_per_seq),
                _ptr(k_cache), _ptr(v_cache), code, ctypes.byref(d), _ptr(block_tables),
                int(block_tables.shape[1]), _ptr(context_lens), float(scale), *ws, _ptr(device_status),
                _stream_handle(stream, q.device))
    _check(rc, "paged_attention_decode_varlen")
    return out


def _host_i32(name, x, n=None) -> np.ndarray:
    """A host int32 array (list, numpy array or CPU tensor) the library reads directly."""
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            raise PagedKVError(f"{name} must be in host memory")
        x = x.numpy()
    a = np.ascontiguousarray(np.asarray(x), dtype=np.int32)
    if a.ndim != 1 or (n is not None and a.shape[0] != n):
        raise PagedKVError(f"{name} must be 1-D" + (f" with {n} entries" if n is not None else ""))
    return a


def paged_attention_decode_chunked(out, q, q_lens, context_lens, k_cache, v_cache, block_tables, scale: float,
                                   kv_dtype=None, *, scales=None, workspace=None, device_status=None,
                                   stream=None):
    """Decode attention for a batch whose sequences carry any number of query tokens
    (prefill chunks beside decode / verify tokens), packed without padding: sequence s
    owns the next q_lens[s] rows of q/out and its token j sees positions
    <= context_lens[s] - q_lens[s] + j. q_lens and context_lens are host arrays
    (lists, numpy arrays or CPU tensors), read when the call is made (a captured CUDA
    graph replays them)."""
    for nm, t in (("out", out), ("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                  ("block_tables", block_tables)):
        _need_cuda_contig(nm, t)
    if block_tables.dtype != torch.int32:
        raise PagedKVError("block_tables must be int32")
    if out.dtype != q.dtype:
        raise PagedKVError("out and q must share a dtype")
    ql = _host_i32("q_lens", q_lens)
    S = int(ql.shape[0])
    cl = _host_i32("context_lens", context_lens, S)
    if S and (ql.min() < 1 or np.any(cl < ql)):
        raise PagedKVError("every sequence needs 1 <= q_lens[s] <= context_lens[s]")
    code = _kv_code(kv_dtype, k_cache)
    d = _pair(k_cache, v_cache, code == KV_INT4)
    if q.dim() != 3 or tuple(out.shape) != tuple(q.shape) or int(q.shape[0]) != int(ql.sum()):
        raise PagedKVError(f"q and out must both be [sum(q_lens) = {int(ql.sum())}, num_q_heads, head_size]")
    if int(q.shape[2]) != d.head_size:
        raise PagedKVError(f"query head size {int(q.shape[2])} != cache head size {d.head_size}")
    if block_tables.dim() != 2 or int(block_tables.shape[0]) < S:
        raise PagedKVError(f"block_tables must be [num_seqs, max_blocks_per_seq], got {tuple(block_tables.shape)}")
    _int8_scales(code, k_cache, scales)
    Hq, mbs = int(q.shape[1]), int(block_tables.shape[1])
    lib = load_library()
    qp, cp = ql.ctypes.data_as(ctypes.c_void_p), cl.ctypes.data_as(ctypes.c_void_p)
    with _on_device(q.device):
        need = int(lib.pkv_decode_chunked_workspace_bytes(qp, S, Hq, mbs, ctypes.byref(d)))
        if S and need == 0:
            raise PagedKVError("paged_attention_decode_chunked: unsupported shape")
        if workspace is None:
            workspace = _scratch("chunked", need, 0, q.get_device(), stream)   # (it clears its counters itself)
        rest = (ctypes.byref(d), _ptr(block_tables), mbs, float(scale), _ptr(workspace),
                int(workspace.numel() * workspace.element_size()), _ptr(device_status),
                _stream_handle(stream, q.device))
        if code == KV_INT4:
            rc = lib.pkv_paged_attention_decode_int4_chunked(
                _ptr(out), _ptr(q), _src_code(q), qp, cp, S, Hq, _ptr(k_cache), _ptr(v_cache), _ptr(scales), *rest)
        else:
            rc = lib.pkv_paged_attention_decode_chunked(
                _ptr(out), _ptr(q), qp, cp, S, Hq, _ptr(k_cache), _ptr(v_cache), _ptr(scales), code, *rest)
    _check(rc, "paged_attention_decode_chunked")
    return out


def selftest_bounded_wait(limit_ns: int, device=None, stream=None):
    """Run the device self-test of the decode kernels' bounded waits (a wait on a
    barrier phase nothing completes gives up after limit_ns and flags
    PKV_DEV_TIMEOUT; a second wait leaves on the CTA's abort flag). Returns
    (status word, [duration of wait 0, duration of wait 1] in ns)."""
    device = torch.device(device or "cuda")
    status = torch.zeros(1, dtype=torch.int32, device=device)
    elapsed = torch.zeros(2, dtype=torch.int64, device=device)
    lib = load_library()
    with _on_device(status.device):
        rc = lib.pkv_selftest_bounded_wait(_ptr(status), int(limit_ns), _ptr(elapsed),
                                           _stream_handle(stream, status.device))
    _check(rc, "selftest_bounded_wait")
    torch.cuda.synchronize(status.device)
    return int(status.item()), [int(x) for x in elapsed.cpu().tolist()]


def paged_attention_decode_tree(out, q, tree_masks, k_cache, v_cache, block_tables, context_lens,
                                max_q_per_seq: int, scale: float, kv_dtype=None, *, cu_q_lens=None,
                                scales=None, workspace=None, device_status=None, stream=None):
    """Speculative verify of a token tree: tree_masks (int64/uint64, one per query row)
    bit i lets a query token attend to its sequence's draft token i; the context before
    the drafts is always visible. cu_q_lens as for paged_attention_decode_varlen, or
    None for max_q_per_seq tokens per sequence. An INT8 or INT4 cache takes its scales."""
    if _is_int4(kv_dtype):
        return _decode_int4("paged_attention_decode_tree", out, q, cu_q_lens, tree_masks, k_cache, v_cache, scales,
                            block_tables, context_lens, max_q_per_seq, scale, workspace, device_status, stream)
    for nm, t in (("out", out), ("q", q), ("tree_masks", tree_masks), ("k_cache", k_cache),
                  ("v_cache", v_cache), ("block_tables", block_tables), ("context_lens", context_lens)):
        _need_cuda_contig(nm, t)
    if tree_masks.dtype not in (torch.int64, torch.uint64):
        raise PagedKVError("tree_masks must be 64-bit")
    if cu_q_lens is not None:
        _need_cuda_contig("cu_q_lens", cu_q_lens)
    if out.dtype != q.dtype:
        raise PagedKVError("out and q must share a dtype")
    S0, n_max = int(context_lens.shape[0]), int(max_q_per_seq)
    if cu_q_lens is None:
        d, S = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens, rows=S0 * n_max)
    else:
        d, S = _decode_shapes(out, q, k_cache, v_cache, block_tables, context_lens, max_rows=S0 * n_max)
        if cu_q_lens.dim() != 1 or int(cu_q_lens.shape[0]) != S + 1 or cu_q_lens.dtype != torch.int32:
            raise PagedKVError("cu_q_lens must be int32 with num_seqs + 1 entries")
    if tree_masks.dim() != 1 or int(tree_masks.shape[0]) != int(q.shape[0]):
        raise PagedKVError("tree_masks must hold one mask per query row")
    code = _kv_code(kv_dtype, k_cache)
    _int8_scales(code, k_cache, scales)
    Hq = int(q.shape[1])
    lib = load_library()
    with _on_device(q.device):
        if workspace is None:
            workspace = _decode_workspace(lib, q.get_device(), stream, S, Hq, int(max_q_per_seq), ctypes.byref(d), d.num_kv_heads,
                                          d.head_size, code)
        ws = (_ptr(workspace), int(workspace.numel() * workspace.element_size()))
        if code == KV_INT8:
            rc = lib.pkv_paged_attention_decode_int8_tree(
                _ptr(out), _ptr(q), _ptr(cu_q_lens), _ptr(tree_masks), int(q.shape[0]), S, Hq,
                int(max_q_per_seq), _ptr(k_cache), _ptr(v_cache), _ptr(scales), ctypes.byref(d),
                _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), float(scale), *ws,
                _ptr(device_status), _stream_handle(stream, q.device))
        else:
            rc = lib.pkv_paged_attention_decode_tree(
                _ptr(out), _ptr(q), _ptr(cu_q_lens), _ptr(tree_masks), int(q.shape[0]), S, Hq,
                int(max_q_per_seq), _ptr(k_cache), _ptr(v_cache), code, ctypes.byref(d),
                _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), float(scale), *ws,
                _ptr(device_status), _stream_handle(stream, q.device))
    _check(rc, "paged_attention_decode_tree")
    return out


# ------------------------------------------------------------------------------------
# Rotary embedding, prefill attention, acceptance of drafts
# ------------------------------------------------------------------------------------

def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                    original_context: int | None = None, low: float = 1.0, high: float | None = None,
                    device=None):
    """Frequencies of a rotary embedding: (inv_freq float64 [rotary_dim / 2], attn_factor).

    inv_freq[i] = base^(-2i / rotary_dim) radians per position, changed for a context
    ``factor`` times as long by ``scaling``:

    * ``"linear"``: every frequency divided by factor.
    * ``"base"``: base * factor^(rotary_dim / (rotary_dim - 2)), which divides the lowest
      frequency by factor and leaves the highest.
    * ``"bands"``: by the turns a pair makes over ``original_context`` positions:
      at least ``high`` (default 4): kept; at most ``low`` (1): divided by factor; linear in
      the turns between.
    * ``"ramp"``: as bands with ``high`` 32, but linear in the pair's index between, and
      attn_factor = 0.1 ln(factor) + 1.
    """
    rd = int(rotary_dim)
    if rd < 2 or rd % 2 or not 0 < base < math.inf or not 0 < factor < math.inf:
        raise PagedKVError("rotary_dim must be even and positive, base and factor positive and finite")
    if scaling not in (None, "linear", "base", "bands", "ramp"):
        raise PagedKVError(f"unknown rotary scaling {scaling!r}")
    if scaling in ("bands", "ramp") and not (original_context and 0 < original_context < math.inf):
        raise PagedKVError(f"scaling {scaling!r} needs original_context")
    if scaling == "ramp" and not base > 1:
        raise PagedKVError("scaling 'ramp' needs base > 1: pairs that make fewer turns the higher their index")
    if scaling == "base":
        if rd == 2:
            raise PagedKVError("scaling 'base' needs rotary_dim > 2")
        if math.log(base) + math.log(factor) * rd / (rd - 2) > 700.0:
            raise PagedKVError("scaling 'base': base * factor^(rotary_dim / (rotary_dim - 2)) is out of range")
        base = base * factor ** (rd / (rd - 2))
    i = np.arange(rd // 2, dtype=np.float64)
    inv = base ** (-2.0 * i / rd)
    attn = 1.0
    if scaling == "linear":
        inv = inv / factor
    elif scaling in ("bands", "ramp"):
        high = (4.0 if scaling == "bands" else 32.0) if high is None else high
        if not math.inf > high > low > 0:
            raise PagedKVError("the bands need high > low > 0")
        if scaling == "bands":
            keep = (original_context * inv / (2 * np.pi) - low) / (high - low)
        else:
            # the (fractional) pair that makes r turns: base^(-2i/rd) * context = 2 pi r
            def pair(r):
                return rd * np.log(original_context / (2 * np.pi * r)) / (2 * np.log(base))
            first, last = max(np.floor(pair(high)), 0.0), min(np.ceil(pair(low)), rd - 1.0)
            keep = 1.0 - (i - first) / max(last - first, 1e-3)
            attn = 0.1 * float(np.log(factor)) + 1.0 if factor > 1 else 1.0
        keep = np.clip(keep, 0.0, 1.0)
        inv = inv * keep + inv / factor * (1.0 - keep)
    return torch.from_numpy(inv).to(device=device or "cuda"), attn


def _placed(names, tensors) -> int:
    """The CUDA device that all of the tensors (None: not given) lie on, contiguous. The calls
    that serve single steps check placement, types and shapes in few attribute reads each: on
    the host they cost as much as the kernels."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0 or not t.is_contiguous()):
            n = next(n for n, x in zip(names, tensors) if x is t)
            _need_cuda_contig(n, t)
            raise PagedKVError(f"{n} is on {t.device}, not on {tensors[0].device}")
    return dev


def _status_word(status):
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise PagedKVError("device_status must be an int32 tensor")


def _head_rows(name, t, dev, heads, head_size) -> int:
    """Token stride of a [tokens, heads, head_size] tensor whose tokens hold contiguous heads
    (None: any size)."""
    if t.get_device() != dev or dev < 0:
        raise PagedKVError(f"{name} must be a CUDA tensor on the inputs' device")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or \
            (head_size is not None and shape[2] != head_size):
        raise PagedKVError(f"{name} must be [tokens, {heads or 'heads'}, {head_size or 'head_size'}], "
                           f"got {tuple(shape)}")
    T, H, D = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (H > 1 and s1 != D):
        raise PagedKVError(f"the heads of a token of {name} must be contiguous")
    if T <= 1:
        return H * D
    if s0 < H * D or s0 % 8:
        raise PagedKVError(f"the tokens of {name} must be at least a row apart, in multiples of 8 elements")
    return s0


_descs: dict = {}


def _desc_of(k_cache, v_cache, packed=False):
    """A descriptor of the cache pair for the library (kept by its sizes), its KV heads and head size
    (packed: an INT4 cache, two dimensions a byte)."""
    shape = k_cache.shape
    if v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise PagedKVError("k_cache and v_cache must have the same shape and dtype")
    if len(shape) != 4 or shape[2] != BLOCK_SIZE:
        raise PagedKVError(f"cache must be [num_blocks, num_kv_heads, 16, head_size], got {tuple(shape)}")
    nb, hkv, _, d = shape
    if packed:
        d *= 2
        if k_cache.dtype is not torch.uint8:
            raise PagedKVError("an INT4 cache is a torch.uint8 tensor (alloc_kv_cache)")
    ref = _descs.get((nb, hkv, d))
    if ref is None:
        if len(_descs) > 256:
            _descs.clear()
        ref = _descs[(nb, hkv, d)] = ctypes.byref(_CacheDesc(nb, BLOCK_SIZE, hkv, d))
    return ref, hkv, d


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, dev: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


# (With a CUDA tensor at hand the device runtime is up: torch.cuda.current_device without its checks.)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _at(dev: int):
    """The device context of a call: entered only when dev is not the current device."""
    return _NOWHERE if _device() == dev else torch.cuda.device(dev)


def _call(dev: int, fn, *args) -> int:
    """fn(*args) on device dev."""
    if _device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


_NOWHERE = contextlib.nullcontext()


def _addr(t):
    return None if t is None else t.data_ptr()


def _rotary_inputs(T, D, positions, inv_freq, attn_factor):
    """Rotary dimension and bytes of a position, checked."""
    pt = positions.dtype
    if (pt is not torch.int64 and pt is not torch.int32) or positions.shape != (T,):
        raise PagedKVError("positions must be int32 or int64, one per token")
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1:
        raise PagedKVError("inv_freq must be float64 [rotary_dim / 2]")
    if not math.isfinite(attn_factor):
        raise PagedKVError("attn_factor must be finite")
    rd = 2 * inv_freq.shape[0]
    if rd < 16 or rd % 16 or rd > D:
        raise PagedKVError(f"rotary_dim = {rd} must be a multiple of 16, at most the head size {D}")
    return rd, 8 if pt is torch.int64 else 4


def rotary_embed(out, x, positions, inv_freq, *, interleaved: bool = False, attn_factor: float = 1.0,
                 inverse: bool = False, stream=None):
    """Turn the first 2 * len(inv_freq) dimensions of x [T, H, D] (fp16 or bf16) by
    positions[t] * inv_freq[i], pairs (i, i + half) or (2i, 2i + 1), times attn_factor; the rest is
    copied. out may be x. ``inverse`` turns back (the gradient of the forward call)."""
    dev = _placed(("positions", "inv_freq"), (positions, inv_freq))
    xs = _head_rows("x", x, dev, None, None)
    T, H, D = x.shape
    os_ = _head_rows("out", out, dev, H, D)
    if out.shape[0] != T or out.dtype is not x.dtype:
        raise PagedKVError("out must have the shape and dtype of x")
    rd, pb = _rotary_inputs(T, D, positions, inv_freq, attn_factor)
    lib = _lib or load_library()
    with _at(dev):
        rc = lib.pkv_rotary_embed(
            out.data_ptr(), os_, x.data_ptr(), xs, _src_code(x), T, H, D, positions.data_ptr(), pb,
            inv_freq.data_ptr(), rd, 1 if interleaved else 0, attn_factor, 1 if inverse else 0,
            _stream_of(stream, dev))
    if rc:
        _check(rc, "rotary_embed")
    return out


_WRITE_NAMES = ("slot_mapping", "positions", "inv_freq", "k_cache", "v_cache", "scales", "device_status")


def rotary_write(q_out, q, key, value, positions, slot_mapping, k_cache, v_cache, inv_freq, kv_dtype=None, *,
                 interleaved: bool = False, attn_factor: float = 1.0, scales=None, device_status=None, stream=None):
    """A layer's rotary embedding and cache write in one pass: q [T, Hq, D] turned into q_out
    (which may be q), key [T, Hkv, D] turned and written with value to the slots of the cache.
    The inputs may be views of one packed QKV tensor (token strides of any multiple of 8).
    An INT8 cache takes its row scales."""
    dev = _placed(_WRITE_NAMES, (slot_mapping, positions, inv_freq, k_cache, v_cache, scales, device_status))
    desc, Hkv, D = _desc_of(k_cache, v_cache)
    qs = _head_rows("q", q, dev, None, D)
    T, Hq, _ = q.shape
    qos = _head_rows("q_out", q_out, dev, Hq, D)
    ks, vs = _head_rows("key", key, dev, Hkv, D), _head_rows("value", value, dev, Hkv, D)
    if q_out.shape[0] != T or key.shape[0] != T or value.shape[0] != T:
        raise PagedKVError("q, q_out, key and value must hold the same tokens")
    dt = q.dtype
    if q_out.dtype is not dt or key.dtype is not dt or value.dtype is not dt:
        raise PagedKVError("q, q_out, key and value must share a dtype")
    if slot_mapping.dtype is not torch.int32 or slot_mapping.shape != (T,):
        raise PagedKVError("slot_mapping must be int32 with one slot per token")
    rd, pb = _rotary_inputs(T, D, positions, inv_freq, attn_factor)
    code = _kv_code(kv_dtype, k_cache)
    _int8_scales(code, k_cache, scales)
    _status_word(device_status)
    lib = _lib or load_library()
    with _at(dev):
        rc = lib.pkv_rotary_write(
            q_out.data_ptr(), qos, q.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs, _src_code(q), T, Hq,
            positions.data_ptr(), pb, slot_mapping.data_ptr(), inv_freq.data_ptr(), rd, 1 if interleaved else 0,
            attn_factor, k_cache.data_ptr(), v_cache.data_ptr(), _addr(scales), code, desc, _addr(device_status),
            _stream_of(stream, dev))
    if rc:
        _check(rc, "rotary_write")
    return q_out


_prefill_workspaces: dict = {}
_prefill_ws_bytes: dict = {}
_PREFILL_COUNTER_BYTES = 4096   # the start of the workspace, where the split counters are


def _prefill_workspace(nbytes: int, dev: int, stream) -> torch.Tensor:
    """Scratch of a prefill call: one buffer per (device, stream the call runs on), grown as
    needed. A call that is being captured gets a buffer of its own from the graph's memory
    pool (its counters cleared by a captured fill), so two graphs, or a graph and eager calls,
    never share one and a later growth takes nothing away from a captured graph."""
    with _NOWHERE if stream is None else torch.cuda.stream(stream):
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
            ws[:_PREFILL_COUNTER_BYTES].zero_()
            return ws
        key = (dev, _stream_of(stream, dev))
        ws = _prefill_workspaces.get(key)
        if ws is None or ws.shape[0] < nbytes:
            ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
            _prefill_workspaces[key] = ws
        return ws


def prefill_workspace_bytes(num_q_rows: int, num_seqs: int, num_q_heads: int, k_cache) -> int:
    """Bytes of workspace paged_attention_prefill needs for this problem on the cache's device."""
    d = _desc(k_cache)
    with torch.cuda.device(k_cache.device):
        return int(load_library().pkv_prefill_workspace_bytes(int(num_q_rows), int(num_seqs), int(num_q_heads),
                                                              ctypes.byref(d)))


_PREFILL_NAMES = ("q", "out", "cu_q_lens", "k_cache", "v_cache", "block_tables", "context_lens", "scales", "workspace",
                  "device_status")


def paged_attention_prefill(out, q, cu_q_lens, k_cache, v_cache, block_tables, context_lens, scale: float,
                            kv_dtype=None, *, scales=None, workspace=None, device_status=None, stream=None):
    """Causal attention of every sequence's newest tokens over its blocks: whole prompts,
    chunks of a prompt, single decode rows beside them, packed without padding. Sequence s
    owns rows cu_q_lens[s]..cu_q_lens[s+1]-1 of q/out [rows, Hq, D] (int32, on the device; any
    count from 0) and its token j sees positions <= context_lens[s] - n_s + j. An INT8 cache
    takes its row scales."""
    dev = _placed(_PREFILL_NAMES, (q, out, cu_q_lens, k_cache, v_cache, block_tables, context_lens, scales, workspace,
                                   device_status))
    i32 = torch.int32
    if block_tables.dtype is not i32 or context_lens.dtype is not i32 or cu_q_lens.dtype is not i32:
        raise PagedKVError("block_tables, context_lens and cu_q_lens must be int32")
    desc, Hkv, D = _desc_of(k_cache, v_cache)
    shape = q.shape
    if len(shape) != 3 or out.shape != shape or shape[2] != D:
        raise PagedKVError(f"q and out must both be [rows, num_q_heads, {D}], got {tuple(shape)} and "
                           f"{tuple(out.shape)}")
    R, Hq, _ = shape
    if context_lens.dim() != 1:
        raise PagedKVError("context_lens must be 1-D [num_seqs]")
    S = context_lens.shape[0]
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] < S:
        raise PagedKVError(f"block_tables must be [num_seqs, max_blocks_per_seq], got {tuple(tables)}")
    if cu_q_lens.shape != (S + 1,):
        raise PagedKVError("cu_q_lens must have num_seqs + 1 entries")
    code = _kv_code(kv_dtype, k_cache)
    want = torch.bfloat16 if code == KV_BF16 else torch.float16
    if q.dtype is not want or out.dtype is not want:
        raise PagedKVError(f"q and out must be {want} over this cache")
    _int8_scales(code, k_cache, scales)
    _status_word(device_status)
    lib = _lib or load_library()
    with _at(dev):
        if workspace is None:
            # The size goes by the device, the head size and whether a unit may hold over 128 rows.
            key = (dev, D, R * Hq > 128 * Hkv)
            need = _prefill_ws_bytes.get(key)
            if need is None:
                need = int(lib.pkv_prefill_workspace_bytes(R, S, Hq, desc))
                if need:
                    _prefill_ws_bytes[key] = need
            workspace = _prefill_workspace(need, dev, stream)
        rc = lib.pkv_paged_attention_prefill(
            out.data_ptr(), q.data_ptr(), cu_q_lens.data_ptr(), R, S, Hq, k_cache.data_ptr(), v_cache.data_ptr(),
            _addr(scales), code, desc, block_tables.data_ptr(), tables[1], context_lens.data_ptr(), scale,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _addr(device_status),
            _stream_of(stream, dev))
    if rc:
        _check(rc, "paged_attention_prefill")
    return out


_ACCEPT_NAMES = ("k_cache", "v_cache", "block_tables", "context_lens", "accepted", "num_accepted", "new_context_lens",
                 "cu_q_lens", "scales", "device_status")


def kv_cache_accept(k_cache, v_cache, block_tables, context_lens, accepted, num_accepted, new_context_lens,
                    max_q_per_seq: int, kv_dtype=None, *, cu_q_lens=None, scales=None, device_status=None,
                    stream=None):
    """Keep the accepted drafts of a speculative verify: with base = context_lens[s] - n_s, cache
    row base + i of sequence s becomes row base + accepted[s, i] for i < num_accepted[s] (all
    rows read before any is written) and new_context_lens[s] = base + num_accepted[s]. n_s is
    max_q_per_seq, or from cu_q_lens. accepted: int32 [num_seqs, max_accepted]; new_context_lens
    may be None. An INT8 or INT4 cache's scales move along."""
    dev = _placed(_ACCEPT_NAMES, (k_cache, v_cache, block_tables, context_lens, accepted, num_accepted,
                                  new_context_lens, cu_q_lens, scales, device_status))
    for nm, t in (("block_tables", block_tables), ("context_lens", context_lens), ("accepted", accepted),
                  ("num_accepted", num_accepted), ("new_context_lens", new_context_lens), ("cu_q_lens", cu_q_lens)):
        if t is not None and t.dtype is not torch.int32:
            raise PagedKVError(f"{nm} must be int32")
    code = _kv_code(kv_dtype, k_cache)
    desc, _, _ = _desc_of(k_cache, v_cache, code == KV_INT4)
    if context_lens.dim() != 1:
        raise PagedKVError("context_lens must be 1-D [num_seqs]")
    S = context_lens.shape[0]
    tables, acc = block_tables.shape, accepted.shape
    if len(tables) != 2 or tables[0] < S:
        raise PagedKVError(f"block_tables must be [num_seqs, max_blocks_per_seq], got {tuple(tables)}")
    if len(acc) != 2 or acc[0] != S or num_accepted.shape != (S,):
        raise PagedKVError("accepted must be [num_seqs, max_accepted] and num_accepted [num_seqs]")
    if new_context_lens is not None and new_context_lens.shape != (S,):
        raise PagedKVError("new_context_lens must be [num_seqs]")
    if cu_q_lens is not None and cu_q_lens.shape != (S + 1,):
        raise PagedKVError("cu_q_lens must have num_seqs + 1 entries")
    _int8_scales(code, k_cache, scales)
    _status_word(device_status)
    lib = _lib or load_library()
    with _at(dev):
        rc = lib.pkv_kv_cache_accept(
            k_cache.data_ptr(), v_cache.data_ptr(), _addr(scales), code, desc, block_tables.data_ptr(), tables[1],
            context_lens.data_ptr(), _addr(cu_q_lens), S, int(max_q_per_seq), accepted.data_ptr(), acc[1],
            num_accepted.data_ptr(), _addr(new_context_lens), _addr(device_status), _stream_of(stream, dev))
    if rc:
        _check(rc, "kv_cache_accept")
    return new_context_lens


# ------------------------------------------------------------------------------------
# INT4 cache; reading any cache back
# ------------------------------------------------------------------------------------

def _is_int4(kv_dtype) -> bool:
    return kv_dtype == "int4" or (type(kv_dtype) is int and kv_dtype == KV_INT4)


_ROW_NAMES = ("key", "value", "slot_mapping", "k_cache", "v_cache", "scales", "device_status")


def _row_shapes(key, value, slot_mapping, hkv, head) -> int:
    """Tokens of key and value [T, Hkv, D] of one 16-bit type with one slot each."""
    shape = key.shape
    if len(shape) != 3 or shape[1] != hkv or shape[2] != head or value.shape != shape:
        raise PagedKVError(f"key and value must both be [T, {hkv}, {head}], got {tuple(shape)} and "
                           f"{tuple(value.shape)}")
    if value.dtype is not key.dtype:
        raise PagedKVError("key and value must share a dtype")
    if slot_mapping.dtype is not torch.int32 or slot_mapping.shape != shape[:1]:
        raise PagedKVError("slot_mapping must be int32 with one slot per token")
    return shape[0]


def kv_cache_write_int4(key, value, slot_mapping, k_cache, v_cache, scales, *, device_status=None, stream=None):
    """Quantise fp16 or bf16 key/value [T, Hkv, D] into the slots of an INT4 cache (alloc_kv_cache(...,
    "int4"), alloc_kv_scales(..., kv_dtype="int4")). Of every 64 dimensions of a row: z, the largest
    fp16 number not above the least value; s, the smallest one not below (largest - z) / 15; and
    the codes 0..15 whose values z + s c are nearest (halfway: the even one)."""
    dev = _placed(_ROW_NAMES, (key, value, slot_mapping, k_cache, v_cache, scales, device_status))
    desc, hkv, head = _desc_of(k_cache, v_cache, True)
    T = _row_shapes(key, value, slot_mapping, hkv, head)
    _scales_shape(k_cache, scales, KV_INT4)
    _status_word(device_status)
    rc = _call(dev, (_lib or load_library()).pkv_kv_cache_write_int4, key.data_ptr(), value.data_ptr(), _src_code(key), T,
               slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), scales.data_ptr(), desc, _addr(device_status),
               _stream_of(stream, dev))
    if rc:
        _check(rc, "kv_cache_write_int4")


def kv_cache_read(key, value, slot_mapping, k_cache, v_cache, kv_dtype=None, *, scales=None, device_status=None,
                  stream=None):
    """key/value [T, Hkv, D] (fp16 or bf16, written) become the values that rows slot_mapping[t] of a
    cache of any type stand for; the rows of a slot -1 stay as they are. An INT8 or INT4 cache
    takes its scales."""
    dev = _placed(_ROW_NAMES, (key, value, slot_mapping, k_cache, v_cache, scales, device_status))
    code = _kv_code(kv_dtype, k_cache)
    desc, hkv, head = _desc_of(k_cache, v_cache, code == KV_INT4)
    T = _row_shapes(key, value, slot_mapping, hkv, head)
    if scales is None or code not in (KV_INT8, KV_INT4):
        _int8_scales(code, k_cache, scales)
    else:
        _scales_shape(k_cache, scales, code)
    _status_word(device_status)
    rc = _call(dev, (_lib or load_library()).pkv_kv_cache_read, key.data_ptr(), value.data_ptr(), _src_code(key), T,
               slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _addr(scales), code, desc,
               _addr(device_status), _stream_of(stream, dev))
    if rc:
        _check(rc, "kv_cache_read")
    return key, value


_DECODE4_NAMES = ("q", "out", "k_cache", "v_cache", "scales", "block_tables", "context_lens", "cu_q_lens", "tree_masks",
                  "workspace", "device_status")


def _decode_int4(what, out, q, cu_q_lens, tree_masks, k_cache, v_cache, scales, block_tables, context_lens,
                 max_q_per_seq, scale, workspace, device_status, stream):
    if scales is None:
        raise PagedKVError("an INT4 cache is read with its scales (alloc_kv_scales)")
    dev = _placed(_DECODE4_NAMES, (q, out, k_cache, v_cache, scales, block_tables, context_lens, cu_q_lens, tree_masks,
                                   workspace, device_status))
    i32 = torch.int32
    if block_tables.dtype is not i32 or context_lens.dtype is not i32:
        raise PagedKVError("block_tables and context_lens must be int32")
    desc, hkv, D = _desc_of(k_cache, v_cache, True)
    _scales_shape(k_cache, scales, KV_INT4)
    shape = q.shape
    if len(shape) != 3 or out.shape != shape or shape[2] != D:
        raise PagedKVError(f"q and out must both be [rows, num_q_heads, {D}], got {tuple(shape)} and "
                           f"{tuple(out.shape)}")
    if out.dtype is not q.dtype:
        raise PagedKVError("out and q must share a dtype")
    R, Hq, _ = shape
    if context_lens.dim() != 1:
        raise PagedKVError("context_lens must be 1-D [num_seqs]")
    S, n = context_lens.shape[0], int(max_q_per_seq)
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] < S:
        raise PagedKVError(f"block_tables must be [num_seqs, max_blocks_per_seq], got {tuple(tables)}")
    if cu_q_lens is None:
        if R != S * n:
            raise PagedKVError(f"q must have num_seqs * q_per_seq = {S * n} rows, got {R}")
    elif cu_q_lens.dtype is not i32 or cu_q_lens.shape != (S + 1,):
        raise PagedKVError("cu_q_lens must be int32 with num_seqs + 1 entries")
    elif not S <= R <= S * n:
        raise PagedKVError(f"q must have between num_seqs and num_seqs * max_q_per_seq rows, got {R}")
    if tree_masks is not None and (tree_masks.dtype not in (torch.int64, torch.uint64) or tree_masks.shape != (R,)):
        raise PagedKVError("tree_masks must be 64-bit, one mask per query row")
    _status_word(device_status)
    lib = _lib or load_library()
    with _at(dev):
        if workspace is None:
            workspace = _decode_workspace(lib, dev, stream, S, Hq, n, desc, hkv, D, KV_INT4)
        rc = lib.pkv_paged_attention_decode_int4(
            out.data_ptr(), q.data_ptr(), _src_code(q), _addr(cu_q_lens), _addr(tree_masks), R, S, Hq, n,
            k_cache.data_ptr(), v_cache.data_ptr(), scales.data_ptr(), desc, block_tables.data_ptr(), tables[1],
            context_lens.data_ptr(), scale, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _addr(device_status), _stream_of(stream, dev))
    if rc:
        _check(rc, what)
    return out


def paged_attention_decode_int4(out, q, k_cache, v_cache, scales, block_tables, context_lens, q_per_seq: int,
                                scale: float, *, workspace=None, device_status=None, stream=None):
    """paged_attention_decode over an INT4 cache with its scales (q/out fp16 or bf16).
    paged_attention_decode_varlen, _tree and _chunked take one with kv_dtype="int4" and ``scales``."""
    return _decode_int4("paged_attention_decode_int4", out, q, None, None, k_cache, v_cache, scales, block_tables,
                        context_lens, q_per_seq, scale, workspace, device_status, stream)


# ------------------------------------------------------------------------------------
# Block pool (host) and block copy (device)
# ------------------------------------------------------------------------------------

OUT_OF_BLOCKS = -6


class BlockAllocator:
    """Host-side block pool of ``num_blocks`` 16-token blocks (the C allocator in
    libpagedkv.so): sequences, fork with copy-on-write, release, and a prefix
    cache of full blocks. Block ids index the caches' first dimension; the
    caches themselves stay with the caller."""

    def __init__(self, num_blocks: int):
        self._lib = load_library()
        self._h = self._lib.pkv_allocator_create(int(num_blocks))
        if not self._h:
            raise PagedKVError(f"pkv_allocator_create({num_blocks}) failed")
        self.num_blocks = int(num_blocks)

    def close(self):
        if self._h:
            self._lib.pkv_allocator_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def free_blocks(self) -> int:
        return int(self._lib.pkv_allocator_free_blocks(self._h))

    def evictable(self) -> int:
        return int(self._lib.pkv_allocator_evictable(self._h))

    def refcount(self, block: int) -> int:
        return int(self._lib.pkv_allocator_refcount(self._h, int(block)))

    def add(self, seq: int):
        _check(self._lib.pkv_seq_add(self._h, int(seq)), "seq_add")

    def fork(self, parent: int, child: int):
        _check(self._lib.pkv_seq_fork(self._h, int(parent), int(child)), "seq_fork")

    def release(self, seq: int):
        _check(self._lib.pkv_seq_release(self._h, int(seq)), "seq_release")

    def length(self, seq: int) -> int:
        return int(self._lib.pkv_seq_length(self._h, int(seq)))

    def block_table(self, seq: int) -> list:
        n = int(self._lib.pkv_seq_block_table(self._h, int(seq), None, 0))
        if n < 0:
            _check(n, "seq_block_table")
        buf = (ctypes.c_int32 * max(n, 1))()
        self._lib.pkv_seq_block_table(self._h, int(seq), buf, n)
        return [int(buf[i]) for i in range(n)]

    def append(self, seq: int, n: int):
        """Reserve n tokens; returns (slots, copies) with copies a list of
        (src, dst) block pairs to copy before the new tokens are written."""
        slots = (ctypes.c_int32 * max(int(n), 1))()
        src, dst, nc = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        rc = self._lib.pkv_seq_append(self._h, int(seq), int(n), slots, ctypes.byref(src),
                                      ctypes.byref(dst), ctypes.byref(nc))
        _check(rc, "seq_append")
        copies = [(int(src.value), int(dst.value))] if nc.value else []
        return [int(slots[i]) for i in range(int(n))], copies

    def truncate(self, seq: int, length: int):
        """Shorten the sequence to its first ``length`` tokens; blocks that hold none of
        them lose one reference each."""
        _check(self._lib.pkv_seq_truncate(self._h, int(seq), int(length)), "seq_truncate")

    def prefix_insert(self, seq: int, tokens) -> int:
        arr = (ctypes.c_int32 * max(len(tokens), 1))(*[int(t) for t in tokens])
        rc = int(self._lib.pkv_prefix_insert(self._h, int(seq), arr, len(tokens)))
        if rc < 0:
            _check(rc, "prefix_insert")
        return rc

    def add_cached(self, seq: int, tokens) -> int:
        """New sequence starting from the longest cached prefix of ``tokens``
        (whole blocks); returns the number of tokens it already holds."""
        arr = (ctypes.c_int32 * max(len(tokens), 1))(*[int(t) for t in tokens])
        got = ctypes.c_int32()
        _check(self._lib.pkv_seq_add_cached(self._h, int(seq), arr, len(tokens), ctypes.byref(got)),
               "seq_add_cached")
        return int(got.value)


def copy_blocks(k_cache, v_cache, src, dst, kv_dtype=None, *, scales=None, device_status=None, stream=None):
    """Physical block dst[i] of both caches becomes a copy of block src[i]
    (int32 device tensors of equal length); an INT8 or INT4 cache's scales
    (``scales``, from alloc_kv_scales) are copied with its blocks."""
    for n_, t in (("k_cache", k_cache), ("v_cache", v_cache), ("src", src), ("dst", dst)):
        _need_cuda_contig(n_, t)
    if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.numel() != dst.numel():
        raise PagedKVError("src and dst must be int32 tensors of equal length")
    code = _kv_code(kv_dtype, k_cache)
    d = _pair(k_cache, v_cache, code == KV_INT4)
    if (code in (KV_INT8, KV_INT4)) != (scales is not None):
        raise PagedKVError("an INT8 or INT4 cache is copied with its scales; other caches take none")
    if scales is not None:
        _need_cuda_contig("scales", scales)
        _scales_shape(k_cache, scales, code)
    rc = load_library().pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(scales), code,
                                        ctypes.byref(d), _ptr(src), _ptr(dst), int(src.numel()),
                                        _ptr(device_status), _stream_handle(stream, k_cache.device))
    _check(rc, "copy_blocks")
