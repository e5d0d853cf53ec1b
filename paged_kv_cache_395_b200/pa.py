"""Python binding of ``libpa.so`` (ctypes; argument marshalling only).

The names mirror the C ABI in ``include/pa.h``:

* ``pa_reshape_and_cache``, ``pa_decode``, ``pa_decode_append``,
  ``pa_decode_append_fused``, ``pa_decode_fixed_scratch``,
  ``pa_decode_stall_selftest``, ``pa_block_copy``, ``pa_quantize_int8``,
  ``pa_quantize_int4``, ``pa_append_int8``, ``pa_step_tables``,
  ``pa_block_bounds``, ``pa_select_blocks``, ``pa_decode_selected``, ``pa_decode_sparse``,
  ``pa_decode_selected_stall_selftest``, ``pa_decode_workspace_size``,
  ``pa_decode_algo``, ``pa_get_error_flags`` take torch CUDA tensors (or raw device pointers via ``lib``), check device,
  dtype and contiguity, and call the library on
  ``torch.cuda.current_stream()``.  Every step of the computation runs in the
  library's kernels; there is no fallback of any kind.  If ``libpa.so`` is
  missing, importing this module raises ImportError.

PyTorch is used only for device memory, streams and ``data_ptr()``.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK, PA_ERR_NULL, PA_ERR_SHAPE, PA_ERR_DTYPE = 0, -1, -2, -3
PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA, PA_ERR_ALIGN = -4, -5, -6, -7
PA_F32, PA_F16, PA_BF16, PA_I8, PA_I4 = 0, 1, 2, 3, 4
PA_ALGO_AUTO, PA_ALGO_SIMT, PA_ALGO_TENSOR, PA_ALGO_TCGEN05 = 0, 1, 2, 3
PA_EFLAG_BAD_BLOCK, PA_EFLAG_BAD_SLOT, PA_EFLAG_BAD_PAIR, PA_EFLAG_WAIT_TIMEOUT = 1, 2, 4, 8
PA_EFLAG_APPEND_SLOT = 16
PA_EFLAG_OUT_OF_BLOCKS, PA_EFLAG_BAD_LENGTH, PA_EFLAG_FREE_LIST = 32, 64, 128
PA_SEQ_FINISHED, PA_STEP_MAX_SEQS, PA_SPARSE_MAX_SEQ_LEN = -1, 8192, 524288
PA_DECODE_INPUTS_READY, PA_DECODE_OUT_F32 = 1, 2
PA_APPEND_OVERLAP_PREVIOUS = 1
BLOCK_SIZE = 16

# a uint8 cache tensor [N][H_kv][16][d/2] holds 4-bit values, two per byte
_TORCH_DTYPE = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16,
                torch.int8: PA_I8, torch.uint8: PA_I4}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m paged_kv_cache_395_b200.build` (no fallback exists)")


class PaDecodeParams(ctypes.Structure):
    """Mirror of ``pa_decode_params``."""
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("block_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("num_blocks", ctypes.c_int64),
        ("max_seq_len", ctypes.c_int),
        ("q_dtype", ctypes.c_int),
        ("kv_dtype", ctypes.c_int),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("partition_size", ctypes.c_int),
        ("algo", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("flags", ctypes.c_int),
        ("query_len", ctypes.c_int),
    ]


class PaSparseParams(ctypes.Structure):
    """Mirror of ``pa_sparse_params``."""
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("block_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("num_blocks", ctypes.c_int64),
        ("max_seq_len", ctypes.c_int),
        ("q_dtype", ctypes.c_int),
        ("kv_dtype", ctypes.c_int),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("query_len", ctypes.c_int),
        ("max_selected", ctypes.c_int),
        ("sink_blocks", ctypes.c_int),
        ("recent_blocks", ctypes.c_int),
        ("flags", ctypes.c_int),
    ]


def _load():
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    L.pa_reshape_and_cache.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i64, i32, i64, i64, P]
    L.pa_reshape_and_cache_ex.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i64, i32, i64, i64, i32, P]
    L.pa_decode.argtypes = [P, P, P, P, P, P, f32, ctypes.POINTER(PaDecodeParams), P]
    L.pa_decode_fixed_scratch.argtypes = [P, P, P, P, P, P, f32, ctypes.POINTER(PaDecodeParams), P]
    L.pa_decode_append.argtypes = [P, P, P, P, P, i64, i64, P, P, P, P, f32, ctypes.POINTER(PaDecodeParams), P]
    L.pa_decode_append_fused.argtypes = [ctypes.POINTER(PaDecodeParams), P, P, P, i64, i64]
    L.pa_decode_workspace_size.argtypes = [ctypes.POINTER(PaDecodeParams)]
    L.pa_decode_workspace_size.restype = ctypes.c_size_t
    L.pa_decode_algo.argtypes = [ctypes.POINTER(PaDecodeParams), P]
    L.pa_decode_launches.argtypes = [ctypes.POINTER(PaDecodeParams), P]
    L.pa_decode_stall_selftest.argtypes = [P, P, P, P, P, P, f32, ctypes.POINTER(PaDecodeParams), i32,
                                           ctypes.c_uint64, P]
    L.pa_block_copy.argtypes = [P, P, P, P, P, i64, i32, i32, i32, i64, i32, P]
    L.pa_quantize_int8.argtypes = [P, i32, P, P, i64, i32, i32, i32, P]
    L.pa_append_int8.argtypes = [P, P, i32, P, P, P, P, P, i64, i32, i32, i32, i64, i64, i64, P]
    L.pa_quantize_int4.argtypes = [P, i32, P, P, i64, i32, i32, i32, P]
    L.pa_step_tables.argtypes = [P] * 11 + [i32, i32, i64, i64, i32, P]
    L.pa_block_bounds.argtypes = [P] * 7 + [i32] * 5 + [i64, i64, i32, P]
    # pa_sparse_params as packed bytes, or a pointer to PaSparseParams
    L.pa_select_blocks.argtypes = [P] * 9
    L.pa_decode_selected.argtypes = [P] * 8 + [f32, P, P]
    L.pa_decode_selected_stall_selftest.argtypes = [P] * 8 + [f32, P, i32, ctypes.c_uint64, P]
    L.pa_decode_sparse.argtypes = [P] * 10 + [f32, P, P]
    L.pa_get_error_flags.argtypes = [ctypes.POINTER(ctypes.c_uint), i32, P]
    L.pa_status_string.argtypes = [i32]
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_version.argtypes = []
    for n in ("pa_reshape_and_cache", "pa_reshape_and_cache_ex", "pa_append_int8", "pa_decode", "pa_decode_append",
              "pa_decode_append_fused", "pa_decode_fixed_scratch",
              "pa_decode_stall_selftest", "pa_decode_algo", "pa_decode_launches", "pa_block_copy",
              "pa_quantize_int8", "pa_quantize_int4", "pa_step_tables", "pa_block_bounds", "pa_select_blocks",
              "pa_decode_selected", "pa_decode_selected_stall_selftest", "pa_decode_sparse", "pa_get_error_flags",
              "pa_version"):
        getattr(L, n).restype = i32
    return L


lib = _load()

# the C-ABI symbols include/pa.h declares
EXPORTED = ("pa_reshape_and_cache", "pa_reshape_and_cache_ex", "pa_append_int8", "pa_decode_workspace_size",
            "pa_decode_algo", "pa_decode_launches", "pa_decode", "pa_decode_append", "pa_decode_append_fused",
            "pa_decode_fixed_scratch", "pa_decode_stall_selftest", "pa_block_copy", "pa_quantize_int8",
            "pa_quantize_int4", "pa_step_tables", "pa_block_bounds", "pa_select_blocks", "pa_decode_selected",
            "pa_decode_selected_stall_selftest", "pa_decode_sparse", "pa_get_error_flags", "pa_status_string",
            "pa_version")
FIXED_SCRATCH_BYTES = 32 << 20  # PA_FIXED_SCRATCH_BYTES


class PaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib.pa_status_string(status).decode()} ({status})")
        self.status = status


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PaError(status, what)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")


def dtype_code(dt: torch.dtype) -> int:
    return _TORCH_DTYPE[dt]


def pa_reshape_and_cache(k, v, key_cache, value_cache, slot_mapping, stream=None, flags=0):
    """k, v [T][H_kv][d] (rows contiguous; token stride free) -> caches [N][H_kv][16][d].
    flags: 0 or PA_APPEND_OVERLAP_PREVIOUS (see include/pa.h)."""
    _dev(k, v, key_cache, value_cache, slot_mapping)
    T, H, d = k.shape
    N = key_cache.shape[0]
    if k.stride(2) != 1 or k.stride(1) != d or v.stride(2) != 1 or v.stride(1) != d:
        raise ValueError("k/v heads must be contiguous rows of head_dim elements")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64")
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    _check(lib.pa_reshape_and_cache_ex(_ptr(k), _ptr(v), _ptr(key_cache), _ptr(value_cache),
                                       _ptr(slot_mapping), T, H, d, key_cache.shape[2], N,
                                       dtype_code(k.dtype), k.stride(0), v.stride(0), int(flags),
                                       _stream(stream)),
           "pa_reshape_and_cache")


def make_params(q, key_cache, block_tables, max_seq_len, k_scales=None, v_scales=None,
                partition_size=0, workspace=None, algo=PA_ALGO_AUTO, flags=0) -> PaDecodeParams:
    """q is [B][H_q][d], or [B][Q][H_q][d] for Q new tokens per sequence."""
    if q.dim() == 4:
        B, Q, Hq, d = q.shape
    else:
        (B, Hq, d), Q = q.shape, 1
    N, Hkv, bs, _ = key_cache.shape
    p = PaDecodeParams()
    p.num_seqs, p.num_q_heads, p.num_kv_heads, p.head_dim, p.block_size = B, Hq, Hkv, d, bs
    p.max_blocks_per_seq = block_tables.shape[1] if block_tables.dim() == 2 else 1
    p.num_blocks = N
    p.max_seq_len = int(max_seq_len)
    p.q_dtype = dtype_code(q.dtype)
    p.kv_dtype = dtype_code(key_cache.dtype)
    p.k_scales = None if k_scales is None else k_scales.data_ptr()
    p.v_scales = None if v_scales is None else v_scales.data_ptr()
    p.partition_size = int(partition_size)
    p.algo = int(algo)
    p.workspace = None if workspace is None else workspace.data_ptr()
    p.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    p.flags = int(flags)
    p.query_len = int(Q)
    return p


def pa_decode_algo(q, key_cache, block_tables, max_seq_len, partition_size=0, k_scales=None,
                   v_scales=None, algo=PA_ALGO_AUTO) -> int:
    """The kernel family pa_decode runs for these operands, as the library
    reports it: PA_ALGO_TENSOR, PA_ALGO_SIMT or PA_ALGO_TCGEN05."""
    p = make_params(q, key_cache, block_tables, max_seq_len, k_scales, v_scales, partition_size,
                    None, algo)
    r = int(lib.pa_decode_algo(ctypes.byref(p), _ptr(q)))
    _check(min(r, 0), "pa_decode_algo")
    return r


def pa_decode_launches(q, key_cache, block_tables, max_seq_len, partition_size=0, k_scales=None,
                       v_scales=None, algo=PA_ALGO_AUTO) -> int:
    """Kernel launches of one pa_decode call with these operands (1 or 2), as the
    library reports it."""
    p = make_params(q, key_cache, block_tables, max_seq_len, k_scales, v_scales, partition_size,
                    None, algo)
    r = int(lib.pa_decode_launches(ctypes.byref(p), _ptr(q)))
    _check(min(r, 0), "pa_decode_launches")
    return r


def pa_decode_workspace_size(q, key_cache, block_tables, max_seq_len, partition_size=0,
                             k_scales=None, v_scales=None, algo=PA_ALGO_AUTO) -> int:
    p = make_params(q, key_cache, block_tables, max_seq_len, k_scales, v_scales, partition_size,
                    None, algo)
    return int(lib.pa_decode_workspace_size(ctypes.byref(p)))


def alloc_workspace(nbytes: int, device) -> torch.Tensor | None:
    """Split-K workspace (left uninitialised: pa_decode needs none)."""
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _out_flag(out, q) -> int:
    """out matches q in shape, and in dtype or is fp32 (PA_DECODE_OUT_F32)."""
    if out.shape != q.shape or out.dtype not in (q.dtype, torch.float32):
        raise ValueError("out must match q in shape, and in dtype or be float32")
    return PA_DECODE_OUT_F32 if out.dtype != q.dtype else 0


def pa_decode(out, q, key_cache, value_cache, block_tables, seq_lens, scale, max_seq_len,
              k_scales=None, v_scales=None, partition_size=0, workspace=None,
              algo=PA_ALGO_AUTO, stream=None, params=None, flags=0):
    """out, q [B][H_q][d] (or [B][Q][H_q][d]: Q new tokens per sequence, causal
    among them); caches [N][H_kv][16][d]; block_tables int32 [B][M]; seq_lens int32
    [B] (including the new tokens).  flags: 0 or PA_DECODE_INPUTS_READY (see
    include/pa.h).  A float32 out of an fp16/bf16 q receives the fp32 result
    before its rounding (PA_DECODE_OUT_F32 is added)."""
    _dev(out, q, key_cache, value_cache, block_tables, seq_lens, k_scales, v_scales, workspace)
    for t, n in ((out, "out"), (q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    flags |= _out_flag(out, q)
    p = params if params is not None else make_params(
        q, key_cache, block_tables, max_seq_len, k_scales, v_scales, partition_size, workspace, algo,
        flags)
    _check(lib.pa_decode(_ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache),
                         _ptr(block_tables), _ptr(seq_lens), ctypes.c_float(scale),
                         ctypes.byref(p), _stream(stream)), "pa_decode")


def _new_rows(k_new, v_new, slot_mapping, key_cache):
    """k_new / v_new [B][H_kv][d] (token stride free, heads contiguous rows), int64 slots [B]."""
    _, H, _, d = key_cache.shape
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        if t.dim() != 3 or t.shape[1:] != (H, d) or t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError(f"{n} must be [B][H_kv][d] with contiguous head rows")
        if t.dtype != key_cache.dtype:
            raise ValueError(f"{n} must have the cache's dtype")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64")


def pa_decode_append(out, q, k_new, v_new, slot_mapping, key_cache, value_cache, block_tables, seq_lens,
                     scale, max_seq_len, partition_size=0, workspace=None, algo=PA_ALGO_AUTO, stream=None,
                     flags=0):
    """pa_reshape_and_cache of one new token per sequence (k_new / v_new row b,
    slot_mapping[b]) then pa_decode, as one kernel where pa_decode_append_fused
    says so (include/pa.h).  seq_lens count the new token."""
    _dev(out, q, k_new, v_new, slot_mapping, key_cache, value_cache, block_tables, seq_lens, workspace)
    for t, n in ((out, "out"), (q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    _new_rows(k_new, v_new, slot_mapping, key_cache)
    if k_new.shape[0] != q.shape[0] or slot_mapping.numel() != q.shape[0]:
        raise ValueError("one new token per sequence")
    flags |= _out_flag(out, q)
    p = make_params(q, key_cache, block_tables, max_seq_len, None, None, partition_size, workspace, algo,
                    flags)
    _check(lib.pa_decode_append(_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                k_new.stride(0), v_new.stride(0), _ptr(key_cache), _ptr(value_cache),
                                _ptr(block_tables), _ptr(seq_lens), ctypes.c_float(scale), ctypes.byref(p),
                                _stream(stream)), "pa_decode_append")


def pa_decode_append_fused(q, k_new, v_new, key_cache, block_tables, max_seq_len, partition_size=0,
                           algo=PA_ALGO_AUTO) -> bool:
    """Whether pa_decode_append with these operands runs as one kernel."""
    p = make_params(q, key_cache, block_tables, max_seq_len, None, None, partition_size, None, algo)
    r = int(lib.pa_decode_append_fused(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new),
                                       k_new.stride(0), v_new.stride(0)))
    _check(min(r, 0), "pa_decode_append_fused")
    return r == 1


def pa_decode_fixed_scratch(out, q, key_cache, value_cache, block_tables, seq_lens, scale,
                            max_seq_len, k_scales=None, v_scales=None, partition_size=-1,
                            algo=PA_ALGO_AUTO, stream=None):
    """pa_decode for callers that cannot allocate a workspace: the split-K
    scratch is the fixed area compiled into the library (FIXED_SCRATCH_BYTES per
    device).  Calls on one device must not overlap; the first call on a device
    looks up the area's address and should come before any stream capture."""
    _dev(out, q, key_cache, value_cache, block_tables, seq_lens, k_scales, v_scales)
    for t, n in ((out, "out"), (q, "q"), (key_cache, "key_cache"), (value_cache, "value_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    p = make_params(q, key_cache, block_tables, max_seq_len, k_scales, v_scales, partition_size,
                    None, algo, _out_flag(out, q))
    _check(lib.pa_decode_fixed_scratch(_ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache),
                                       _ptr(block_tables), _ptr(seq_lens), ctypes.c_float(scale),
                                       ctypes.byref(p), _stream(stream)), "pa_decode_fixed_scratch")


def pa_decode_stall_selftest(out, q, key_cache, value_cache, block_tables, seq_lens, scale, max_seq_len,
                             stall_at, limit_ns, partition_size=-1, workspace=None, stream=None,
                             algo=PA_ALGO_TENSOR):
    """pa_decode on the tensor-core family (algo PA_ALGO_TENSOR or PA_ALGO_TCGEN05)
    with the failure path exercised: the first worker leaves its stall_at-th copy
    unissued, so its bounded wait runs out after limit_ns (see include/pa.h).
    Returns after the launch; the error word then holds PA_EFLAG_WAIT_TIMEOUT."""
    _dev(out, q, key_cache, value_cache, block_tables, seq_lens, workspace)
    p = make_params(q, key_cache, block_tables, max_seq_len, None, None, partition_size, workspace,
                    algo, _out_flag(out, q))
    _check(lib.pa_decode_stall_selftest(_ptr(out), _ptr(q), _ptr(key_cache), _ptr(value_cache),
                                        _ptr(block_tables), _ptr(seq_lens), ctypes.c_float(scale),
                                        ctypes.byref(p), int(stall_at), int(limit_ns), _stream(stream)),
           "pa_decode_stall_selftest")


def pa_block_copy(key_cache, value_cache, pairs, k_scales=None, v_scales=None, stream=None):
    """pairs int64 [n][2] (src, dst) on the device.  A uint8 (4-bit) cache
    [N][H_kv][16][d/2] is copied as such."""
    _dev(key_cache, value_cache, pairs, k_scales, v_scales)
    N, H, bs, d = key_cache.shape
    if key_cache.dtype == torch.uint8:
        d *= 2  # head_dim of a 4-bit cache
    if pairs.dtype != torch.int64 or not pairs.is_contiguous():
        raise ValueError("pairs must be contiguous int64")
    n = pairs.numel() // 2
    _check(lib.pa_block_copy(_ptr(key_cache), _ptr(value_cache), _ptr(k_scales), _ptr(v_scales),
                             _ptr(pairs), n, H, d, bs, N, dtype_code(key_cache.dtype),
                             _stream(stream)), "pa_block_copy")


def pa_quantize_int8(src_cache, dst_cache, scales, stream=None):
    """src [N][H_kv][16][d] fp32/fp16/bf16 -> dst int8 (same shape), scales fp32 [N][H_kv]."""
    _dev(src_cache, dst_cache, scales)
    N, H, bs, d = src_cache.shape
    if dst_cache.dtype != torch.int8 or scales.dtype != torch.float32:
        raise ValueError("dst must be int8 and scales float32")
    _check(lib.pa_quantize_int8(_ptr(src_cache), dtype_code(src_cache.dtype), _ptr(dst_cache),
                                _ptr(scales), N, H, d, bs, _stream(stream)), "pa_quantize_int8")


def pa_append_int8(k, v, key_cache, value_cache, k_scales, v_scales, slot_mapping, stream=None):
    """Append tokens k, v ([T][H_kv][d] fp32/fp16/bf16, rows contiguous) into int8
    caches [N][H_kv][16][d] with fp32 scales [N][H_kv], raising a tile's scale and
    re-rounding its other codes when a token needs it.  The tokens of one call must
    fall in distinct blocks (see include/pa.h)."""
    _dev(k, v, key_cache, value_cache, k_scales, v_scales, slot_mapping)
    T, H, d = k.shape
    N = key_cache.shape[0]
    if k.stride(2) != 1 or k.stride(1) != d or v.stride(2) != 1 or v.stride(1) != d or v.shape != k.shape:
        raise ValueError("k/v heads must be contiguous rows of head_dim elements")
    if k.dtype != v.dtype:
        raise ValueError("k and v must share a dtype")
    if key_cache.dtype != torch.int8 or value_cache.dtype != torch.int8:
        raise ValueError("caches must be int8")
    if k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32:
        raise ValueError("scales must be float32")
    if tuple(key_cache.shape) != (N, H, 16, d) or value_cache.shape != key_cache.shape or \
            tuple(k_scales.shape) != (N, H) or v_scales.shape != k_scales.shape:
        raise ValueError("caches must be [N][H_kv][16][d] and scales [N][H_kv]")
    for t in (key_cache, value_cache, k_scales, v_scales):
        if not t.is_contiguous():
            raise ValueError("caches and scales must be contiguous")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous int64")
    _check(lib.pa_append_int8(_ptr(k), _ptr(v), dtype_code(k.dtype), _ptr(key_cache), _ptr(value_cache),
                              _ptr(k_scales), _ptr(v_scales), _ptr(slot_mapping), T, H, d, 16, N,
                              k.stride(0), v.stride(0), _stream(stream)), "pa_append_int8")


def pa_quantize_int4(src_cache, dst_cache, scales, stream=None):
    """src [N][H_kv][16][d] fp32/fp16/bf16 -> dst uint8 [N][H_kv][16][d/2] (4-bit
    values q + 8, element 2k in the low half of byte k), scales fp32 [N][H_kv]."""
    _dev(src_cache, dst_cache, scales)
    N, H, bs, d = src_cache.shape
    if dst_cache.dtype != torch.uint8 or tuple(dst_cache.shape) != (N, H, bs, d // 2):
        raise ValueError("dst must be uint8 [N][H_kv][16][d/2]")
    if scales.dtype != torch.float32:
        raise ValueError("scales must be float32")
    _check(lib.pa_quantize_int4(_ptr(src_cache), dtype_code(src_cache.dtype), _ptr(dst_cache),
                                _ptr(scales), N, H, d, bs, _stream(stream)), "pa_quantize_int4")


# The calls below run once per layer of a decode step, so their checks are written to be
# cheap: one expression over a call's tensors, and only when it fails the search for the
# message.
_I32, _I64, _F32, _I8 = torch.int32, torch.int64, torch.float32, torch.int8
_get_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_SPARSE_PARAMS = struct.Struct("@6iq3iPP5i4x")  # pa_sparse_params
assert _SPARSE_PARAMS.size == ctypes.sizeof(PaSparseParams)


def _refuse(tensors, rules):
    """Raises the ValueError of the first thing that is wrong: devices, then rules
    (broken, message)."""
    devs = [t.get_device() for t in tensors if t is not None]
    if -1 in devs:
        raise ValueError("all tensors must be CUDA tensors")
    if any(d != _get_device() for d in devs):
        raise ValueError("all tensors must be on the current device")
    for broken, message in rules:
        if broken:
            raise ValueError(message)
    raise ValueError("invalid arguments")


def _on(dev, *ts):
    """Whether the optional tensors ts are absent or on device dev and contiguous."""
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            return False
    return True


def pa_step_tables(block_tables, seq_lens, new_lens, free_blocks, free_count, slot_mapping, seq_lens_out=None,
                   free_count_out=None, positions=None, row_starts=None, refcounts=None, stream=None):
    """One step's block tables, slots, positions and lengths from the sequences'
    lengths (see include/pa.h).  block_tables int32 [B][M] (updated in place);
    seq_lens, new_lens int32 [B] (new_lens PA_SEQ_FINISHED: the sequence ended);
    free_blocks int32 [N], a stack of the pool's N blocks of which the first
    free_count (int32 [1]) are unused (updated in place); slot_mapping int64 [T],
    filled, with -1 past the step's tokens; positions int32 [T]; row_starts int32
    [B + 1]; refcounts int32 [N] (updated in place).  Without seq_lens_out /
    free_count_out the inputs are updated in place."""
    lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    count_out = free_count if free_count_out is None else free_count_out
    B, M = block_tables.shape
    N, T = free_blocks.numel(), slot_mapping.numel()
    dev = block_tables.get_device()
    good = (dev >= 0 and dev == _get_device() and slot_mapping.dtype is _I64 and
            block_tables.dtype is seq_lens.dtype is new_lens.dtype is free_blocks.dtype is free_count.dtype is _I32 and
            seq_lens.numel() == new_lens.numel() == B and free_count.numel() == 1 and
            seq_lens.get_device() == new_lens.get_device() == free_blocks.get_device() == free_count.get_device() ==
            slot_mapping.get_device() == dev and block_tables.is_contiguous() and seq_lens.is_contiguous() and
            new_lens.is_contiguous() and free_blocks.is_contiguous() and slot_mapping.is_contiguous())
    for t, n in ((seq_lens_out, B), (free_count_out, 1), (positions, T), (row_starts, B + 1), (refcounts, N)):
        if t is not None and (t.numel() != n or t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous()):
            good = False
    if not good:
        ints = dict(block_tables=(block_tables, B * M), seq_lens=(seq_lens, B), new_lens=(new_lens, B),
                    seq_lens_out=(lens_out, B), free_blocks=(free_blocks, N), free_count=(free_count, 1),
                    free_count_out=(count_out, 1), positions=(positions, T), row_starts=(row_starts, B + 1),
                    refcounts=(refcounts, N))
        _refuse([t for t, _ in ints.values()] + [slot_mapping],
                [(t is not None and (t.dtype != _I32 or t.numel() != n or not t.is_contiguous()),
                  f"{name} must be contiguous int32 with {n} elements") for name, (t, n) in ints.items()] +
                [(True, "slot_mapping must be contiguous int64")])
    rc = lib.pa_step_tables(
        block_tables.data_ptr(), seq_lens.data_ptr(), new_lens.data_ptr(), lens_out.data_ptr(), free_blocks.data_ptr(),
        free_count.data_ptr(), count_out.data_ptr(), None if refcounts is None else refcounts.data_ptr(),
        slot_mapping.data_ptr(), None if positions is None else positions.data_ptr(),
        None if row_starts is None else row_starts.data_ptr(), B, M, N, T, BLOCK_SIZE,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "pa_step_tables")


def _box_rules(bounds, bound_scales, N, H, d):
    return [(bounds.dtype != _I8 or tuple(bounds.shape) != (N, H, 2, d) or not bounds.is_contiguous(),
             "bounds must be contiguous int8 [N][H_kv][2][d]"),
            (bound_scales.dtype != _F32 or tuple(bound_scales.shape) != (N, H) or not bound_scales.is_contiguous(),
             "bound_scales must be contiguous float32 [N][H_kv]")]


def pa_block_bounds(bounds, bound_scales, key_cache, block_tables, seq_lens, max_new_tokens, first_lens=None,
                    k_scales=None, stream=None):
    """Boxes of the blocks that filled up: for each sequence the full blocks between
    first_lens (int32 [B], tokens whose blocks have their boxes; None: 0) and seq_lens,
    at most ceil(max_new_tokens / 16) of them (see include/pa.h).  bounds int8
    [N][H_kv][2][d], bound_scales fp32 [N][H_kv] (updated in place); key_cache
    [N][H_kv][16][d] fp32/fp16/bf16, or int8 with k_scales [N][H_kv]."""
    N, H, bs, d = key_cache.shape
    B, M = block_tables.shape
    dev = key_cache.get_device()
    if not (dev >= 0 and dev == _get_device() and key_cache.is_contiguous() and bounds.dtype is _I8 and
            bounds.shape == (N, H, 2, d) and bound_scales.dtype is _F32 and bound_scales.shape == (N, H) and
            block_tables.dtype is _I32 and seq_lens.dtype is _I32 and seq_lens.numel() == B and
            (first_lens is None or (first_lens.dtype is _I32 and first_lens.numel() == B)) and
            (k_scales is None or (k_scales.dtype is _F32 and k_scales.shape == (N, H))) and
            _on(dev, bounds, bound_scales, block_tables, seq_lens, first_lens, k_scales)):
        _refuse([bounds, bound_scales, key_cache, block_tables, seq_lens, first_lens, k_scales],
                _box_rules(bounds, bound_scales, N, H, d) +
                [(not key_cache.is_contiguous(), "key_cache must be contiguous"),
                 (block_tables.dtype != _I32 or not block_tables.is_contiguous(), "block_tables must be contiguous int32")] +
                [(t is not None and (t.dtype != _I32 or t.numel() != B or not t.is_contiguous()),
                  f"{name} must be contiguous int32 with {B} elements")
                 for t, name in ((seq_lens, "seq_lens"), (first_lens, "first_lens"))] +
                [(True, "k_scales must be contiguous float32 [N][H_kv]")])
    rc = lib.pa_block_bounds(
        bounds.data_ptr(), bound_scales.data_ptr(), key_cache.data_ptr(), None if k_scales is None else k_scales.data_ptr(),
        block_tables.data_ptr(), None if first_lens is None else first_lens.data_ptr(), seq_lens.data_ptr(), B, H, d, bs,
        M, N, max_new_tokens, _TORCH_DTYPE[key_cache.dtype], _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "pa_block_bounds")


def _list_rules(q, H, block_tables, seq_lens, selected, num_selected):
    lead = q.shape[:-2]
    return [(q.dim() not in (3, 4), "q must be [B][H_q][d] or [B][Q][H_q][d]"),
            (tuple(selected.shape[:-1]) != lead + (H,) or tuple(num_selected.shape) != lead + (H,),
             "selected must be q's leading sizes, then [H_kv][K], and num_selected the same without K"),
            (block_tables.dim() != 2 or block_tables.shape[0] != q.shape[0] or seq_lens.numel() != q.shape[0],
             "block_tables must be [B][M] and seq_lens [B]"),
            (any(t.dtype != _I32 for t in (selected, num_selected, block_tables, seq_lens)),
             "selected, num_selected, block_tables and seq_lens must be int32")] + \
        [(not t.is_contiguous(), f"{name} must be contiguous")
         for t, name in ((q, "q"), (selected, "selected"), (num_selected, "num_selected"),
                         (block_tables, "block_tables"), (seq_lens, "seq_lens"))]


def _lists_good(q, shape, H, dev, block_tables, seq_lens, selected, num_selected):
    """What the block-sparse calls ask of q (of that shape), the lists, tables and lengths."""
    if dev < 0 or dev != _get_device():
        return False
    n, listed, B = len(shape), selected.shape, shape[0]
    if n == 3:
        if len(listed) != 3 or listed[0] != B or listed[1] != H or num_selected.shape != (B, H):
            return False
    elif n != 4 or len(listed) != 4 or listed[:3] != (B, shape[1], H) or num_selected.shape != (B, shape[1], H):
        return False
    t = block_tables.shape
    return (len(t) == 2 and t[0] == B and seq_lens.numel() == B and
            selected.dtype is _I32 and num_selected.dtype is _I32 and block_tables.dtype is _I32 and
            seq_lens.dtype is _I32 and q.is_contiguous() and selected.is_contiguous() and
            num_selected.is_contiguous() and block_tables.is_contiguous() and seq_lens.is_contiguous() and
            selected.get_device() == num_selected.get_device() == block_tables.get_device() ==
            seq_lens.get_device() == dev)


def pa_select_blocks(selected, num_selected, q, bounds, bound_scales, block_tables, seq_lens, max_seq_len,
                     sink_blocks=1, recent_blocks=2, stream=None):
    """The blocks that each query row and KV head attends to (see include/pa.h):
    selected int32 [B][H_kv][K] (or [B][Q][H_kv][K]), filled with logical blocks,
    ascending, then -1; num_selected int32 without the K.  q [B][H_q][d] or
    [B][Q][H_q][d]; bounds, bound_scales as pa_block_bounds leaves them."""
    shape, dev = q.shape, q.get_device()
    N, H = bound_scales.shape
    d = shape[-1]
    if not (_lists_good(q, shape, H, dev, block_tables, seq_lens, selected, num_selected) and bounds.dtype is _I8 and
            bounds.shape == (N, H, 2, d) and bound_scales.dtype is _F32 and _on(dev, bounds, bound_scales)):
        _refuse([selected, num_selected, q, bounds, bound_scales, block_tables, seq_lens],
                _list_rules(q, H, block_tables, seq_lens, selected, num_selected) +
                _box_rules(bounds, bound_scales, N, H, d))
    dt = _TORCH_DTYPE[q.dtype]
    p = _SPARSE_PARAMS.pack(shape[0], shape[-2], H, d, BLOCK_SIZE, block_tables.shape[1], N, max_seq_len, dt, dt, 0, 0,
                            shape[1] if len(shape) == 4 else 1, selected.shape[-1], sink_blocks, recent_blocks, 0)
    rc = lib.pa_select_blocks(selected.data_ptr(), num_selected.data_ptr(), q.data_ptr(), bounds.data_ptr(),
                              bound_scales.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), p,
                              _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "pa_select_blocks")


def _sparse_decode_params(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected, max_seq_len,
                          sink_blocks, recent_blocks, k_scales, v_scales):
    """Checks the attention's operands; the packed pa_sparse_params, N, H_kv and the device."""
    shape, dev = q.shape, q.get_device()
    N, H, bs, d = kshape = key_cache.shape
    f32 = out.dtype is not q.dtype
    if not (_lists_good(q, shape, H, dev, block_tables, seq_lens, selected, num_selected) and
            value_cache.shape == kshape and value_cache.dtype is key_cache.dtype and bs == BLOCK_SIZE and
            shape[-1] == d and out.shape == shape and (not f32 or out.dtype is _F32) and
            out.is_contiguous() and key_cache.is_contiguous() and value_cache.is_contiguous() and
            out.get_device() == key_cache.get_device() == value_cache.get_device() == dev and
            (k_scales is None or (k_scales.dtype is _F32 and k_scales.shape == (N, H) and _on(dev, k_scales))) and
            (v_scales is None or (v_scales.dtype is _F32 and v_scales.shape == (N, H) and _on(dev, v_scales)))):
        _refuse([out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected, k_scales, v_scales],
                _list_rules(q, H, block_tables, seq_lens, selected, num_selected) +
                [(value_cache.shape != kshape or value_cache.dtype != key_cache.dtype or bs != BLOCK_SIZE or
                  shape[-1] != d, "caches must be [N][H_kv][16][d] of one dtype, with q's d"),
                 (out.shape != shape or out.dtype not in (q.dtype, _F32),
                  "out must match q in shape, and in dtype or be float32")] +
                [(not t.is_contiguous(), f"{name} must be contiguous")
                 for t, name in ((out, "out"), (key_cache, "key_cache"), (value_cache, "value_cache"))] +
                [(True, "scales must be contiguous float32 [N][H_kv]")])
    p = _SPARSE_PARAMS.pack(shape[0], shape[-2], H, d, bs, block_tables.shape[1], N, max_seq_len, _TORCH_DTYPE[q.dtype],
                            _TORCH_DTYPE[key_cache.dtype], 0 if k_scales is None else k_scales.data_ptr(),
                            0 if v_scales is None else v_scales.data_ptr(), shape[1] if len(shape) == 4 else 1,
                            selected.shape[-1], sink_blocks, recent_blocks, PA_DECODE_OUT_F32 if f32 else 0)
    return p, N, H, dev


def pa_decode_selected(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected, scale,
                       max_seq_len, k_scales=None, v_scales=None, stream=None):
    """Decode attention over the blocks that selected / num_selected list (int32
    [B][H_kv][K], [B][H_kv], or with a Q after the B; see include/pa.h).  out, q, caches,
    block_tables and seq_lens as in pa_decode; int8 caches with their scales."""
    p, _, _, dev = _sparse_decode_params(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected,
                                         max_seq_len, 0, 1, k_scales, v_scales)
    rc = lib.pa_decode_selected(out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                                block_tables.data_ptr(), seq_lens.data_ptr(), selected.data_ptr(),
                                num_selected.data_ptr(), scale, p,
                                _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "pa_decode_selected")


def pa_decode_selected_stall_selftest(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected,
                                      scale, max_seq_len, stall_at, limit_ns, k_scales=None, v_scales=None, stream=None):
    """pa_decode_selected with the failure path exercised: the first warp of row 0 leaves the
    copies of its stall_at-th block unissued, so its bounded wait runs out after limit_ns (see
    include/pa.h).  Returns after the launch; the error word then holds PA_EFLAG_WAIT_TIMEOUT."""
    p, _, _, dev = _sparse_decode_params(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected,
                                         max_seq_len, 0, 1, k_scales, v_scales)
    _check(lib.pa_decode_selected_stall_selftest(
        out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), selected.data_ptr(), num_selected.data_ptr(), scale, p, int(stall_at), int(limit_ns),
        _raw_stream(dev) if stream is None else stream.cuda_stream), "pa_decode_selected_stall_selftest")


def pa_decode_sparse(out, q, key_cache, value_cache, bounds, bound_scales, block_tables, seq_lens, selected,
                     num_selected, scale, max_seq_len, sink_blocks=1, recent_blocks=2, k_scales=None, v_scales=None,
                     stream=None):
    """pa_select_blocks and pa_decode_selected in one call: selected and num_selected
    are filled and attended to.  Arguments as in those."""
    p, N, H, dev = _sparse_decode_params(out, q, key_cache, value_cache, block_tables, seq_lens, selected, num_selected,
                                         max_seq_len, sink_blocks, recent_blocks, k_scales, v_scales)
    if not (bounds.dtype is _I8 and bounds.shape == (N, H, 2, q.shape[-1]) and bound_scales.dtype is _F32 and
            bound_scales.shape == (N, H) and _on(dev, bounds, bound_scales)):
        _refuse([bounds, bound_scales], _box_rules(bounds, bound_scales, N, H, q.shape[-1]))
    rc = lib.pa_decode_sparse(out.data_ptr(), q.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
                              bounds.data_ptr(), bound_scales.data_ptr(), block_tables.data_ptr(),
                              seq_lens.data_ptr(), selected.data_ptr(), num_selected.data_ptr(), scale, p,
                              _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "pa_decode_sparse")


def pa_get_error_flags(reset: bool = True, stream=None) -> int:
    f = ctypes.c_uint(0)
    _check(lib.pa_get_error_flags(ctypes.byref(f), int(reset), _stream(stream)),
           "pa_get_error_flags")
    return int(f.value)


def version() -> int:
    return int(lib.pa_version())
