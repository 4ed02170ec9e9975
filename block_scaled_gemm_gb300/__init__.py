"""Python binding of the GB300 MX block-scaled FP8 GEMM C library.

Argument marshalling only: every step of the product runs in the CUDA
library ``libmxgemm.so`` (built from ``csrc/`` by ``_build.build()``); there is
no fallback.  The functions mirror the C interface of ``include/mxgemm.h``:

    h = mxgemm_create(device)
    mxgemm_run(h, M, N, K, A, A_scale, B, B_scale, C, use_acc, out_dtype, stream)
    mxgemm_destroy(h)

Tensor arguments may be anything with ``data_ptr()`` (torch CUDA tensors) or
raw integer device addresses.  ``stream`` may be a ``torch.cuda.Stream``, a
raw ``cudaStream_t`` integer, or None (the legacy default stream).
The operation is the scaled product documented as ``tlx.async_dot_scaled``
("TLX API Quick Reference", section "Matrix Multiply (MMA)").
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

from . import _build

__all__ = [
    "OUT_F32", "OUT_BF16", "OPT_MODE", "OPT_WAIT_TIMEOUT_NS", "OPT_TEST_STALL_PRODUCER",
    "OPT_SCHEDULER", "OPT_STREAM_K", "OPT_A_FORMAT", "OPT_B_FORMAT", "FMT_E4M3", "FMT_E5M2",
    "FMT_E2M3", "FMT_E3M2", "FMT_E2M1", "MxgemmError", "library", "library_path", "mxgemm_create", "mxgemm_run",
    "mxgemm_destroy", "mxgemm_set_option", "mxgemm_get_device_status", "mxgemm_status_string",
    "mxgemm_set_profile_events", "mxgemm_get_launch_count", "mxgemm_run_noalloc", "mxgemm_run_host",
    "mxgemm_quantize", "IN_F32", "IN_BF16", "EXPORTED_SYMBOLS", "Gemm", "OPT_SCALE_LAYOUT", "OPT_ELEMENT_LAYOUT", "OPT_B_MAJOR", "B_K_BY_N", "B_N_BY_K", "ELEMS_BYTE", "ELEMS_PACKED",
    "SCALES_ROW_MAJOR", "SCALES_PACKED", "mxgemm_scale_bytes", "mxgemm_noalloc_get_status",
    "mxgemm_noalloc_set_option", "mxgemm_run_block128", "mxgemm_quantize_block128", "BLOCK_ROWS", "BLOCK_COLS",
    "BLOCK_TILES", "Cache", "mxgemm_cache_append", "mxgemm_cache_attention", "OUT_E4M3", "ACT_SILU", "ACT_GELU_TANH",
    "mxgemm_run_gated_block128", "mxgemm_gated_backward", "mxgemm_norm_rope", "mxgemm_norm_rope_backward",
    "mxgemm_rope_frequencies", "ROPE_PLAIN", "ROPE_LINEAR", "ROPE_BASE", "ROPE_BY_PARTS", "mxgemm_cache_attention_shared", "OPT_SHARED_KEYS",
]

OUT_F32 = 0
OUT_BF16 = 1
OUT_E4M3 = 2

OPT_MODE = 1
OPT_WAIT_TIMEOUT_NS = 2
OPT_TEST_STALL_PRODUCER = 3
OPT_SCHEDULER = 4
OPT_STREAM_K = 5
OPT_A_FORMAT = 6
OPT_B_FORMAT = 7
OPT_SCALE_LAYOUT = 8
OPT_ELEMENT_LAYOUT = 10
OPT_B_MAJOR = 11
OPT_SHARED_KEYS = 12
B_K_BY_N = 0
B_N_BY_K = 1
ELEMS_BYTE = 0
ELEMS_PACKED = 1

# scale layouts (mxgemm_scale_layout_t)
SCALES_ROW_MAJOR = 0
SCALES_PACKED = 1

# blocks of mxgemm_quantize_block128 (mxgemm_block_t)
BLOCK_ROWS = 0
BLOCK_COLS = 1
BLOCK_TILES = 2

# activations of a gated block (mxgemm_act_t)
ACT_SILU = 0
ACT_GELU_TANH = 1

# frequencies of the rotation (mxgemm_rope_scaling_t)
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_BY_PARTS = 3

# element formats (mxgemm_format_t); one element per byte, sub-byte codes in
# the low bits
FMT_E4M3 = 0
FMT_E5M2 = 1
FMT_E2M3 = 2
FMT_E3M2 = 3
FMT_E2M1 = 4

OK = 0
ERR_INVALID_VALUE = 1
ERR_MISALIGNED = 2
ERR_UNSUPPORTED_DEVICE = 3
ERR_OUT_OF_MEMORY = 4
ERR_CUDA = 5
ERR_TIMEOUT = 6
ERR_TOO_LARGE = 7

EXPORTED_SYMBOLS = (
    "mxgemm_create", "mxgemm_run", "mxgemm_destroy", "mxgemm_set_option",
    "mxgemm_get_device_status", "mxgemm_status_string", "mxgemm_set_profile_events",
    "mxgemm_get_launch_count", "mxgemm_run_noalloc", "mxgemm_run_host", "mxgemm_quantize",
    "mxgemm_quantize_sr", "mxgemm_quantize_ex", "mxgemm_scale_bytes", "mxgemm_noalloc_get_status",
    "mxgemm_noalloc_set_option", "mxgemm_run_block128", "mxgemm_quantize_block128",
    "mxgemm_cache_append", "mxgemm_cache_attention", "mxgemm_run_gated_block128", "mxgemm_gated_backward",
    "mxgemm_norm_rope", "mxgemm_norm_rope_backward", "mxgemm_rope_frequencies", "mxgemm_cache_attention_shared",
)

_lib = None


# mxgemm_cache_t
_CACHE_STRUCT = struct.Struct("PPPPqiii4x")
# mxgemm_gated_grads_t, mxgemm_heads_t, mxgemm_rope_t
_GRADS_STRUCT = struct.Struct("12P")
_HEADS_STRUCT = struct.Struct("PqPqPqPPq")
_ROPE_STRUCT = struct.Struct("PPiif4x")


class MxgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {mxgemm_status_string(status)} (status {status})")


def library_path() -> Path:
    return _build.LIB


def library():
    """Load the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not path.exists():
            raise RuntimeError(
                f"CUDA library {path} is missing: build it with "
                "`python -m block_scaled_gemm_gb300._build` (there is no CPU fallback)")
        lib = ctypes.CDLL(str(path))
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.mxgemm_create.argtypes = [ctypes.POINTER(vp), i32]
        lib.mxgemm_create.restype = i32
        lib.mxgemm_run.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp]
        lib.mxgemm_run.restype = i32
        lib.mxgemm_destroy.argtypes = [vp]
        lib.mxgemm_destroy.restype = i32
        lib.mxgemm_set_option.argtypes = [vp, i32, i64]
        lib.mxgemm_set_option.restype = i32
        lib.mxgemm_get_device_status.argtypes = [vp, vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.mxgemm_get_device_status.restype = i32
        lib.mxgemm_set_profile_events.argtypes = [vp, vp, vp]
        lib.mxgemm_set_profile_events.restype = i32
        lib.mxgemm_get_launch_count.argtypes = [vp, ctypes.POINTER(i64)]
        lib.mxgemm_get_launch_count.restype = i32
        lib.mxgemm_quantize.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
        lib.mxgemm_quantize.restype = i32
        lib.mxgemm_quantize_sr.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp, vp]
        lib.mxgemm_quantize_sr.restype = i32
        lib.mxgemm_quantize_ex.argtypes = [vp, i32, i64, i64, i32, vp, i32, vp, vp, vp]
        lib.mxgemm_quantize_ex.restype = i32
        lib.mxgemm_scale_bytes.argtypes = [i64, i64, i32, i32, ctypes.POINTER(i64)]
        lib.mxgemm_scale_bytes.restype = i32
        lib.mxgemm_run_host.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp]
        lib.mxgemm_run_host.restype = i32
        lib.mxgemm_run_noalloc.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp]
        lib.mxgemm_run_noalloc.restype = i32
        lib.mxgemm_noalloc_get_status.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        lib.mxgemm_noalloc_get_status.restype = i32
        lib.mxgemm_noalloc_set_option.argtypes = [i32, i64]
        lib.mxgemm_noalloc_set_option.restype = i32
        lib.mxgemm_run_block128.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, i32, vp, i32, i32, vp]
        lib.mxgemm_run_block128.restype = i32
        lib.mxgemm_quantize_block128.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
        lib.mxgemm_quantize_block128.restype = i32
        lib.mxgemm_cache_append.argtypes = [vp, ctypes.c_char_p, i64, vp, i64, vp, vp, i64, vp, vp, i64, i32, vp]
        lib.mxgemm_cache_append.restype = i32
        lib.mxgemm_cache_attention.argtypes = [vp, ctypes.c_char_p, i64, i64, vp, i64, vp, vp, i64, vp, i64,
                                               ctypes.c_float, i32, i64, i64, vp, vp, vp]
        lib.mxgemm_cache_attention.restype = i32
        f32, f64 = ctypes.c_float, ctypes.c_double
        lib.mxgemm_run_gated_block128.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp]
        lib.mxgemm_run_gated_block128.restype = i32
        lib.mxgemm_gated_backward.argtypes = [vp, vp, vp, i32, i64, i64, i32, ctypes.c_char_p, vp]
        lib.mxgemm_gated_backward.restype = i32
        lib.mxgemm_norm_rope.argtypes = [ctypes.c_char_p, ctypes.c_char_p, i64, i64, i32, i32, f32, ctypes.c_char_p, vp]
        lib.mxgemm_norm_rope.restype = i32
        lib.mxgemm_norm_rope_backward.argtypes = [vp, *lib.mxgemm_norm_rope.argtypes]
        lib.mxgemm_norm_rope_backward.restype = i32
        lib.mxgemm_rope_frequencies.argtypes = [i64, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64)]
        lib.mxgemm_rope_frequencies.restype = i32
        lib.mxgemm_cache_attention_shared.argtypes = [vp, ctypes.c_char_p, i64, i64, vp, i64, vp, vp, i64, i64, vp, i64,
                                                      f32, i32, vp, vp, vp]
        lib.mxgemm_cache_attention_shared.restype = i32
        lib.mxgemm_status_string.argtypes = [i32]
        lib.mxgemm_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def mxgemm_status_string(status: int) -> str:
    return library().mxgemm_status_string(int(status)).decode()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str):
    if st != OK:
        raise MxgemmError(st, where)


def mxgemm_create(device: int = 0):
    h = ctypes.c_void_p()
    _check(library().mxgemm_create(ctypes.byref(h), int(device)), "mxgemm_create")
    return h


def mxgemm_run(h, M, N, K, A, A_scale, B, B_scale, C, use_acc=0, out_dtype=OUT_F32, stream=None,
               check: bool = True) -> int:
    st = library().mxgemm_run(h, int(M), int(N), int(K), _ptr(A), _ptr(A_scale), _ptr(B),
                              _ptr(B_scale), _ptr(C), int(bool(use_acc)), int(out_dtype),
                              _stream(stream))
    if check:
        _check(st, "mxgemm_run")
    return st


IN_F32 = 0
IN_BF16 = 1


def _in_dtype(X) -> int:
    """IN_F32 or IN_BF16 as X's dtype says; a bare address counts as float32."""
    import torch
    dtype = getattr(X, "dtype", torch.float32)
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError(f"X: float32 or bfloat16 (or x_dtype given), not {dtype}")
    return IN_BF16 if dtype is torch.bfloat16 else IN_F32


def mxgemm_quantize(X, R, C, codes, scales, along_cols=False, x_dtype=None, stream=None,
                    check: bool = True, rand_bits=None, scale_layout=SCALES_ROW_MAJOR) -> int:
    """MX-quantize the R x C device matrix X (float32 or bfloat16) into E4M3
    codes (R x C bytes) and E8M0 scales per 32 values, along the rows
    (A_scale of an M x K X) or down the columns (B_scale of a K x N X).
    With rand_bits (an R x C device tensor of 32-bit words) the codes round
    stochastically, else to nearest even.  scale_layout SCALES_ROW_MAJOR
    gives R x C/32 (rows) or C x R/32 (columns) scales, SCALES_PACKED the
    order a run with OPT_SCALE_LAYOUT = SCALES_PACKED reads
    (mxgemm_scale_bytes bytes)."""
    if x_dtype is None:
        x_dtype = _in_dtype(X)
    lib = library()
    if rand_bits is None and scale_layout == SCALES_ROW_MAJOR:
        st = lib.mxgemm_quantize(_ptr(X), int(x_dtype), int(R), int(C), int(bool(along_cols)),
                                 _ptr(codes), _ptr(scales), _stream(stream))
        name = "mxgemm_quantize"
    elif scale_layout == SCALES_ROW_MAJOR:
        st = lib.mxgemm_quantize_sr(_ptr(X), int(x_dtype), int(R), int(C), int(bool(along_cols)),
                                    _ptr(rand_bits), _ptr(codes), _ptr(scales), _stream(stream))
        name = "mxgemm_quantize_sr"
    else:
        st = lib.mxgemm_quantize_ex(_ptr(X), int(x_dtype), int(R), int(C), int(bool(along_cols)),
                                    _ptr(rand_bits), int(scale_layout), _ptr(codes), _ptr(scales),
                                    _stream(stream))
        name = "mxgemm_quantize_ex"
    if check:
        _check(st, name)
    return st


def mxgemm_scale_bytes(R, C, along_cols=False, scale_layout=SCALES_ROW_MAJOR) -> int:
    """Bytes of the scales of an R x C matrix quantized along the rows or
    down the columns, in the given layout."""
    out = ctypes.c_int64(0)
    _check(library().mxgemm_scale_bytes(int(R), int(C), int(bool(along_cols)), int(scale_layout),
                                        ctypes.byref(out)), "mxgemm_scale_bytes")
    return int(out.value)


def mxgemm_run_host(h, M, N, K, A, A_scale, B, B_scale, C, use_acc=0, out_dtype=OUT_F32,
                    stream=None, check: bool = True) -> int:
    """C (+)= A.B with every operand and C in host memory (CPU tensors,
    contiguous; pinned ones let the copies overlap the GEMM).  C is complete
    once `stream` is synchronized (see include/mxgemm.h)."""
    st = library().mxgemm_run_host(h, int(M), int(N), int(K), _ptr(A), _ptr(A_scale), _ptr(B),
                                   _ptr(B_scale), _ptr(C), int(bool(use_acc)), int(out_dtype),
                                   _stream(stream))
    if check:
        _check(st, "mxgemm_run_host")
    return st


def mxgemm_run_noalloc(M, N, K, A, A_scale, B, B_scale, C, use_acc=0, out_dtype=OUT_F32,
                       stream=None, check: bool = True) -> int:
    """C (+)= A.B on the current device without allocating device memory
    (fixed 16 MiB scratch shared by all calls; see include/mxgemm.h)."""
    st = library().mxgemm_run_noalloc(int(M), int(N), int(K), _ptr(A), _ptr(A_scale), _ptr(B),
                                      _ptr(B_scale), _ptr(C), int(bool(use_acc)), int(out_dtype),
                                      _stream(stream))
    if check:
        _check(st, "mxgemm_run_noalloc")
    return st


def mxgemm_noalloc_get_status(stream=None):
    """Synchronize `stream`, then read and clear the current device's status
    word of mxgemm_run_noalloc: (status, detail), the first failure since the
    last read."""
    st, det = ctypes.c_int(), ctypes.c_int()
    _check(library().mxgemm_noalloc_get_status(_stream(stream), ctypes.byref(st), ctypes.byref(det)),
           "mxgemm_noalloc_get_status")
    return st.value, det.value


def mxgemm_noalloc_set_option(option: int, value: int) -> None:
    """Process-wide option of mxgemm_run_noalloc (OPT_WAIT_TIMEOUT_NS or
    OPT_TEST_STALL_PRODUCER)."""
    _check(library().mxgemm_noalloc_set_option(int(option), int(value)), "mxgemm_noalloc_set_option")


def mxgemm_run_block128(h, M, N, K, A, A_scale, B, B_scale, C, use_acc=0, out_dtype=OUT_F32,
                        b_block=128, stream=None, check: bool = True) -> int:
    """C (+)= A.B with one float32 scale per block of 128 along K: A M x K with
    scales M x ceil(K/128); B N x K or K x N as the handle's OPT_B_MAJOR says,
    with a scale per 128 x 128 block (b_block=128) or per column and block of
    128 (b_block=1), laid out as B is (see include/mxgemm.h)."""
    st = library().mxgemm_run_block128(h, int(M), int(N), int(K), _ptr(A), _ptr(A_scale), _ptr(B),
                                       _ptr(B_scale), int(b_block), _ptr(C), int(bool(use_acc)),
                                       int(out_dtype), _stream(stream))
    if check:
        _check(st, "mxgemm_run_block128")
    return st


def mxgemm_quantize_block128(X, R, C, codes, scales, block=BLOCK_ROWS, x_dtype=None, stream=None,
                             check: bool = True) -> int:
    """Quantize the R x C device matrix X (float32 or bfloat16) into E4M3 codes
    with one float32 scale per block: BLOCK_ROWS 1 x 128 (codes R x C, scales
    R x ceil(C/128)), BLOCK_COLS 128 x 1 stored transposed (codes
    C x round_up(R, 16), scales C x ceil(R/128)), BLOCK_TILES 128 x 128 (codes
    R x C, scales ceil(R/128) x ceil(C/128))."""
    if x_dtype is None:
        x_dtype = _in_dtype(X)
    st = library().mxgemm_quantize_block128(_ptr(X), int(x_dtype), int(R), int(C), int(block),
                                            _ptr(codes), _ptr(scales), _stream(stream))
    if check:
        _check(st, "mxgemm_quantize_block128")
    return st


class Cache:
    """An 8-bit key/value cache: tensors K and V of E4M3 codes (uint8 or float8_e4m3fn,
    pages x kv heads x page size x head dim) and float32 tensors of their scales
    (pages x kv heads)."""

    def __init__(self, K, V, K_scale, V_scale):
        shape, dims = K.shape, K_scale.shape
        if len(shape) != 4 or V.shape != shape or dims != shape[:2] or V_scale.shape != dims:
            raise ValueError("K and V: pages x kv heads x page size x head dim, scales: pages x kv heads")
        import torch
        if not (all(t.element_size() == 1 and (t.dtype is torch.float8_e4m3fn or not t.is_floating_point()) for t in (K, V))
                and K_scale.dtype is V_scale.dtype is torch.float32
                and K.is_contiguous() and V.is_contiguous() and K_scale.is_contiguous() and V_scale.is_contiguous()):
            raise ValueError("a cache is dense, with E4M3 codes and float32 scales")
        self.K, self.V, self.K_scale, self.V_scale = K, V, K_scale, V_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = shape
        self._c = _CACHE_STRUCT.pack(K.data_ptr(), V.data_ptr(), K_scale.data_ptr(), V_scale.data_ptr(),
                                     self.num_pages, self.page_size, self.kv_heads, self.head_dim)


def _token_pitch(shape, stride, name):
    """Elements from token to token of a (tokens, heads, head dim) tensor whose tokens are dense."""
    if len(shape) != 3 or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name}: tokens x heads x head dim, each token dense")
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


def _batch(page_table, kv_len, q_start):
    """A batch's size, its table's width, and the pointers of its page table, lengths and row starts."""
    for t in (page_table, kv_len) if q_start is None else (page_table, kv_len, q_start):
        if t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous():
            raise ValueError("page_table, kv_len and q_start: dense int32 tensors")
    shape = page_table.shape
    if len(shape) != 2 or kv_len.numel() != shape[0] or (q_start is not None and q_start.numel() != shape[0] + 1):
        raise ValueError("page_table: batch x pages, kv_len: batch, q_start: batch + 1")
    return (shape[0], shape[1], page_table.data_ptr(), kv_len.data_ptr(),
            None if q_start is None else q_start.data_ptr())


def mxgemm_cache_append(h, cache: Cache, page_table, kv_len, new_K, new_V, q_start=None, stream=None,
                        check: bool = True) -> int:
    """Append new keys and values (tokens x kv heads x head dim, float32 or
    bfloat16; slices of a projection's output will do) to the sequences of a
    cache.  page_table: batch x pages int32; kv_len: lengths with the new
    tokens; q_start: batch + 1 row starts, None for one token each."""
    import torch
    shape, stride, dtype = new_K.shape, new_K.stride(), new_K.dtype
    pitch = _token_pitch(shape, stride, "new_K")
    if new_V.shape != shape or new_V.dtype != dtype or (new_V.stride() != stride and
                                                        _token_pitch(shape, new_V.stride(), "new_V") != pitch):
        raise ValueError("new_V is laid out as new_K is")
    if shape[1] != cache.kv_heads or shape[2] != cache.head_dim:
        raise ValueError("new_K: tokens x kv heads x head dim")
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("new_K: float32 or bfloat16")
    batch, width, table, lens, starts = _batch(page_table, kv_len, q_start)
    st = library().mxgemm_cache_append(h, cache._c, batch, table, width, lens, starts, shape[0], new_K.data_ptr(),
                                       new_V.data_ptr(), pitch, IN_BF16 if dtype is torch.bfloat16 else IN_F32,
                                       _stream(stream))
    if check:
        _check(st, "mxgemm_cache_append")
    return st


def _queries(cache, Q, O, lse):
    """Shape and pitch of an attention's queries, with its outputs checked against them."""
    import torch
    shape = Q.shape
    pitch = _token_pitch(shape, Q.stride(), "Q")
    if Q.dtype is not torch.bfloat16 or O.dtype is not torch.bfloat16 or O.shape != shape or not O.is_contiguous():
        raise ValueError("Q and O: bfloat16 of one shape, O dense")
    if shape[2] != cache.head_dim:
        raise ValueError("Q: tokens x heads x head dim")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:2] or not lse.is_contiguous()):
        raise ValueError("lse: a dense float32 tensor, tokens x heads")
    return shape, pitch


def mxgemm_cache_attention(h, cache: Cache, page_table, kv_len, Q, O, q_start=None, scale=None,
                           causal=True, window=0, sinks=0, lse=None, stream=None,
                           check: bool = True) -> int:
    """Attention of Q (tokens x heads x head dim bfloat16) over a cache into O
    (the same shape, dense) and, where given, lse (tokens x heads float32).
    page_table, kv_len and q_start as for mxgemm_cache_append; scale defaults
    to 1 / sqrt(head dim); window = 0 is no window."""
    shape, pitch = _queries(cache, Q, O, lse)
    batch, width, table, lens, starts = _batch(page_table, kv_len, q_start)
    st = library().mxgemm_cache_attention(
        h, cache._c, batch, shape[1], table, width, lens, starts, shape[0], Q.data_ptr(), pitch,
        shape[2] ** -0.5 if scale is None else scale, 1 if causal else 0, window, sinks, O.data_ptr(),
        None if lse is None else lse.data_ptr(), _stream(stream))
    if check:
        _check(st, "mxgemm_cache_attention")
    return st


def mxgemm_cache_attention_shared(h, cache: Cache, page_table, kv_len, shared, Q, O, q_start=None, scale=None,
                                  causal=True, lse=None, stream=None, check: bool = True) -> int:
    """mxgemm_cache_attention for sequences whose first `shared` tokens are in the same
    pages (as far as each sequence reaches): those are read once for the whole batch.
    Other arguments as there, without a window."""
    shape, pitch = _queries(cache, Q, O, lse)
    batch, width, table, lens, starts = _batch(page_table, kv_len, q_start)
    st = library().mxgemm_cache_attention_shared(
        h, cache._c, batch, shape[1], table, width, lens, starts, shape[0], shared, Q.data_ptr(), pitch,
        shape[2] ** -0.5 if scale is None else scale, 1 if causal else 0, O.data_ptr(),
        None if lse is None else lse.data_ptr(), _stream(stream))
    if check:
        _check(st, "mxgemm_cache_attention_shared")
    return st


_codes = {}  # IN_F32 and IN_BF16 by torch's types, once torch is there


def _type_codes():
    if not _codes:
        import torch
        _codes.update({torch.float32: IN_F32, torch.bfloat16: IN_BF16})
    return _codes


_kinds = {}  # torch's types of what is passed on as plain addresses, by IN_F32, IN_BF16 and (None) one byte a value


def _type_sets():
    if not _kinds:
        import torch
        one = (x for x in vars(torch).values() if isinstance(x, torch.dtype) and x.itemsize == 1)
        _kinds.update({IN_F32: {torch.float32}, IN_BF16: {torch.bfloat16}, None: set(one)})
    return _kinds


def _address(name, t, types, n):
    """The address of a tensor, refused unless it is of one of the types and dense with n
    values or more.  (An address and None are taken as they are.)"""
    if t is None or t.__class__ is int:
        return t
    if t.dtype in types and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    of = "one byte a value" if len(types) > 1 else "".join(map(str, types)) or "of out_dtype"
    raise ValueError(f"{name}: a dense tensor of {n} values, {of}; not {t.dtype}, {tuple(t.shape)} with strides {t.stride()}")


def mxgemm_run_gated_block128(h, M, N, K, A, A_scale, G, G_scale, U, U_scale, H, H_scale=None, act=ACT_SILU,
                              out_dtype=OUT_BF16, gate=None, up=None, stream=None, check: bool = True) -> int:
    """H = act(A.G) * (A.U) with the operands of mxgemm_run_block128 (both weights as the
    handle's OPT_B_MAJOR says): float32, bfloat16, or OUT_E4M3 codes with H_scale
    (M x ceil(N/128)), the operand of the next product.  gate and up (M x N bfloat16)
    receive A.G and A.U for mxgemm_gated_backward.  All tensors dense; scales float32."""
    M, N, K = int(M), int(N), int(K)
    kb, nb, w, n = -(-K // 128), -(-N // 128), N * K, M * N
    types = _type_sets()
    one, f32, bf16 = types[None], types[IN_F32], types[IN_BF16]
    of_h = one if out_dtype == OUT_E4M3 else types.get(out_dtype, ())
    st = library().mxgemm_run_gated_block128(
        h, M, N, K, _address("A", A, one, M * K), _address("A_scale", A_scale, f32, M * kb), _address("G", G, one, w),
        _address("G_scale", G_scale, f32, nb * kb), _address("U", U, one, w), _address("U_scale", U_scale, f32, nb * kb), int(act),
        _address("H", H, of_h, n), _address("H_scale", H_scale, f32, M * nb), int(out_dtype), _address("gate", gate, bf16, n),
        _address("up", up, bf16, n), _stream(stream))
    if check:
        _check(st, "mxgemm_run_gated_block128")
    return st


def mxgemm_gated_backward(gate, up, dH, R, C, dgate=None, dup=None, dgate_rows=None, dup_rows=None, dgate_cols=None,
                          dup_cols=None, hidden_cols=None, act=ACT_SILU, x_dtype=None, stream=None,
                          check: bool = True) -> int:
    """The gradient of act(gate) * up (R x C bfloat16) for dH (float32 or bfloat16).
    dgate, dup: R x C bfloat16; the others pairs (codes, scales) as
    mxgemm_quantize_block128 makes them, by rows or by columns.  All tensors dense.
    What is None is left out."""
    if x_dtype is None:
        x_dtype = _in_dtype(dH)
    R, C = int(R), int(C)
    n = R * C
    types = _type_sets()
    one, f32, bf16 = types[None], types[IN_F32], types[IN_BF16]
    dgate, dup = _address("dgate", dgate, bf16, n), _address("dup", dup, bf16, n)
    # (another x_dtype is the library's to refuse)
    dh = _address("dH", dH, types[x_dtype], n) if x_dtype in (IN_F32, IN_BF16) else _ptr(dH)
    pairs = [p if p is not None else (None, None) for p in (dgate_rows, dup_rows, dgate_cols, dup_cols, hidden_cols)]
    if C % 16 == 0:  # (else the library refuses quantized outputs)
        rows, cols = (n, R * -(-C // 128)), (C * (-(-R // 16) * 16), C * -(-R // 128))
        for name, (codes, scales), of in zip(("dgate_rows", "dup_rows", "dgate_cols", "dup_cols", "hidden_cols"), pairs, (rows, rows, cols, cols, cols)):
            if hasattr(codes, "dtype") and hasattr(scales, "dtype"):
                _address(name + "' codes", codes, one, of[0])
                _address(name + "' scales", scales, f32, of[1])
    out = _GRADS_STRUCT.pack(dgate or 0, dup or 0, *(_ptr(y) or 0 for p in pairs for y in p))
    st = library().mxgemm_gated_backward(_address("gate", gate, bf16, n), _address("up", up, bf16, n), dh, int(x_dtype), R, C, int(act),
                                         out, _stream(stream))
    if check:
        _check(st, "mxgemm_gated_backward")
    return st


def _rows(name, t, shape, dtype):
    """Address and pitch of a tensor of (tokens, heads, d) values."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name}: tokens x heads x head dim, all tensors of one type")
    pitch, head, step = t.stride()
    tokens, heads, d = shape
    if step != 1 or (head != d and heads > 1):
        raise ValueError(f"{name}: tokens x heads x head dim, each token dense")
    return t.data_ptr(), pitch if tokens > 1 else heads * d


def _heads(name, tokens, d, dtype, x, y, weight, dy, dweight):
    """mxgemm_heads_t of a tensor's values, result and gradient, each (tokens, heads, d) of one type."""
    shape = y.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != d:
        raise ValueError(f"{name}: tokens x heads x head dim, all tensors of one type")
    out, out_pitch = _rows(name, y, shape, dtype)
    at, pitch = (0, 0) if x is None else _rows(name, x, shape, dtype)
    g, g_pitch = (0, 0) if dy is None else _rows(name, dy, shape, dtype)
    w = dw = 0
    if weight is not None:
        if x is None:
            raise ValueError(f"{name}: a norm needs the values")
        if weight.shape != (d,) or not weight.is_contiguous():
            raise ValueError(f"{name}'s weight: head dim values")
        w = weight.data_ptr()
    if dweight is not None:
        if weight is None or _type_codes().get(dweight.dtype) != IN_F32 or dweight.shape != (d,) or not dweight.is_contiguous():
            raise ValueError(f"{name}'s weight's gradient: head dim float32 values, of a weight")
        dw = dweight.data_ptr()
    return _HEADS_STRUCT.pack(at, pitch, g, g_pitch, out, out_pitch, w, dw, shape[1])


_rope_types = {}  # the types of positions and frequencies


def _rope(positions, freqs, interleaved, factor, tokens):
    if freqs is None:
        return None
    if not _rope_types:
        import torch
        _rope_types.update(pos=torch.int32, freqs=torch.float64)
    if positions is None or positions.dtype is not _rope_types["pos"] or positions.shape != (tokens,) or not positions.is_contiguous():
        raise ValueError("positions: a dense int32 tensor, one for each token")
    n = freqs.numel()
    if freqs.dtype is not _rope_types["freqs"] or freqs.shape != (n,) or not freqs.is_contiguous():
        raise ValueError("freqs: a dense float64 tensor, one for each pair")
    return _ROPE_STRUCT.pack(positions.data_ptr(), freqs.data_ptr(), 2 * n, 1 if interleaved else 0, factor)


def _rope_call(name, handle, q, k, positions, freqs, interleaved, factor, eps, stream, check):
    """q and k: (values, result, weight, dy, dweight) each, k's result None for none."""
    y = q[1]
    if y is None or y.dim() != 3:
        raise ValueError("q: tokens x heads x head dim")
    if k[1] is None and (k[0] is not None or k[3] is not None or k[4] is not None):
        raise ValueError("k: without a result nothing of it would be computed")
    tokens, _, d = y.shape
    dtype = y.dtype
    types = _type_codes()
    x_dtype = types.get(dtype)
    if x_dtype is None:
        raise ValueError("q: float32 or bfloat16")
    w_dtype = None
    for w in (q[2], k[2]):
        if w is not None:
            code = types.get(w.dtype)
            if code is None or (w_dtype is not None and code != w_dtype):
                raise ValueError("weights: float32 or bfloat16, q's and k's of one type")
            w_dtype = code
    st = getattr(library(), name)(*handle, _heads("q", tokens, d, dtype, *q), None if k[1] is None else _heads("k", tokens, d, dtype, *k),
                                  tokens, d, x_dtype, w_dtype or 0, eps, _rope(positions, freqs, interleaved, factor, tokens),
                                  _stream(stream))
    if check:
        _check(st, name)
    return st


def mxgemm_norm_rope(q, k, q_out, k_out, positions=None, freqs=None, interleaved=False, factor=1.0, q_weight=None,
                     k_weight=None, eps=1e-6, stream=None, check: bool = True) -> int:
    """Norms of queries and keys for each head (with a weight; without one no norm) and
    the rotation of each head's first 2 * len(freqs) values by positions[t] * freqs[j],
    in one pass.  q, k and the results: tokens x heads x head dim, float32 or bfloat16,
    slices of a projection's output will do; k and k_out may be None, and a result may be
    its input.  positions: int32; freqs: float64 (mxgemm_rope_frequencies), None for no
    rotation."""
    return _rope_call("mxgemm_norm_rope", (), (q, q_out, q_weight, None, None), (k, k_out, k_weight, None, None),
                      positions, freqs, interleaved, factor, eps, stream, check)


def mxgemm_norm_rope_backward(h, dq_out, dk_out, dq, dk, q=None, k=None, positions=None, freqs=None, interleaved=False,
                              factor=1.0, q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, eps=1e-6,
                              stream=None, check: bool = True) -> int:
    """The gradient of mxgemm_norm_rope: from dq_out and dk_out (of its results) to dq and
    dk (of its inputs q and k, which a norm needs) and, where given, the weights'
    dq_weight and dk_weight (float32, set)."""
    return _rope_call("mxgemm_norm_rope_backward", (h,), (q, dq, q_weight, dq_out, dq_weight),
                      (k, dk, k_weight, dk_out, dk_weight), positions, freqs, interleaved, factor, eps, stream, check)


def mxgemm_rope_frequencies(rot, base=10000.0, scaling=ROPE_PLAIN, scale=1.0, trained=0.0, slow=1.0, fast=4.0):
    """Frequencies for mxgemm_norm_rope, a float64 CPU tensor of rot / 2: base^(-2j/rot),
    stretched for long contexts as `scaling` says (ROPE_LINEAR, ROPE_BASE,
    ROPE_BY_PARTS)."""
    import torch
    out = (ctypes.c_double * max(1, int(rot) // 2))()
    _check(library().mxgemm_rope_frequencies(int(rot), float(base), int(scaling), float(scale), float(trained), float(slow),
                                             float(fast), out), "mxgemm_rope_frequencies")
    return torch.tensor(out[:int(rot) // 2], dtype=torch.float64)


def mxgemm_set_option(h, option: int, value: int) -> None:
    _check(library().mxgemm_set_option(h, int(option), int(value)), "mxgemm_set_option")


def mxgemm_get_device_status(h, stream=None):
    st, det = ctypes.c_int(), ctypes.c_int()
    _check(library().mxgemm_get_device_status(h, _stream(stream), ctypes.byref(st), ctypes.byref(det)),
           "mxgemm_get_device_status")
    return st.value, det.value


def mxgemm_set_profile_events(h, ev_before, ev_after) -> None:
    """Record these CUDA events (torch.cuda.Event, raw handles or None)
    around the GEMM kernel launch of later runs.  torch events must already
    have been recorded once (torch creates the CUDA event lazily)."""
    def raw(e):
        if e is None or isinstance(e, int):
            return e
        return e.cuda_event
    _check(library().mxgemm_set_profile_events(h, raw(ev_before), raw(ev_after)),
           "mxgemm_set_profile_events")


def mxgemm_get_launch_count(h) -> int:
    n = ctypes.c_int64()
    _check(library().mxgemm_get_launch_count(h, ctypes.byref(n)), "mxgemm_get_launch_count")
    return n.value


def mxgemm_destroy(h) -> None:
    _check(library().mxgemm_destroy(h), "mxgemm_destroy")


class Gemm:
    """Owns one handle.  ``g(A, As, B, Bs, C, use_acc, out_dtype)`` enqueues
    C (+)= A.B on the current torch stream (shapes taken from the tensors)."""

    def __init__(self, device: int = 0, mode: int | None = None):
        self.h = mxgemm_create(device)
        if mode is not None:
            mxgemm_set_option(self.h, OPT_MODE, mode)

    def __call__(self, A, A_scale, B, B_scale, C, use_acc=False, out_dtype=OUT_F32, stream=None):
        M, K = A.shape
        N = B.shape[1]
        if stream is None:
            import torch
            stream = torch.cuda.current_stream(A.device)
        return mxgemm_run(self.h, M, N, K, A, A_scale, B, B_scale, C, use_acc, out_dtype, stream)

    def set_option(self, option: int, value: int):
        mxgemm_set_option(self.h, option, value)

    def status(self, stream=None):
        return mxgemm_get_device_status(self.h, stream)

    def close(self):
        if self.h is not None:
            mxgemm_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
