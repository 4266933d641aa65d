"""ctypes loader for libi8mp.so (no compute here: argument marshalling only)."""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, Structure, c_char_p, c_float, c_int32, c_int64, c_size_t, c_void_p

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libi8mp.so")

I8MP_OK = 0
I8MP_EINVAL = -1
I8MP_ERANGE = -2
I8MP_EWORKSPACE = -3
I8MP_EDEVICE = -4
I8MP_ELAUNCH = -5
I8MP_ESCRATCH = -6
I8MP_MAX_K = 133144
I8MP_NOALLOC_SCRATCH_BYTES = 32 << 20

# Every symbol include/i8mp.h declares.
EXPORTS = (
    "i8mp_status_string",
    "i8mp_abi_version",
    "i8mp_quant_workspace_bytes",
    "i8mp_int8_vectorwise_quant",
    "i8mp_outlier_extract",
    "i8mp_int8_linear_matmul",
    "i8mp_int8_mm_dequant",
    "i8mp_int8_vectorwise_dequant",
    "i8mp_linear_workspace_query",
    "i8mp_linear_quantize",
    "i8mp_linear_matmul_dequant",
    "i8mp_linear_forward",
    "i8mp_linear_forward_noalloc",
    "i8mp_colwise_quant_workspace_bytes",
    "i8mp_int8_colwise_quant",
    "i8mp_linear_backward_workspace_query",
    "i8mp_linear_backward",
    "i8mp_fp4_quantize",
    "i8mp_fp4_double_quant",
    "i8mp_fp4_dequantize",
    "i8mp_fp4_linear",
    "i8mp_fp4_cache_bytes",
    "i8mp_fp4_cache_write",
    "i8mp_fp4_cache_read",
    "i8mp_fp4_attention_workspace_bytes",
    "i8mp_fp4_cache_attention",
    "i8mp_fp4_cache_append",
    "i8mp_mx4_quantize",
    "i8mp_mx4_dequantize",
    "i8mp_mx4_matmul_workspace_bytes",
    "i8mp_mx4_matmul",
    "i8mp_mx4_linear_workspace_bytes",
    "i8mp_mx4_linear",
    "i8mp_mx4_linear_backward_workspace_bytes",
    "i8mp_mx4_linear_backward",
)


class LinearWorkspaceLayout(Structure):
    _fields_ = [
        ("bytes", c_size_t),
        ("q_offset", c_size_t),
        ("ldq", c_int64),
        ("absmax_offset", c_size_t),
        ("bitmap_offset", c_size_t),
        ("idx_offset", c_size_t),
        ("count_offset", c_size_t),
        ("xo_offset", c_size_t),
        ("cap_pad", c_int32),
        ("scratch_offset", c_size_t),
        ("scratch_bytes", c_size_t),
        ("idx_len", c_int64),
    ]


class BackwardWorkspaceLayout(Structure):
    _fields_ = [
        ("bytes", c_size_t),
        ("ld_n", c_int64),
        ("ld_m", c_int64),
        ("gq_offset", c_size_t),
        ("gs_offset", c_size_t),
        ("wtq_offset", c_size_t),
        ("wts_offset", c_size_t),
        ("gtq_offset", c_size_t),
        ("gts_offset", c_size_t),
        ("xtq_offset", c_size_t),
        ("xts_offset", c_size_t),
        ("scratch_offset", c_size_t),
        ("scratch_bytes", c_size_t),
    ]


class Fp4CacheStruct(Structure):
    _fields_ = [
        ("data", c_void_p),
        ("pages", c_int64),
        ("kv_heads", c_int32),
        ("page_size", c_int32),
        ("head_dim", c_int32),
        ("dtype", c_int32),
    ]


class Fp4AttentionStruct(Structure):
    _fields_ = [
        ("q", c_void_p),
        ("ldq", c_int64),
        ("hsq", c_int64),
        ("out", c_void_p),
        ("ldo", c_int64),
        ("hso", c_int64),
        ("lse", c_void_p),
        ("table", c_void_p),
        ("ldt", c_int64),
        ("table_cols", c_int32),
        ("lengths", c_void_p),
        ("q_offsets", c_void_p),
        ("alibi", c_void_p),
        ("prefix", c_void_p),
        ("tokens", c_int64),
        ("batch", c_int32),
        ("q_heads", c_int32),
        ("max_q", c_int32),
        ("max_len", c_int32),
        ("window", c_int32),
        ("scale", c_float),
        ("softcap", c_float),
        ("fill", c_int32),
    ]


class Fp4AppendStruct(Structure):
    _fields_ = [
        ("k", c_void_p),
        ("ldk", c_int64),
        ("hsk", c_int64),
        ("v", c_void_p),
        ("ldv", c_int64),
        ("hsv", c_int64),
        ("slots", c_void_p),
        ("positions", c_void_p),
        ("cos", c_void_p),
        ("sin", c_void_p),
        ("ldcos", c_int64),
        ("ldsin", c_int64),
        ("table_rows", c_int64),
        ("q", c_void_p),
        ("ldq", c_int64),
        ("hsq", c_int64),
        ("out", c_void_p),
        ("ldo", c_int64),
        ("hso", c_int64),
        ("tokens", c_int64),
        ("q_heads", c_int32),
        ("rotary", c_int32),
        ("interleaved", c_int32),
    ]


class Mx4Struct(Structure):
    _fields_ = [
        ("codes", c_void_p),
        ("scales", c_void_p),
        ("rows", c_int64),
        ("k", c_int64),
        ("ldc", c_int64),
        ("lds", c_int64),
    ]


class I8mpError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def _declare(lib):
    lib.i8mp_status_string.argtypes = [c_int32]
    lib.i8mp_status_string.restype = c_char_p
    lib.i8mp_abi_version.argtypes = []
    lib.i8mp_abi_version.restype = c_int32
    lib.i8mp_quant_workspace_bytes.argtypes = [c_int64, c_int64]
    lib.i8mp_quant_workspace_bytes.restype = c_size_t
    lib.i8mp_int8_vectorwise_quant.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_float, c_void_p,
                                               c_int64, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.i8mp_int8_vectorwise_quant.restype = c_int32
    lib.i8mp_outlier_extract.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int32, c_void_p,
                                         c_void_p, c_void_p, c_int64, c_void_p]
    lib.i8mp_outlier_extract.restype = c_int32
    lib.i8mp_int8_linear_matmul.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int64, c_int64,
                                            c_void_p, c_int64, c_void_p]
    lib.i8mp_int8_linear_matmul.restype = c_int32
    lib.i8mp_int8_mm_dequant.argtypes = [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                                         c_void_p, c_int64, c_void_p, c_void_p, c_int32, c_void_p, c_int64,
                                         c_int64, c_void_p, c_int64, c_void_p]
    lib.i8mp_int8_mm_dequant.restype = c_int32
    lib.i8mp_int8_vectorwise_dequant.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int32, c_void_p,
                                                 c_int64, c_void_p]
    lib.i8mp_int8_vectorwise_dequant.restype = c_int32
    lib.i8mp_linear_workspace_query.argtypes = [c_int64, c_int64, c_int64, c_int32,
                                                POINTER(LinearWorkspaceLayout)]
    lib.i8mp_linear_workspace_query.restype = c_int32
    lib.i8mp_linear_forward.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p,
                                        c_int64, c_void_p, c_float, c_int32, c_void_p, c_int64, c_void_p,
                                        c_size_t, c_void_p]
    lib.i8mp_linear_forward.restype = c_int32
    lib.i8mp_linear_forward_noalloc.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p,
                                                c_int64, c_void_p, c_float, c_int32, c_void_p, c_int64, c_void_p]
    lib.i8mp_linear_forward_noalloc.restype = c_int32
    lib.i8mp_linear_quantize.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_float, c_int32, c_void_p,
                                         c_size_t, c_void_p]
    lib.i8mp_linear_quantize.restype = c_int32
    lib.i8mp_linear_matmul_dequant.argtypes = [c_void_p, c_int64, c_void_p, c_size_t, c_int64, c_int64, c_int32,
                                               c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_int64,
                                               c_void_p]
    lib.i8mp_linear_matmul_dequant.restype = c_int32
    lib.i8mp_colwise_quant_workspace_bytes.argtypes = [c_int64, c_int64]
    lib.i8mp_colwise_quant_workspace_bytes.restype = c_size_t
    lib.i8mp_int8_colwise_quant.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_int32,
                                            c_void_p, c_int64, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.i8mp_int8_colwise_quant.restype = c_int32
    lib.i8mp_linear_backward_workspace_query.argtypes = [c_int64, c_int64, c_int64, c_int32,
                                                         POINTER(BackwardWorkspaceLayout)]
    lib.i8mp_linear_backward_workspace_query.restype = c_int32
    lib.i8mp_linear_backward.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int64,
                                         c_int64, c_int64, c_int32, c_void_p, c_size_t, c_void_p, c_int64,
                                         c_void_p, c_int64, c_void_p, c_size_t, c_void_p]
    lib.i8mp_linear_backward.restype = c_int32
    lib.i8mp_fp4_quantize.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p, c_void_p]
    lib.i8mp_fp4_quantize.restype = c_int32
    lib.i8mp_fp4_double_quant.argtypes = [c_void_p, c_int64, c_void_p, c_void_p, c_void_p]
    lib.i8mp_fp4_double_quant.restype = c_int32
    lib.i8mp_fp4_dequantize.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p, c_int32,
                                        c_void_p, c_int64, c_void_p]
    lib.i8mp_fp4_dequantize.restype = c_int32
    lib.i8mp_fp4_linear.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p, c_void_p,
                                    c_void_p, c_int64, c_void_p, c_void_p, c_int64, c_void_p]
    lib.i8mp_fp4_linear.restype = c_int32
    cache = POINTER(Fp4CacheStruct)
    lib.i8mp_fp4_cache_bytes.argtypes = [cache]
    lib.i8mp_fp4_cache_bytes.restype = c_size_t
    lib.i8mp_fp4_cache_write.argtypes = [cache, c_void_p, c_int64, c_int64, c_void_p, c_int64, c_int64, c_void_p,
                                         c_int64, c_void_p]
    lib.i8mp_fp4_cache_write.restype = c_int32
    lib.i8mp_fp4_cache_read.argtypes = [cache, c_void_p, c_int64, c_int32, c_void_p, c_int64, c_int64, c_void_p,
                                        c_int64, c_int64, c_void_p]
    lib.i8mp_fp4_cache_read.restype = c_int32
    lib.i8mp_fp4_attention_workspace_bytes.argtypes = [cache, POINTER(Fp4AttentionStruct)]
    lib.i8mp_fp4_attention_workspace_bytes.restype = c_size_t
    lib.i8mp_fp4_cache_attention.argtypes = [cache, POINTER(Fp4AttentionStruct), c_void_p, c_size_t, c_void_p]
    lib.i8mp_fp4_cache_attention.restype = c_int32
    lib.i8mp_fp4_cache_append.argtypes = [cache, POINTER(Fp4AppendStruct), c_void_p]
    lib.i8mp_fp4_cache_append.restype = c_int32
    mx4 = POINTER(Mx4Struct)
    lib.i8mp_mx4_quantize.argtypes = [c_void_p, c_int32, c_int64, c_int64, c_int64, c_int32, mx4, c_void_p]
    lib.i8mp_mx4_quantize.restype = c_int32
    lib.i8mp_mx4_dequantize.argtypes = [mx4, c_int32, c_void_p, c_int64, c_void_p]
    lib.i8mp_mx4_dequantize.restype = c_int32
    for query in (lib.i8mp_mx4_matmul_workspace_bytes, lib.i8mp_mx4_linear_workspace_bytes,
                  lib.i8mp_mx4_linear_backward_workspace_bytes):
        query.argtypes = [c_int64, c_int64, c_int64]
        query.restype = c_size_t
    lib.i8mp_mx4_matmul.argtypes = [mx4, mx4, c_void_p, c_int32, c_void_p, c_int64, c_void_p, c_size_t, c_void_p]
    lib.i8mp_mx4_matmul.restype = c_int32
    lib.i8mp_mx4_linear.argtypes = [c_void_p, c_int32, c_int64, c_int64, mx4, c_void_p, c_void_p, c_int64, c_void_p,
                                    c_size_t, c_void_p]
    lib.i8mp_mx4_linear.restype = c_int32
    lib.i8mp_mx4_linear_backward.argtypes = [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_int32, c_int64,
                                             c_int64, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_size_t,
                                             c_void_p]
    lib.i8mp_mx4_linear_backward.restype = c_int32


def lib():
    """The loaded library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m int8_mixed_precision_vectorwise_amd.build_lib` (there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        _declare(handle)
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().i8mp_status_string(status).decode()
    except RuntimeError:
        return "library not loaded"


def check(status: int, what: str) -> None:
    if status != I8MP_OK:
        raise I8mpError(status, what)
