"""Python binding for libtgemm (dense FP16 GEMM on GB300, sm_103a).

Argument marshalling only: every step of C = epi(A·B), of the products with
4-bit weights and 8-bit codes and of the norms around a block runs in the CUDA
kernels of ``libtgemm.so``, called through its C ABI (``include/tgemm.h``).
PyTorch is used for device memory and streams.  There is no fallback: if the
shared library is missing, the first call raises ImportError.

Build the library with ``tiled_fp16_gemm_gb300.build.build()`` (nvcc, sm_103a).
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtgemm.so")

TG_EPI_NONE = 0
TG_EPI_RELU = 1

TG_OK = 0
TG_ERR_INVALID_VALUE = 1
TG_ERR_MISALIGNED = 2
TG_ERR_UNSUPPORTED_DEVICE = 3
TG_ERR_LAUNCH = 4
TG_ERR_NO_MEMORY = 5
TG_ERR_TIMEOUT = 6

TG_DTYPE_F16 = 0
TG_DTYPE_BF16 = 1
TG_DTYPE_F32 = 2

TG_KERNEL_NONE = 0
TG_KERNEL_FILL = 1
TG_KERNEL_PERSISTENT = 2
TG_KERNEL_SKINNY = 3

#: every symbol include/tgemm.h declares
EXPORTS = (
    "tg_gemm_f16", "tg_sync_status", "tg_status_string", "tg_version", "tg_plan_f16",
    "tg_tile_coord", "tg_ring_bytes", "tg_debug_set_wait_timeout_ns", "tg_debug_inject",
    "tg_gemm_f16_noalloc", "tg_gemm_bf16", "tg_gemm_ex", "tg_gemm_mxfp4", "tg_gemm_sp24",
    "tg_gemm_f16_host", "tg_plan_f16_limits", "tg_device_limits", "tg_debug_last_launch",
    "tg_debug_map_cache_stats", "tg_gemm_w4", "tg_norm_residual", "tg_norm_residual_backward",
    "tg_layer_norm", "tg_layer_norm_i8", "tg_quantize_rows", "tg_layer_norm_backward_workspace",
    "tg_layer_norm_backward", "tg_gemm_i8_workspace", "tg_gemm_i8",
)

#: bytes of the library's fixed scratch array used by tg_gemm_f16_noalloc
TG_NOALLOC_SCRATCH_BYTES = 24 * 1024 * 1024


class tg_plan_t(ctypes.Structure):
    _fields_ = [
        ("kernel", ctypes.c_int32), ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
        ("bk", ctypes.c_int32), ("stages", ctypes.c_int32), ("mma_m", ctypes.c_int32),
        ("mma_n", ctypes.c_int32), ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64),
        ("k_blocks", ctypes.c_int64), ("num_tiles", ctypes.c_int64), ("grid", ctypes.c_int64),
        ("threads", ctypes.c_int32), ("group_m", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int64), ("ring_bytes", ctypes.c_int64),
        ("split_k", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
        ("cluster", ctypes.c_int32), ("split_n", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class tg_epilogue_ex_t(ctypes.Structure):
    _fields_ = [
        ("activation", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
    ]


class tg_norm_t(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("stream_dtype", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("post_weight", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
        ("pre_weight", ctypes.c_void_p), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
    ]


class tg_norm_grad_t(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
        ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
        ("dresidual", ctypes.c_void_p), ("lddr", ctypes.c_int64),
        ("dgate", ctypes.c_void_p), ("lddg", ctypes.c_int64),
        ("dpost_weight", ctypes.c_void_p), ("dpre_weight", ctypes.c_void_p),
    ]


class tg_layer_norm_t(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("stream_dtype", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("eps", ctypes.c_float),
    ]


class tg_layer_norm_grad_t(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
        ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
        ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
        ("dresidual", ctypes.c_void_p), ("lddr", ctypes.c_int64),
        ("dweight", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_lib = None
_DTYPES: dict = {}


def _L():
    """Load libtgemm.so on first use; there is no fallback if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libtgemm.so not found at {LIB_PATH}; build it with "
            "`python -m tiled_fp16_gemm_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.tg_gemm_f16.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, ctypes.c_int,
                                _vp]
    lib.tg_gemm_f16.restype = ctypes.c_int
    lib.tg_gemm_bf16.argtypes = lib.tg_gemm_f16.argtypes
    lib.tg_gemm_bf16.restype = ctypes.c_int
    lib.tg_gemm_f16_host.argtypes = lib.tg_gemm_f16.argtypes
    lib.tg_gemm_f16_host.restype = ctypes.c_int
    lib.tg_gemm_ex.argtypes = [ctypes.c_int32, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                               ctypes.POINTER(tg_epilogue_ex_t), _vp]
    lib.tg_gemm_ex.restype = ctypes.c_int
    lib.tg_gemm_mxfp4.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64,
                                  ctypes.POINTER(tg_epilogue_ex_t), _vp]
    lib.tg_gemm_mxfp4.restype = ctypes.c_int
    lib.tg_gemm_sp24.argtypes = [ctypes.c_int32, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                 _i64, _i64, _i64, ctypes.POINTER(tg_epilogue_ex_t), _vp]
    lib.tg_gemm_sp24.restype = ctypes.c_int
    lib.tg_gemm_w4.argtypes = [ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                               ctypes.c_int32, _i64, _i64, _i64, _i64, _i64,
                               ctypes.POINTER(tg_epilogue_ex_t), _vp]
    lib.tg_gemm_w4.restype = ctypes.c_int
    lib.tg_norm_residual.argtypes = [ctypes.POINTER(tg_norm_t), _vp, _i64, _vp, _i64, _vp]
    lib.tg_norm_residual.restype = ctypes.c_int
    lib.tg_norm_residual_backward.argtypes = [ctypes.POINTER(tg_norm_t),
                                              ctypes.POINTER(tg_norm_grad_t), _vp]
    lib.tg_norm_residual_backward.restype = ctypes.c_int
    ln = ctypes.POINTER(tg_layer_norm_t)
    lib.tg_layer_norm.argtypes = [ln, _vp, _i64, _vp, _i64, _vp]
    lib.tg_layer_norm.restype = ctypes.c_int
    lib.tg_layer_norm_i8.argtypes = [ln, _vp, _i64, _vp, _i64, _vp, _vp]
    lib.tg_layer_norm_i8.restype = ctypes.c_int
    lib.tg_quantize_rows.argtypes = [ctypes.c_int32, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp]
    lib.tg_quantize_rows.restype = ctypes.c_int
    lib.tg_layer_norm_backward_workspace.argtypes = [_i64, _i64]
    lib.tg_layer_norm_backward_workspace.restype = _i64
    lib.tg_layer_norm_backward.argtypes = [ln, ctypes.POINTER(tg_layer_norm_grad_t), _vp]
    lib.tg_layer_norm_backward.restype = ctypes.c_int
    lib.tg_gemm_i8_workspace.argtypes = [_i64, _i64, _i64]
    lib.tg_gemm_i8_workspace.restype = _i64
    lib.tg_gemm_i8.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64,
                               ctypes.POINTER(tg_epilogue_ex_t), _vp, _i64, _vp]
    lib.tg_gemm_i8.restype = ctypes.c_int
    lib.tg_sync_status.argtypes = [_vp]
    lib.tg_sync_status.restype = ctypes.c_int
    lib.tg_status_string.argtypes = [ctypes.c_int]
    lib.tg_status_string.restype = ctypes.c_char_p
    lib.tg_version.restype = ctypes.c_char_p
    lib.tg_plan_f16.argtypes = [_i64, _i64, _i64, ctypes.c_int32, ctypes.POINTER(tg_plan_t)]
    lib.tg_plan_f16.restype = ctypes.c_int
    lib.tg_tile_coord.argtypes = [ctypes.POINTER(tg_plan_t), _i64, ctypes.POINTER(_i64),
                                  ctypes.POINTER(_i64)]
    lib.tg_tile_coord.restype = ctypes.c_int
    lib.tg_ring_bytes.argtypes = [ctypes.c_int32] * 5
    lib.tg_ring_bytes.restype = _i64
    lib.tg_debug_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.tg_debug_set_wait_timeout_ns.restype = None
    lib.tg_debug_inject.argtypes = [ctypes.c_int32]
    lib.tg_debug_inject.restype = None
    lib.tg_plan_f16_limits.argtypes = [_i64, _i64, _i64] + [ctypes.c_int32] * 4 + [
        ctypes.POINTER(tg_plan_t)]
    lib.tg_plan_f16_limits.restype = ctypes.c_int
    lib.tg_device_limits.argtypes = [ctypes.POINTER(ctypes.c_int32)] * 4
    lib.tg_device_limits.restype = ctypes.c_int
    lib.tg_debug_last_launch.argtypes = [ctypes.POINTER(tg_plan_t)]
    lib.tg_debug_last_launch.restype = ctypes.c_int
    lib.tg_debug_map_cache_stats.argtypes = [ctypes.POINTER(ctypes.c_uint64)] * 2
    lib.tg_debug_map_cache_stats.restype = None
    _lib = lib
    return lib


def library():
    """The loaded ctypes.CDLL of libtgemm.so."""
    return _L()


class TgemmError(RuntimeError):
    def __init__(self, status: int, what: str = "tg_gemm_f16"):
        self.status = status
        super().__init__(f"{what}: {tg_status_string(status)}")


# ------------------------------------------------------------------ raw C ABI

def tg_gemm_f16(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                epilogue: int, stream: int | None) -> int:
    """The C entry point with integer device pointers; returns the status code."""
    return _L().tg_gemm_f16(A, B, C, M, N, K, lda, ldb, ldc, epilogue, stream or None)


def tg_gemm_bf16(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                 epilogue: int, stream: int | None) -> int:
    """The bfloat16 entry point with integer device pointers; returns the status code."""
    return _L().tg_gemm_bf16(A, B, C, M, N, K, lda, ldb, ldc, epilogue, stream or None)


def tg_gemm_f16_host(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int,
                     ldc: int, epilogue: int, stream: int | None) -> int:
    """The C entry point with integer HOST pointers; returns the status code."""
    return _L().tg_gemm_f16_host(A, B, C, M, N, K, lda, ldb, ldc, epilogue, stream or None)


def tg_gemm_ex(in_dtype: int, A: int, B: int, C: int, M: int, N: int, K: int, lda: int,
               ldb: int, ldc: int, epi: tg_epilogue_ex_t | None, stream: int | None) -> int:
    """C = out(act(A·B + bias) + R) with integer device pointers; returns the status code."""
    return _L().tg_gemm_ex(in_dtype, A, B, C, M, N, K, lda, ldb, ldc,
                           ctypes.byref(epi) if epi is not None else None, stream or None)


def tg_gemm_mxfp4(A: int, Bq: int, Bscale: int, C: int, M: int, N: int, K: int, lda: int,
                  ldbq: int, ldbs: int, ldc: int, epi: tg_epilogue_ex_t | None,
                  stream: int | None) -> int:
    """C = out(act(A·Bdeq + bias) + R) with B in MXFP4 (packed E2M1 codes and
    E8M0 scales per 32 k), integer device pointers; returns the status code."""
    return _L().tg_gemm_mxfp4(A, Bq, Bscale, C, M, N, K, lda, ldbq, ldbs, ldc,
                              ctypes.byref(epi) if epi is not None else None, stream or None)


def tg_gemm_sp24(in_dtype: int, Ac: int, E: int, B: int, C: int, M: int, N: int, K: int,
                 ldac: int, lde: int, ldb: int, ldc: int, epi: tg_epilogue_ex_t | None,
                 stream: int | None) -> int:
    """C = out(act(A·B + bias) + R) with A 2:4 sparse (compressed values Ac and
    metadata words E), integer device pointers; returns the status code."""
    return _L().tg_gemm_sp24(in_dtype, Ac, E, B, C, M, N, K, ldac, lde, ldb, ldc,
                             ctypes.byref(epi) if epi is not None else None, stream or None)


def tg_gemm_w4(in_dtype: int, A: int, Bq: int, Bscale: int, Bzero: int | None, C: int, M: int,
               N: int, K: int, group: int, lda: int, ldbq: int, ldbs: int, ldbz: int, ldc: int,
               epi: tg_epilogue_ex_t | None, stream: int | None) -> int:
    """C = out(act(A·W^T + bias) + R) with W in 4-bit codes and group scales,
    integer device pointers; returns the status code."""
    return _L().tg_gemm_w4(in_dtype, A, Bq, Bscale, Bzero or None, C, M, N, K, group, lda, ldbq,
                           ldbs, ldbz, ldc, ctypes.byref(epi) if epi is not None else None,
                           stream or None)


def tg_norm_residual(n: tg_norm_t, y: int | None, ldy: int, h: int | None, ldh: int,
                     stream: int | None) -> int:
    """The norms around a block with integer device pointers; returns the status code."""
    return _L().tg_norm_residual(ctypes.byref(n), y or None, ldy, h or None, ldh, stream or None)


def tg_norm_residual_backward(n: tg_norm_t, g: tg_norm_grad_t, stream: int | None) -> int:
    """Their gradient with integer device pointers; returns the status code."""
    return _L().tg_norm_residual_backward(ctypes.byref(n), ctypes.byref(g), stream or None)


def tg_layer_norm(n: tg_layer_norm_t, y: int | None, ldy: int, h: int | None, ldh: int,
                  stream: int | None) -> int:
    """The layer norm and its residual sum, integer device pointers; returns the status code."""
    return _L().tg_layer_norm(ctypes.byref(n), y or None, ldy, h or None, ldh, stream or None)


def tg_layer_norm_i8(n: tg_layer_norm_t, y: int | None, ldy: int, codes: int, ldc: int, scale: int,
                     stream: int | None) -> int:
    """The same with its result as 8-bit codes and scales; returns the status code."""
    return _L().tg_layer_norm_i8(ctypes.byref(n), y or None, ldy, codes or None, ldc, scale or None,
                                 stream or None)


def tg_quantize_rows(dtype: int, x: int, ldx: int, codes: int, ldc: int, scale: int, rows: int,
                     cols: int, stream: int | None) -> int:
    """Rows as 8-bit codes with a scale each; returns the status code."""
    return _L().tg_quantize_rows(dtype, x or None, ldx, codes or None, ldc, scale or None, rows, cols,
                                 stream or None)


def tg_layer_norm_backward_workspace(rows: int, cols: int) -> int:
    return _L().tg_layer_norm_backward_workspace(rows, cols)


def tg_layer_norm_backward(n: tg_layer_norm_t, g: tg_layer_norm_grad_t, stream: int | None) -> int:
    """The layer norm's gradient with integer device pointers; returns the status code."""
    return _L().tg_layer_norm_backward(ctypes.byref(n), ctypes.byref(g), stream or None)


def tg_gemm_i8_workspace(M: int, N: int, K: int) -> int:
    return _L().tg_gemm_i8_workspace(M, N, K)


def tg_gemm_i8(A: int, lda: int, Ascale: int, B: int, ldb: int, Bscale: int, C: int, ldc: int,
               M: int, N: int, K: int, epi: tg_epilogue_ex_t | None, workspace: int | None,
               workspace_bytes: int, stream: int | None) -> int:
    """C = out(act(scales · A·B^T + bias) + R) of 8-bit integers, integer device
    pointers; returns the status code."""
    return _L().tg_gemm_i8(A, lda, Ascale or None, B, ldb, Bscale or None, C, ldc, M, N, K,
                           ctypes.byref(epi) if epi is not None else None, workspace or None,
                           workspace_bytes, stream or None)


def tg_sync_status(stream: int | None) -> int:
    return _L().tg_sync_status(stream or None)


def tg_status_string(status: int) -> str:
    return _L().tg_status_string(status).decode()


def tg_version() -> str:
    return _L().tg_version().decode()


def tg_plan_f16(M: int, N: int, K: int, num_sms: int) -> tg_plan_t:
    plan = tg_plan_t()
    st = _L().tg_plan_f16(M, N, K, num_sms, ctypes.byref(plan))
    if st != TG_OK:
        raise TgemmError(st, "tg_plan_f16")
    return plan


def tg_plan_f16_limits(M: int, N: int, K: int, num_sms: int, max_pairs: int,
                       max_quads_narrow: int, max_quads_wide: int) -> tg_plan_t:
    plan = tg_plan_t()
    st = _L().tg_plan_f16_limits(M, N, K, num_sms, max_pairs, max_quads_narrow, max_quads_wide,
                                 ctypes.byref(plan))
    if st != TG_OK:
        raise TgemmError(st, "tg_plan_f16_limits")
    return plan


def tg_device_limits() -> tuple[int, int, int, int]:
    """(num_sms, max_pairs, max_quads_narrow, max_quads_wide) of the current device."""
    v = [ctypes.c_int32() for _ in range(4)]
    st = _L().tg_device_limits(*[ctypes.byref(x) for x in v])
    if st != TG_OK:
        raise TgemmError(st, "tg_device_limits")
    return tuple(x.value for x in v)


def tg_debug_last_launch() -> tg_plan_t:
    plan = tg_plan_t()
    st = _L().tg_debug_last_launch(ctypes.byref(plan))
    if st != TG_OK:
        raise TgemmError(st, "tg_debug_last_launch")
    return plan


def tg_debug_map_cache_stats() -> tuple[int, int]:
    """(hits, misses) of the library's tensor-map cache since it was loaded."""
    h, m = ctypes.c_uint64(), ctypes.c_uint64()
    _L().tg_debug_map_cache_stats(ctypes.byref(h), ctypes.byref(m))
    return h.value, m.value


def tg_tile_coord(plan: tg_plan_t, tile: int) -> tuple[int, int]:
    m, n = _i64(), _i64()
    st = _L().tg_tile_coord(ctypes.byref(plan), tile, ctypes.byref(m), ctypes.byref(n))
    if st != TG_OK:
        raise TgemmError(st, "tg_tile_coord")
    return m.value, n.value


def tg_ring_bytes(bm: int, bn: int, bk: int, stages: int, elem_bytes: int) -> int:
    return _L().tg_ring_bytes(bm, bn, bk, stages, elem_bytes)


def tg_debug_set_wait_timeout_ns(ns: int) -> None:
    _L().tg_debug_set_wait_timeout_ns(ns)


def tg_debug_inject(mode: int) -> None:
    _L().tg_debug_inject(mode)


def tg_gemm_f16_noalloc(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int,
                        ldc: int, epilogue: int, stream: int | None) -> int:
    """C = epi(A·B) for M <= 128 with no device allocation: the split-K
    scratch lives in a fixed 24 MiB array inside the library.  For callers
    that cannot allocate device memory at call time.  Calls that overlap on
    the GPU share that array and race; the first call on a device does a
    one-time set-up and should come before any stream capture.  Returns the
    status code."""
    lib = _L()
    fn = lib.tg_gemm_f16_noalloc
    fn.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _vp]
    fn.restype = ctypes.c_int
    return fn(A, B, C, M, N, K, lda, ldb, ldc, epilogue, stream or None)


# ------------------------------------------------------------------ torch helpers

def _check_operand(t, name: str):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")


def _ld(t) -> int:
    if t.shape[0] > 1:
        return int(t.stride(0))
    # a single row: the row stride is never used, pass the 8-aligned width
    return max(8, (int(t.shape[1]) + 7) // 8 * 8)


def gemm(a, b, relu: bool = False, out=None, stream=None, *, bias=None, residual=None,
         out_dtype=None):
    """C = out(act(a @ b + bias) + residual) for CUDA float16 (or bfloat16)
    tensors a (M×K) and b (K×N); act = ReLU if ``relu`` else identity.

    bias: optional float32 tensor of N elements (added to the fp32
    accumulator before the activation).  residual: optional M×N tensor of a's
    dtype (added after the activation; may be ``out`` itself).  out_dtype:
    a's dtype (default) or torch.float32.  Any row-major 2-D views are
    accepted (unit column stride); ``out`` (M×N) is written in place when
    given.  Runs on ``stream`` (default: torch's current stream of a's device).
    """
    import torch
    _check_operand(a, "a")
    _check_operand(b, "b")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if not (a.is_cuda and b.is_cuda and a.device == b.device):
        raise ValueError("a and b must be CUDA tensors on the same device")
    if a.dtype != b.dtype:
        raise TypeError(f"a and b must share a dtype, got {a.dtype} and {b.dtype}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else a.dtype
    if out_dtype not in (a.dtype, torch.float32):
        raise TypeError(f"out_dtype must be {a.dtype} or torch.float32, got {out_dtype}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    else:
        if out.dtype != out_dtype or out.dim() != 2 or tuple(out.shape) != (M, N) \
                or out.device != a.device:
            raise ValueError("out must be M×N on a's device with dtype out_dtype")
        if N > 1 and out.stride(1) != 1:
            raise ValueError("out must be row-major (unit column stride)")
    extended = bias is not None or residual is not None or out_dtype == torch.float32
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 \
                or bias.device != a.device or bias.numel() != N or bias.dim() != 1 \
                or (N > 1 and bias.stride(0) != 1):
            raise ValueError("bias must be a contiguous float32 CUDA tensor of N elements")
    if residual is not None:
        _check_operand(residual, "residual")
        if residual.dtype != a.dtype or tuple(residual.shape) != (M, N) \
                or residual.device != a.device:
            raise ValueError("residual must be M×N on a's device with a's dtype")
    in_code = TG_DTYPE_BF16 if a.dtype == torch.bfloat16 else TG_DTYPE_F16
    with torch.cuda.device(a.device):
        s = stream if stream is not None else torch.cuda.current_stream(a.device)
        if extended:
            epi = tg_epilogue_ex_t(
                TG_EPI_RELU if relu else TG_EPI_NONE,
                TG_DTYPE_F32 if out_dtype == torch.float32 else in_code,
                bias.data_ptr() if bias is not None else None,
                residual.data_ptr() if residual is not None else None,
                _ld(residual) if residual is not None else 0)
            st = tg_gemm_ex(in_code, a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K,
                            _ld(a), _ld(b), _ld(out), epi, s.cuda_stream)
            what = "tg_gemm_ex"
        else:
            entry = tg_gemm_bf16 if in_code == TG_DTYPE_BF16 else tg_gemm_f16
            st = entry(a.data_ptr(), b.data_ptr(), out.data_ptr(), M, N, K, _ld(a), _ld(b),
                       _ld(out), TG_EPI_RELU if relu else TG_EPI_NONE, s.cuda_stream)
            what = entry.__name__
    if st != TG_OK:
        raise TgemmError(st, what)
    return out


def gemm_mxfp4(a, bq, bscale, N: int, relu: bool = False, out=None, stream=None, *, bias=None,
               residual=None, out_dtype=None):
    """C = out(act(a @ Bdeq + bias) + residual) with the weight in MXFP4.

    a: CUDA float16 tensor M×K (row-major).  bq: CUDA uint8 tensor of N rows
    (one per weight column, the [out][in] orientation) of packed E2M1 codes
    along k, low nibble first (row stride a multiple of 16 bytes, at least
    ceil(K/2)); bscale: CUDA uint8 tensor of ceil(K/32) rows of E8M0 scales
    (row stride a multiple of 16, at least N).  N is the number of weight
    columns.  bias, residual, out_dtype, out and stream as for ``gemm``.
    """
    import torch
    _check_operand(a, "a")
    if a.dtype != torch.float16:
        raise TypeError("a must be float16 for the MXFP4 GEMM")
    M, K = a.shape
    for t, name, rows, width in ((bq, "bq", N, (K + 1) // 2), (bscale, "bscale", (K + 31) // 32, N)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D uint8 tensor")
        if t.shape[0] != rows or t.shape[1] < width or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be {rows} rows of at least {width} bytes, row-major")
        if t.device != a.device:
            raise ValueError(f"{name} must be on a's device")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float16
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be torch.float16 or torch.float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    elif out.dtype != out_dtype or tuple(out.shape) != (M, N) or out.device != a.device:
        raise ValueError("out must be M×N on a's device with dtype out_dtype")
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != N or bias.dim() != 1
                             or bias.device != a.device or (N > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a contiguous float32 CUDA tensor of N elements")
    if residual is not None:
        _check_operand(residual, "residual")
        if residual.dtype != torch.float16 or tuple(residual.shape) != (M, N) \
                or residual.device != a.device:
            raise ValueError("residual must be M×N float16 on a's device")
    epi = tg_epilogue_ex_t(TG_EPI_RELU if relu else TG_EPI_NONE,
                           TG_DTYPE_F32 if out_dtype == torch.float32 else TG_DTYPE_F16,
                           bias.data_ptr() if bias is not None else None,
                           residual.data_ptr() if residual is not None else None,
                           _ld(residual) if residual is not None else 0)
    ldb = lambda t: int(t.stride(0)) if t.shape[0] > 1 else (int(t.shape[1]) + 15) // 16 * 16  # noqa
    with torch.cuda.device(a.device):
        s = stream if stream is not None else torch.cuda.current_stream(a.device)
        st = tg_gemm_mxfp4(a.data_ptr(), bq.data_ptr(), bscale.data_ptr(), out.data_ptr(), M, N,
                           K, _ld(a), ldb(bq), ldb(bscale), _ld(out), epi, s.cuda_stream)
    if st != TG_OK:
        raise TgemmError(st, "tg_gemm_mxfp4")
    return out


def gemm_sp24(ac, e, b, relu: bool = False, out=None, stream=None, *, bias=None, residual=None,
              out_dtype=None):
    """C = out(act(A @ b + bias) + residual) with A 2:4 structured-sparse.

    ac: CUDA float16/bfloat16 tensor M × K/2 of kept values; e: CUDA int32 (or
    uint32 bits in int32) tensor M × K/32 of metadata words; b: K × N of ac's
    dtype.  Rows 16-byte aligned (row strides multiples of 8 elements, 4 words).
    bias, residual, out_dtype, out and stream as for ``gemm``.
    """
    import torch
    _check_operand(ac, "ac")
    _check_operand(b, "b")
    M, half = ac.shape
    K, N = b.shape
    if half * 2 != K or K % 32 != 0:
        raise ValueError("ac must be M × K/2 for b of K rows, K a multiple of 32")
    if ac.dtype != b.dtype:
        raise TypeError("ac and b must share a dtype")
    if not isinstance(e, torch.Tensor) or e.dtype != torch.int32 or e.dim() != 2 \
            or tuple(e.shape) != (M, K // 32) or (K > 32 and e.stride(1) != 1):
        raise ValueError("e must be an int32 tensor of M × K/32 metadata words")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else ac.dtype
    if out_dtype not in (ac.dtype, torch.float32):
        raise TypeError(f"out_dtype must be {ac.dtype} or torch.float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=ac.device)
    in_code = TG_DTYPE_BF16 if ac.dtype == torch.bfloat16 else TG_DTYPE_F16
    epi = tg_epilogue_ex_t(TG_EPI_RELU if relu else TG_EPI_NONE,
                           TG_DTYPE_F32 if out_dtype == torch.float32 else in_code,
                           bias.data_ptr() if bias is not None else None,
                           residual.data_ptr() if residual is not None else None,
                           _ld(residual) if residual is not None else 0)
    lde = int(e.stride(0)) if M > 1 else max(4, (K // 32 + 3) // 4 * 4)
    with torch.cuda.device(ac.device):
        s = stream if stream is not None else torch.cuda.current_stream(ac.device)
        st = tg_gemm_sp24(in_code, ac.data_ptr(), e.data_ptr(), b.data_ptr(), out.data_ptr(), M,
                          N, K, _ld(ac), lde, _ld(b), _ld(out), epi, s.cuda_stream)
    if st != TG_OK:
        raise TgemmError(st, "tg_gemm_sp24")
    return out


# The operators below are also called for single tokens, where this binding's own
# time counts.  A plain call (current stream of the current device, results to be made)
# is checked and made by csrc/calls.cpp; what that does not take comes here, where each
# tensor is looked at once, with few attribute reads.

_torch = None
_plain = None


def _bind():
    """torch, and what of it the operators call for every launch."""
    global _torch, _DTYPES, _get_device, _raw_stream, _plain
    if _torch is None:
        import torch
        lib = _L()
        from . import _calls as calls  # built with libtgemm.so; no fallback if it is missing
        calls.bind(*(ctypes.cast(f, _vp).value for f in
                     (lib.tg_gemm_w4, lib.tg_norm_residual, lib.tg_norm_residual_backward)), NormGrads)
        calls.bind_i8(*(ctypes.cast(f, _vp).value for f in
                        (lib.tg_layer_norm, lib.tg_layer_norm_i8, lib.tg_quantize_rows,
                         lib.tg_layer_norm_backward, lib.tg_layer_norm_backward_workspace,
                         lib.tg_gemm_i8, lib.tg_gemm_i8_workspace)), LayerNormGrads)
        _plain = calls
        _DTYPES = {torch.float16: TG_DTYPE_F16, torch.bfloat16: TG_DTYPE_BF16,
                   torch.float32: TG_DTYPE_F32}
        _get_device = torch.cuda.current_device
        # the stream's handle without a Stream object around it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def _made(result, name: str):
    """What a native call made; a status it returned is raised."""
    if type(result) is int:
        raise TgemmError(result, name)
    return result


def _matrix(t, name: str, dtype, rows: int, cols: int, index: int):
    """(address, row stride) of a rows × cols tensor of ``dtype`` on device ``index``."""
    try:
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be a {dtype} tensor, got {t.dtype}")
        shape = t.shape
        if len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.get_device() != index:
            raise ValueError(f"{name} must be {rows}×{cols} on cuda:{index}")
        stride = t.stride()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major (unit column stride)")
    # a single row's stride is never used
    return t.data_ptr(), stride[0] if rows > 1 else (cols + 15) // 16 * 16


def _vector(t, name: str, size: int, index: int) -> int:
    """Address of a contiguous float32 vector of ``size`` elements."""
    try:
        shape = t.shape
        if t.dtype is _torch.float32 and len(shape) == 1 and shape[0] == size \
                and t.get_device() == index and (size < 2 or t.stride()[0] == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {size} elements")


def _on_stream(index: int, stream, used, body):
    """``body(raw stream)`` where it is not just the current stream of the current
    device: with device ``index`` current, and its allocations made on the stream
    that it launches on.  ``used``: the caller's tensors, kept from reuse until that
    stream is done with them where it is not the current one."""
    torch = _torch
    with torch.cuda.device(index):
        if stream is None:
            return body(_raw_stream(index))
        here = torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            made = body(stream.cuda_stream)
        if here.cuda_stream != stream.cuda_stream:
            for t in used:
                if t is not None:
                    t.record_stream(stream)
            for t in made if isinstance(made, tuple) else (made,):
                if t is not None:
                    t.record_stream(here)
    return made


def gemm_w4(a, bq, bscale, N: int, group: int, relu: bool = False, out=None, stream=None, *,
            bzero=None, bias=None, residual=None, out_dtype=None):
    """C = out(act(a @ W.T + bias) + residual) with the weight W (N × K) in
    4-bit codes: W[n][k] = (code[n][k] - zero[k // group][n]) · scale[k // group][n].

    a: CUDA float16 or bfloat16 tensor M×K (row-major).  bq: CUDA uint8 tensor
    of N rows of packed codes along k, low nibble first (row stride a multiple
    of 16 bytes, at least ceil(K/2)).  group: 32, 64 or 128.  bscale: tensor of
    a's dtype, ceil(K/group) rows of N scales (row stride a multiple of 8).
    bzero: optional uint8 tensor of ceil(K/group) rows of N zero points 0..15
    (row stride a multiple of 16); without it every zero point is 8.  bias,
    residual, out_dtype, out and stream as for ``gemm``.
    """
    torch = _torch or _bind()
    if out is None and stream is None:
        made = _plain.gemm_w4(a, bq, bscale, N, group, relu, bzero, bias, residual, out_dtype)
        if made is not None:
            return _made(made, "tg_gemm_w4")
    try:
        dtype = a.dtype
        M, K = a.shape
        index = a.get_device()
    except (AttributeError, ValueError):
        _check_operand(a, "a")
        raise
    if dtype is not torch.float16 and dtype is not torch.bfloat16 or index < 0:
        _check_operand(a, "a")
        raise ValueError("a must be a CUDA tensor")
    pa, lda = _matrix(a, "a", dtype, M, K, index)
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    groups = (K + group - 1) // group

    def rows_of(t, name, kind, rows, width):  # rows of at least `width`
        try:
            if t.dtype is not kind:
                raise TypeError(f"{name} must be a 2-D {kind} tensor, got {t.dtype}")
            have = t.shape[-1]
        except (AttributeError, IndexError):
            raise TypeError(f"{name} must be a 2-D {kind} tensor") from None
        if have < width:
            raise ValueError(f"{name} must be {rows} rows of at least {width}, row-major")
        return _matrix(t, name, kind, rows, have, index)

    pq, ldq = rows_of(bq, "bq", torch.uint8, N, (K + 1) // 2)
    ps, lds = rows_of(bscale, "bscale", dtype, groups, N)
    pz, ldz = rows_of(bzero, "bzero", torch.uint8, groups, N) if bzero is not None else (None, 0)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be {dtype} or torch.float32, got {out_dtype}")
    if out is not None:
        pc, ldc = _matrix(out, "out", out_dtype, M, N, index)
    pb = _vector(bias, "bias", N, index) if bias is not None else None
    pr, ldr = _matrix(residual, "residual", dtype, M, N, index) if residual is not None else (None, 0)
    code = _DTYPES[dtype]
    epi = tg_epilogue_ex_t(1 if relu else 0, _DTYPES[out_dtype], pb, pr, ldr)

    def body(s):
        c = torch.empty((M, N), dtype=out_dtype, device=a.device) if out is None else out
        st = _lib.tg_gemm_w4(code, pa, pq, ps, pz, c.data_ptr(), M, N, K, group, lda, ldq, lds, ldz,
                             N if out is None else ldc, ctypes.byref(epi), s)
        if st != TG_OK:
            raise TgemmError(st, "tg_gemm_w4")
        return c

    return _on_stream(index, stream, (a, bq, bscale, bzero, bias, residual, out), body)


def _norm_args(x, residual, post_weight, gate, scale, pre_weight, eps):
    """Checks and packs what the norms and their gradient share."""
    torch = _torch or _bind()
    try:
        dtype = x.dtype
        rows, cols = x.shape
        index = x.get_device()
    except AttributeError:
        raise TypeError("x must be a torch.Tensor") from None
    except ValueError:
        raise ValueError("x must be 2-D") from None
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {dtype}")
    if index < 0:
        raise ValueError("x must be a CUDA tensor")
    if cols > 32768:
        raise ValueError(f"x must have at most 32768 columns, got {cols}")
    px, ldx = _matrix(x, "x", dtype, rows, cols, index)
    kind, kind_code, pr, ldr = dtype, code, None, 0
    if residual is not None:
        kind = getattr(residual, "dtype", None)
        if kind is not dtype:
            if kind is not torch.float32:
                raise TypeError(f"residual must be a {dtype} or float32 tensor")
            kind_code = TG_DTYPE_F32
        pr, ldr = _matrix(residual, "residual", kind, rows, cols, index)
    pg, ldg, gate_rows = None, 0, 0
    if gate is not None:
        try:
            shape = gate.shape
        except AttributeError:
            raise TypeError(f"gate must be a {dtype} tensor") from None
        if len(shape) == 1:
            gate_rows = 1
            pg, ldg = _matrix(gate.unsqueeze(0), "gate", dtype, 1, cols, index)
        else:
            gate_rows = shape[0]
            pg, ldg = _matrix(gate, "gate", dtype, gate_rows, cols, index)
        if gate_rows < 1 or (rows > 0 and (gate_rows > rows or rows % gate_rows)):
            raise ValueError(f"the gate's {gate_rows} rows must divide x's {rows}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    n = tg_norm_t(
        code, kind_code, rows, cols, px, ldx, pr, ldr,
        _vector(post_weight, "post_weight", cols, index) if post_weight is not None else None,
        pg, ldg, gate_rows,
        _vector(pre_weight, "pre_weight", cols, index) if pre_weight is not None else None,
        scale, eps)
    return n, rows, cols, dtype, kind, index


def norm_residual(x, residual=None, *, post_weight=None, gate=None, scale: float = 1.0,
                  pre_weight=None, eps: float = 1e-6, out=None, normed=None, stream=None):
    """The norms after and before a block with its gate and residual scale:

        y = residual + scale · gate ⊙ rms(x)·post_weight,   h = rms(y)·pre_weight

    with rms(v) = v / sqrt(mean(v²) + eps) over each row.  Returns (y, h).

    x: CUDA float16, bfloat16 or float32 tensor of rows × cols (the block's
    output).  residual: optional tensor of x's dtype or float32; y has its dtype.
    post_weight, pre_weight: optional float32 vectors of cols; without
    post_weight x is taken as it is, without pre_weight h is None.  gate:
    optional tensor of x's dtype, cols values for all rows or G rows of them,
    each for rows / G consecutive rows of x.  y is written to ``out`` (which may
    be ``residual`` itself) and h to ``normed`` where given.  Runs on ``stream``
    (default: torch's current stream of x's device).  Like every result of this
    library y and h carry no autograd graph: their gradient is
    ``norm_residual_backward``.
    """
    if _torch is None:
        _bind()
    if out is None and normed is None and stream is None:
        made = _plain.norm_residual(x, residual, post_weight, gate, scale, pre_weight, eps)
        if made is not None:
            return _made(made, "tg_norm_residual")
    n, rows, cols, dtype, kind, index = _norm_args(x, residual, post_weight, gate, scale,
                                                   pre_weight, eps)
    torch = _torch
    py = ph = None
    if out is not None:
        py, ldy = _matrix(out, "out", kind, rows, cols, index)
    if normed is not None:
        if pre_weight is None:
            raise ValueError("normed needs pre_weight")
        ph, ldh = _matrix(normed, "normed", dtype, rows, cols, index)

    def body(s):
        shape, device = (rows, cols), x.device
        y, h = out, normed
        y_at, y_ld, h_at, h_ld = py, cols, ph, cols
        if y is None:
            y = torch.empty(shape, dtype=kind, device=device)
            y_at = y.data_ptr()
        else:
            y_ld = ldy
        if h is not None:
            h_ld = ldh
        elif pre_weight is not None:
            h = torch.empty(shape, dtype=dtype, device=device)
            h_at = h.data_ptr()
        st = _lib.tg_norm_residual(ctypes.byref(n), y_at, y_ld, h_at, h_ld, s)
        if st != TG_OK:
            raise TgemmError(st, "tg_norm_residual")
        return y, h

    if stream is None and index == _get_device():
        return body(_raw_stream(index))
    return _on_stream(index, stream, (x, residual, post_weight, gate, pre_weight, out, normed), body)


class NormGrads(NamedTuple):
    """Gradients of ``norm_residual``; None for an input that was not given."""
    x: object
    residual: object
    gate: object
    post_weight: object
    pre_weight: object


def norm_residual_backward(dy, dh, x, residual=None, *, post_weight=None, gate=None,
                           scale: float = 1.0, pre_weight=None, eps: float = 1e-6, stream=None):
    """The gradients of ``norm_residual`` called with the same arguments, given
    dy and dh, the gradients of its two results (either may be None: zero).

    dy has residual's dtype, dh x's.  Returns NormGrads, each gradient with its
    input's dtype and shape.  x and residual are those of the forward call: no
    ``out`` may have been written over them.
    """
    if _torch is None:
        _bind()
    if stream is None:
        made = _plain.norm_residual_backward(dy, dh, x, residual, post_weight, gate, scale,
                                             pre_weight, eps)
        if made is not None:
            return _made(made, "tg_norm_residual_backward")
    n, rows, cols, dtype, kind, index = _norm_args(x, residual, post_weight, gate, scale,
                                                   pre_weight, eps)
    torch = _torch
    pdy, lddy = _matrix(dy, "dy", kind, rows, cols, index) if dy is not None else (None, 0)
    pdh, lddh = None, 0
    if dh is not None:
        if pre_weight is None:
            raise ValueError("dh needs pre_weight")
        pdh, lddh = _matrix(dh, "dh", dtype, rows, cols, index)

    def body(s):
        empty, shape, device = torch.empty, (rows, cols), x.device
        dx = empty(shape, dtype=dtype, device=device)
        dr = dg = dpost = dpre = at_r = at_g = at_post = at_pre = None
        if residual is not None:
            dr = empty(shape, dtype=kind, device=device)
            at_r = dr.data_ptr()
        if gate is not None:
            dg = empty(gate.shape, dtype=dtype, device=device)
            at_g = dg.data_ptr()
        if post_weight is not None:
            dpost = empty(cols, dtype=torch.float32, device=device)
            at_post = dpost.data_ptr()
        if pre_weight is not None:
            dpre = empty(cols, dtype=torch.float32, device=device)
            at_pre = dpre.data_ptr()
        g = tg_norm_grad_t(pdy, lddy, pdh, lddh, dx.data_ptr(), cols, at_r, cols, at_g, cols,
                           at_post, at_pre)
        st = _lib.tg_norm_residual_backward(ctypes.byref(n), ctypes.byref(g), s)
        if st != TG_OK:
            raise TgemmError(st, "tg_norm_residual_backward")
        return NormGrads(dx, dr, dg, dpost, dpre)

    if stream is None and index == _get_device():
        return body(_raw_stream(index))
    return _on_stream(index, stream, (dy, dh, x, residual, post_weight, gate, pre_weight), body)

def _layer_norm_args(x, residual, weight, bias, eps):
    """Checks and packs what the layer norm's calls share."""
    if _torch is None:
        _bind()
    try:
        dtype = x.dtype
        rows, cols = x.shape
        index = x.get_device()
    except AttributeError:
        raise TypeError("x must be a torch.Tensor") from None
    except ValueError:
        raise ValueError("x must be 2-D") from None
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"x must be float16, bfloat16 or float32, got {dtype}")
    if index < 0:
        raise ValueError("x must be a CUDA tensor")
    if cols > 131071:
        raise ValueError(f"x must have at most 131071 columns, got {cols}")
    px, ldx = _matrix(x, "x", dtype, rows, cols, index)
    kind, kind_code, pr, ldr = dtype, code, None, 0
    if residual is not None:
        kind = getattr(residual, "dtype", None)
        if kind is not dtype:
            if kind is not _torch.float32:
                raise TypeError(f"residual must be a {dtype} or float32 tensor")
            kind_code = TG_DTYPE_F32
        pr, ldr = _matrix(residual, "residual", kind, rows, cols, index)
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    n = tg_layer_norm_t(
        code, kind_code, rows, cols, px, ldx, pr, ldr,
        _vector(weight, "weight", cols, index) if weight is not None else None,
        _vector(bias, "bias", cols, index) if bias is not None else None, eps)
    return n, rows, cols, dtype, kind, index


def layer_norm(x, residual=None, *, weight=None, bias=None, eps: float = 1e-5, out=None, normed=None,
               stream=None):
    """Layer norm with the residual sum before it:

        y = residual + x,   h = (y - mean(y)) / sqrt(var(y) + eps) · weight + bias

    over each row (var: the mean of the squared differences).  Returns (y, h); without
    residual h is the norm of x, and y is None.

    x: CUDA float16, bfloat16 or float32 tensor of rows × cols.  residual: optional
    tensor of x's dtype or float32; y has its dtype.  weight, bias: optional float32
    vectors of cols.  h has x's dtype, and comes from y before it is rounded.  y is
    written to ``out`` (which may be ``residual`` itself) and h to ``normed`` where given.
    Runs on ``stream`` (default: torch's current stream of x's device).  Like every result
    of this library y and h carry no autograd graph: their gradient is
    ``layer_norm_backward``.
    """
    if _torch is None:
        _bind()
    if out is None and normed is None and stream is None:
        made = _plain.layer_norm(x, residual, weight, bias, eps)
        if made is not None:
            return _made(made, "tg_layer_norm")
    n, rows, cols, dtype, kind, index = _layer_norm_args(x, residual, weight, bias, eps)
    torch = _torch
    py = ph = None
    if out is not None:
        if residual is None:
            raise ValueError("out needs residual")
        py, ldy = _matrix(out, "out", kind, rows, cols, index)
    if normed is not None:
        ph, ldh = _matrix(normed, "normed", dtype, rows, cols, index)

    def body(s):
        y, h = out, normed
        y_at, y_ld, h_at, h_ld = py, cols, ph, cols
        if y is not None:
            y_ld = ldy
        elif residual is not None:
            y = torch.empty((rows, cols), dtype=kind, device=x.device)
            y_at = y.data_ptr()
        if h is not None:
            h_ld = ldh
        else:
            h = torch.empty((rows, cols), dtype=dtype, device=x.device)
            h_at = h.data_ptr()
        st = _lib.tg_layer_norm(ctypes.byref(n), y_at, y_ld, h_at, h_ld, s)
        if st != TG_OK:
            raise TgemmError(st, "tg_layer_norm")
        return y, h

    return _on_stream(index, stream, (x, residual, weight, bias, out, normed), body)


def _codes(rows: int, cols: int, device):
    """An int8 tensor whose rows begin on 16 bytes."""
    return _torch.empty_strided((rows, cols), ((cols + 15) // 16 * 16, 1), dtype=_torch.int8,
                                device=device)


def layer_norm_i8(x, residual=None, *, weight=None, bias=None, eps: float = 1e-5, out=None,
                  stream=None):
    """``layer_norm`` with its result in 8-bit codes, for ``gemm_i8``: (y, codes, scale).

    codes and scale are those of ``quantize_rows`` for h before it is rounded.  All
    arguments as for ``layer_norm``.
    """
    if _torch is None:
        _bind()
    if out is None and stream is None:
        made = _plain.layer_norm_i8(x, residual, weight, bias, eps)
        if made is not None:
            return _made(made, "tg_layer_norm_i8")
    n, rows, cols, dtype, kind, index = _layer_norm_args(x, residual, weight, bias, eps)
    torch = _torch
    py = None
    if out is not None:
        if residual is None:
            raise ValueError("out needs residual")
        py, ldy = _matrix(out, "out", kind, rows, cols, index)

    def body(s):
        y, y_at, y_ld = out, py, cols
        if y is not None:
            y_ld = ldy
        elif residual is not None:
            y = torch.empty((rows, cols), dtype=kind, device=x.device)
            y_at = y.data_ptr()
        codes = _codes(rows, cols, x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        if cols == 0:
            scale.zero_()
        st = _lib.tg_layer_norm_i8(ctypes.byref(n), y_at, y_ld, codes.data_ptr(),
                                   (cols + 15) // 16 * 16, scale.data_ptr(), s)
        if st != TG_OK:
            raise TgemmError(st, "tg_layer_norm_i8")
        return y, codes, scale

    return _on_stream(index, stream, (x, residual, weight, bias, out), body)


def quantize_rows(x, *, stream=None):
    """Each row of x as 8-bit codes with a scale, for ``gemm_i8``: (codes, scale) with
    scale[i] = max|x[i]| / 127 and codes[i] = x[i] / scale[i] to the nearest whole number
    (ties to even).

    x: CUDA float16, bfloat16 or float32 tensor of rows × cols (at most 131071).  codes:
    int8, rows × cols, whose rows begin on 16 bytes; scale: float32, rows values.  A row
    of zeros has scale 0; a row with a NaN or an infinity has scale NaN and codes 0, so
    that its products are NaN.  Runs on ``stream`` (default: torch's current stream of
    x's device).
    """
    if _torch is None:
        _bind()
    if stream is None:
        made = _plain.quantize_rows(x)
        if made is not None:
            return _made(made, "tg_quantize_rows")
    n, rows, cols, _, _, index = _layer_norm_args(x, None, None, None, 0.0)
    torch = _torch

    def body(s):
        codes = _codes(rows, cols, x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        if cols == 0:
            scale.zero_()
        st = _lib.tg_quantize_rows(n.dtype, n.x, n.ldx, codes.data_ptr(), (cols + 15) // 16 * 16,
                                   scale.data_ptr(), rows, cols, s)
        if st != TG_OK:
            raise TgemmError(st, "tg_quantize_rows")
        return codes, scale

    return _on_stream(index, stream, (x,), body)


class LayerNormGrads(NamedTuple):
    """Gradients of ``layer_norm``; None for an input that was not given."""
    x: object
    residual: object
    weight: object
    bias: object


def layer_norm_backward(dy, dh, x, residual=None, *, weight=None, bias=None, eps: float = 1e-5,
                        stream=None):
    """The gradients of ``layer_norm`` called with the same arguments, given dy and dh, the
    gradients of its two results (either may be None: zero).  Without residual dy is what
    else x receives (where it goes on beside its norm).

    dy has residual's dtype (x's without one), dh x's.  Returns LayerNormGrads, each gradient
    with its input's dtype and shape.  x and residual are those of the forward call: no
    ``out`` may have been written over them.
    """
    if _torch is None:
        _bind()
    if stream is None:
        made = _plain.layer_norm_backward(dy, dh, x, residual, weight, bias, eps)
        if made is not None:
            return _made(made, "tg_layer_norm_backward")
    n, rows, cols, dtype, kind, index = _layer_norm_args(x, residual, weight, bias, eps)
    torch = _torch
    pdy, lddy = _matrix(dy, "dy", kind, rows, cols, index) if dy is not None else (None, 0)
    pdh, lddh = _matrix(dh, "dh", dtype, rows, cols, index) if dh is not None else (None, 0)

    def body(s):
        empty, shape, device = torch.empty, (rows, cols), x.device
        dx = empty(shape, dtype=dtype, device=device)
        dr = empty(shape, dtype=kind, device=device) if residual is not None else None
        dw = empty(cols, dtype=torch.float32, device=device) if weight is not None else None
        db = empty(cols, dtype=torch.float32, device=device) if bias is not None else None
        size = _lib.tg_layer_norm_backward_workspace(rows, cols)
        # (of this call's own: graphs captured on one stream share none)
        work = empty(size, dtype=torch.uint8, device=device)
        at = [t.data_ptr() if t is not None else None for t in (dx, dr, dw, db)]
        g = tg_layer_norm_grad_t(pdy, lddy, pdh, lddh, at[0], cols, at[1], cols, at[2], at[3],
                                 work.data_ptr() or None, size)
        st = _lib.tg_layer_norm_backward(ctypes.byref(n), ctypes.byref(g), s)
        if st != TG_OK:
            raise TgemmError(st, "tg_layer_norm_backward")
        return LayerNormGrads(dx, dr, dw, db)

    return _on_stream(index, stream, (dy, dh, x, residual, weight), body)


def gemm_i8(a, b, ascale, bscale, relu: bool = False, out=None, stream=None, *, bias=None,
            residual=None, out_dtype=None):
    """C = out(act(ascale[m] · bscale[n] · (a @ b.T) + bias) + residual) of 8-bit integers
    with a scale per row of a (token) and per row of b (channel).  The sums a @ b.T are
    exact; scales, bias and residual are applied in fp32, and C is rounded once.

    a: CUDA int8 tensor M×K (unit column stride), for instance the codes of ``quantize_rows``
    or ``layer_norm_i8``.  b: CUDA int8 tensor N×K, the [out][in] orientation of a weight,
    each row on 16 bytes (row stride a multiple of 16).  K is 131071 at most.  ascale, bscale:
    float32 vectors of M and N.  out_dtype: float16, bfloat16 or float32 (default: that of
    ``out``, else of residual, else float16).  bias: optional float32 tensor of N elements.
    residual: optional M×N tensor of C's dtype, added after the activation (may be ``out``
    itself).  ``out`` (M×N) is written in place when given.  Runs on ``stream`` (default:
    torch's current stream of a's device).
    """
    if _torch is None:
        _bind()
    if out is None and stream is None:
        made = _plain.gemm_i8(a, b, ascale, bscale, relu, bias, residual, out_dtype)
        if made is not None:
            return _made(made, "tg_gemm_i8")
    torch = _torch
    try:
        M, K = a.shape
        index = a.get_device()
    except AttributeError:
        raise TypeError("a must be a torch.Tensor") from None
    except ValueError:
        raise ValueError("a must be 2-D") from None
    if index < 0:
        raise ValueError("a must be a CUDA tensor")
    pa, lda = _matrix(a, "a", torch.int8, M, K, index)
    if K > 131071:
        raise ValueError(f"a must have at most 131071 columns, got {K}")
    try:
        N = b.shape[0]
    except (AttributeError, IndexError):
        raise TypeError("b must be a 2-D torch.int8 tensor") from None
    pb, ldb = _matrix(b, "b", torch.int8, N, K, index)
    psa, psb = _vector(ascale, "ascale", M, index), _vector(bscale, "bscale", N, index)
    if out_dtype is None:
        given = out if out is not None else residual
        out_dtype = given.dtype if given is not None else torch.float16
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    if out is not None:
        pc, ldc = _matrix(out, "out", out_dtype, M, N, index)
    pbias = _vector(bias, "bias", N, index) if bias is not None else None
    pr, ldr = _matrix(residual, "residual", out_dtype, M, N, index) if residual is not None else (None, 0)
    epi = tg_epilogue_ex_t(1 if relu else 0, code, pbias, pr, ldr)

    def body(s):
        c = torch.empty((M, N), dtype=out_dtype, device=a.device) if out is None else out
        size = _lib.tg_gemm_i8_workspace(M, N, K)
        # (of this call's own: graphs captured on one stream share none)
        work = torch.empty(size, dtype=torch.uint8, device=a.device) if size > 0 else None
        st = _lib.tg_gemm_i8(pa, lda, psa, pb, ldb, psb, c.data_ptr(), N if out is None else ldc, M, N,
                             K, ctypes.byref(epi), work.data_ptr() if work is not None else None, size, s)
        if st != TG_OK:
            raise TgemmError(st, "tg_gemm_i8")
        return c

    return _on_stream(index, stream, (a, b, ascale, bscale, bias, residual, out), body)



def gemm_host(a, b, relu: bool = False, stream=None, device=None):
    """End-to-end C = epi(a @ b) from host (CPU) float16 tensors, through
    tg_gemm_f16_host: the library uploads a and B and downloads C block by
    block on its own copy streams, overlapped with the products.  Returns C
    in a pinned host tensor once it is complete.  Pinned a and b let the
    copies overlap; pageable ones work, without overlap.
    """
    import torch
    for t, name in ((a, "a"), (b, "b")):
        if t.device.type != "cpu" or t.dtype != torch.float16 or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D float16 CPU tensor")
        if t.stride(1) != 1:
            raise ValueError(f"{name} must have unit column stride")
    M, K = a.shape
    if b.shape[0] != K:
        raise ValueError(f"inner sizes differ: a is {tuple(a.shape)}, b is {tuple(b.shape)}")
    N = b.shape[1]
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    hc = torch.empty((M, N), dtype=torch.float16, pin_memory=True)
    with torch.cuda.device(dev):
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        st = tg_gemm_f16_host(a.data_ptr(), b.data_ptr(), hc.data_ptr(), M, N, K,
                              max(a.stride(0), 1), max(b.stride(0), 1), max(N, 1),
                              TG_EPI_RELU if relu else TG_EPI_NONE, s.cuda_stream)
        if st != TG_OK:
            raise TgemmError(st, "tg_gemm_f16_host")
        st = tg_sync_status(s.cuda_stream)
        if st != TG_OK:
            raise TgemmError(st, "tg_sync_status")
    return hc


def sync_status(stream=None) -> None:
    """Wait for the stream and raise TgemmError if a kernel reported a timeout."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    st = tg_sync_status(s.cuda_stream)
    if st != TG_OK:
        raise TgemmError(st, "tg_sync_status")
