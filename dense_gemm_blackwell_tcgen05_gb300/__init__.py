"""Python binding of the GB300 tcgen05 GEMM library (``include/gemm_gb300.h``).

Argument marshalling only: every step of the GEMM runs in the CUDA library's
own kernels.  The entry points keep the C names and arguments (raw device
pointers as integers, sizes, leading dimensions in elements, a CUDA stream
handle); ``matmul_bf16`` / ``matmul_mxfp8``, ``matmul_grouped`` with its two
gradients, ``newton_schulz``, ``matmul_cross_entropy`` and ``matmul_distill``
with their gradients are conveniences that take torch CUDA tensors, call the same entry points on the current stream (or on ``stream``,
which the caller orders with the tensors' other uses) and raise on a non-zero
status.  There is no CPU or library fallback: when the CUDA
library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import threading

from . import _build

__all__ = [
    "GEMM_OK", "GEMM_ERR_INVALID_ARG", "GEMM_ERR_ALIGNMENT", "GEMM_ERR_UNSUPPORTED_DEVICE",
    "GEMM_ERR_LAUNCH", "GEMM_ERR_TIMEOUT", "GEMM_ERR_DEVICE_FAULT",
    "VARIANT_AUTO", "VARIANT_1CTA", "VARIANT_2CTA", "VARIANT_SYNC", "VARIANT_SMALLK",
    "VARIANT_SMALLK_TC",
    "VARIANT_DIRECT_STORE",
    "GemmError", "load", "library_path", "EXPORTED_SYMBOLS",
    "gemm_bf16", "gemm_bf16_variant", "gemm_mxfp8", "gemm_mxfp8_variant", "gemm_mxfp8_tiled",
    "matmul_mxfp8_tiled", "gemm_mxfp8_quantize_tiled", "quantize_mxfp8_tiled", "gemm_last_status", "gemm_last_status_word", "gemm_status_string", "gemm_set_watchdog_ms",
    "gemm_kernel_plan", "gemm_last_cuda_error", "gemm_debug_stall_next_launch",
    "gemm_mxfp8_quantize", "quantize_mxfp8", "gemm_bf16_streamk", "gemm_mxfp8_streamk",
    "gemm_streamk_workspace_bytes", "gemm_last_schedule", "streamk_workspace",
    "gemm_bf16_streamk_noalloc", "gemm_set_streamk_mode", "STREAMK_AUTO", "STREAMK_ALWAYS",
    "STREAMK_NEVER", "gemm_streamk_plan", "gemm_set_tail_split", "gemm_tail_split_plan",
    "gemm_set_edge_last", "gemm_bf16_fused", "gemm_mxfp8_fused", "GemmEpilogue",
    "make_epilogue", "matmul_fused", "DTYPE_BF16", "DTYPE_F32", "ACT_NONE", "ACT_RELU", "ACT_GELU", "matmul_bf16",
    "matmul_mxfp8", "MAX_GROUPS", "gemm_bf16_grouped", "gemm_bf16_grouped_dgrad",
    "gemm_bf16_grouped_wgrad", "matmul_grouped", "matmul_grouped_dgrad", "matmul_grouped_wgrad",
    "NEWTON_SCHULZ_COEFFICIENTS", "gemm_newton_schulz", "gemm_newton_schulz_workspace_bytes",
    "newton_schulz", "newton_schulz_workspace",
    "INDEX_I32", "INDEX_I64", "MAX_TOP", "gemm_bf16_cross_entropy", "gemm_bf16_cross_entropy_grad",
    "gemm_bf16_cross_entropy_workspace_bytes", "gemm_bf16_distill", "gemm_bf16_distill_grad",
    "gemm_bf16_distill_workspace_bytes", "matmul_cross_entropy", "matmul_cross_entropy_grad",
    "cross_entropy_workspace", "matmul_distill", "matmul_distill_grad", "distill_workspace",
]

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = -1
GEMM_ERR_ALIGNMENT = -2
GEMM_ERR_UNSUPPORTED_DEVICE = -3
GEMM_ERR_LAUNCH = -4
GEMM_ERR_TIMEOUT = -5
GEMM_ERR_DEVICE_FAULT = -6

VARIANT_AUTO = 0
VARIANT_1CTA = 1
VARIANT_2CTA = 2
VARIANT_SYNC = 3
VARIANT_SMALLK = 4
VARIANT_SMALLK_TC = 5
VARIANT_DIRECT_STORE = 0x100

# Every function include/gemm_gb300.h declares.
EXPORTED_SYMBOLS = (
    "gemm_bf16", "gemm_bf16_variant", "gemm_mxfp8", "gemm_mxfp8_variant", "gemm_last_status",
    "gemm_last_status_word", "gemm_status_string", "gemm_set_watchdog_ms", "gemm_kernel_plan",
    "gemm_last_cuda_error", "gemm_debug_stall_next_launch", "gemm_mxfp8_quantize",
    "gemm_bf16_streamk", "gemm_mxfp8_streamk", "gemm_streamk_workspace_bytes",
    "gemm_last_schedule", "gemm_bf16_streamk_noalloc", "gemm_set_streamk_mode",
    "gemm_streamk_plan", "gemm_bf16_fused", "gemm_mxfp8_fused", "gemm_mxfp8_tiled",
    "gemm_mxfp8_quantize_tiled", "gemm_set_tail_split", "gemm_tail_split_plan",
    "gemm_set_edge_last", "gemm_bf16_grouped", "gemm_bf16_grouped_dgrad", "gemm_bf16_grouped_wgrad",
    "gemm_newton_schulz", "gemm_newton_schulz_workspace_bytes",
    "gemm_bf16_cross_entropy", "gemm_bf16_cross_entropy_grad",
    "gemm_bf16_cross_entropy_workspace_bytes", "gemm_bf16_distill", "gemm_bf16_distill_grad",
    "gemm_bf16_distill_workspace_bytes",
)

_lock = threading.Lock()
_lib = None
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        if status == GEMM_ERR_LAUNCH:
            what = f"{what} (cuda error {gemm_last_cuda_error()})"
        super().__init__(f"{what}: {gemm_status_string(status)} ({status})" if what
                         else f"{gemm_status_string(status)} ({status})")


def library_path() -> str:
    return _build.LIB_PATH


DTYPE_BF16, DTYPE_F32 = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU = 0, 1, 2


class GemmEpilogue(ctypes.Structure):
    """Mirror of gemm_epilogue_t: D = act(alpha acc + beta C + bias[col])."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("C", ctypes.c_void_p),
                ("ldc", ctypes.c_int64), ("bias", ctypes.c_void_p), ("bias_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def load() -> ctypes.CDLL:
    """Load the CUDA library, building it in-tree first if it is missing or
    older than its sources.  Raises if it cannot be built or loaded."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            L = ctypes.CDLL(path)
            L.gemm_bf16.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp]
            L.gemm_bf16_variant.argtypes = [ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                            _i64, _i64, _vp]
            L.gemm_mxfp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                                     _i64, _i64, _vp]
            L.gemm_mxfp8_variant.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                             _i64, _i64, _i64, _i64, _i64, _i64, _vp]
            L.gemm_mxfp8_tiled.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                           _i64, _i64, _i64, _vp]
            for name in ("gemm_bf16", "gemm_bf16_variant", "gemm_mxfp8", "gemm_mxfp8_variant",
                         "gemm_mxfp8_tiled"):
                getattr(L, name).restype = ctypes.c_int
            L.gemm_bf16_streamk.argtypes = [ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                            _i64, _i64, _vp, _i64, _vp]
            L.gemm_bf16_streamk.restype = ctypes.c_int
            L.gemm_mxfp8_streamk.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                             _i64, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp]
            L.gemm_mxfp8_streamk.restype = ctypes.c_int
            L.gemm_streamk_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
            L.gemm_streamk_workspace_bytes.restype = _i64
            L.gemm_bf16_streamk_noalloc.argtypes = [ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64,
                                                    _i64, _i64, _i64, _vp]
            L.gemm_bf16_streamk_noalloc.restype = ctypes.c_int
            L.gemm_bf16_fused.argtypes = [ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                                          _i64, ctypes.POINTER(GemmEpilogue), _vp]
            L.gemm_bf16_fused.restype = ctypes.c_int
            L.gemm_mxfp8_fused.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                           _i64, _i64, _i64, _i64, _i64,
                                           ctypes.POINTER(GemmEpilogue), _vp]
            L.gemm_mxfp8_fused.restype = ctypes.c_int
            L.gemm_streamk_plan.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int,
                                            ctypes.POINTER(_i64)]
            L.gemm_streamk_plan.restype = ctypes.c_int
            L.gemm_set_streamk_mode.argtypes = [ctypes.c_int]
            L.gemm_set_streamk_mode.restype = ctypes.c_int
            L.gemm_last_schedule.argtypes = [ctypes.POINTER(_i64)]
            L.gemm_last_schedule.restype = ctypes.c_int
            L.gemm_set_tail_split.argtypes = [ctypes.c_int]
            L.gemm_set_tail_split.restype = ctypes.c_int
            L.gemm_set_edge_last.argtypes = [ctypes.c_int]
            L.gemm_set_edge_last.restype = ctypes.c_int
            L.gemm_tail_split_plan.argtypes = [_i64, _i64]
            L.gemm_tail_split_plan.restype = _i64
            L.gemm_mxfp8_quantize.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]
            L.gemm_mxfp8_quantize.restype = ctypes.c_int
            L.gemm_mxfp8_quantize_tiled.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp]
            L.gemm_mxfp8_quantize_tiled.restype = ctypes.c_int
            for name in ("gemm_bf16_grouped", "gemm_bf16_grouped_dgrad"):
                getattr(L, name).argtypes = [_vp, _vp, _vp, _vp, *[_i64] * 8, ctypes.c_int, _vp]
                getattr(L, name).restype = ctypes.c_int
            L.gemm_bf16_grouped_wgrad.argtypes = [_vp, _vp, _vp, _vp, *[_i64] * 8, ctypes.c_int,
                                                  ctypes.c_int, _vp]
            L.gemm_bf16_grouped_wgrad.restype = ctypes.c_int
            L.gemm_newton_schulz_workspace_bytes.argtypes = [_i64, _i64, _i64]
            L.gemm_newton_schulz_workspace_bytes.restype = _i64
            L.gemm_newton_schulz.argtypes = [_vp, _vp, *[_i64] * 7, *[ctypes.c_int] * 3,
                                             *[ctypes.c_float] * 4, _vp, _i64, _vp]
            L.gemm_newton_schulz.restype = ctypes.c_int
            i, f = ctypes.c_int, ctypes.c_float
            L.gemm_bf16_cross_entropy_workspace_bytes.argtypes = [_i64, _i64, _i64, i]
            L.gemm_bf16_cross_entropy_workspace_bytes.restype = _i64
            L.gemm_bf16_cross_entropy.argtypes = [*[_vp] * 5, *[_i64] * 5, i, f, f, f, _vp, _i64, _vp]
            L.gemm_bf16_cross_entropy_grad.argtypes = [*[_vp] * 7, *[_i64] * 8, i, i, i, f, f, f, i,
                                                       _vp, _i64, _vp]
            L.gemm_bf16_distill_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, i]
            L.gemm_bf16_distill_workspace_bytes.restype = _i64
            L.gemm_bf16_distill.argtypes = [*[_vp] * 6, *[_i64] * 8, i, i, f, _vp, _i64, _vp]
            L.gemm_bf16_distill_grad.argtypes = [*[_vp] * 8, *[_i64] * 11, i, i, i, i, f, i, _vp, _i64,
                                                 _vp]
            for name in ("gemm_bf16_cross_entropy", "gemm_bf16_cross_entropy_grad",
                         "gemm_bf16_distill", "gemm_bf16_distill_grad"):
                getattr(L, name).restype = i
            L.gemm_last_status.argtypes = [_vp]
            L.gemm_last_status.restype = ctypes.c_int
            L.gemm_last_status_word.argtypes = [_vp]
            L.gemm_last_status_word.restype = ctypes.c_uint64
            L.gemm_status_string.argtypes = [ctypes.c_int]
            L.gemm_status_string.restype = ctypes.c_char_p
            L.gemm_debug_stall_next_launch.argtypes = [_i64]
            L.gemm_debug_stall_next_launch.restype = ctypes.c_int
            L.gemm_last_cuda_error.argtypes = []
            L.gemm_last_cuda_error.restype = ctypes.c_int
            L.gemm_set_watchdog_ms.argtypes = [_i64]
            L.gemm_set_watchdog_ms.restype = _i64
            P = ctypes.POINTER(ctypes.c_int32)
            L.gemm_kernel_plan.argtypes = [ctypes.c_int, ctypes.c_int, P, P, P, P, P, P, P]
            L.gemm_kernel_plan.restype = ctypes.c_int
            _lib = L
    return _lib


# ------------------------------------------------------------- C entry points

def gemm_bf16(A: int, B: int, D: int, M: int, N: int, K: int, lda: int, ldb: int, ldd: int,
              stream: int = 0) -> int:
    return load().gemm_bf16(A, B, D, M, N, K, lda, ldb, ldd, stream)


def gemm_bf16_variant(variant: int, A: int, B: int, D: int, M: int, N: int, K: int, lda: int,
                      ldb: int, ldd: int, stream: int = 0) -> int:
    return load().gemm_bf16_variant(variant, A, B, D, M, N, K, lda, ldb, ldd, stream)


def gemm_mxfp8(A: int, B: int, SFA: int, SFB: int, D: int, M: int, N: int, K: int, lda: int,
               ldb: int, ldsfa: int, ldsfb: int, ldd: int, stream: int = 0) -> int:
    return load().gemm_mxfp8(A, B, SFA, SFB, D, M, N, K, lda, ldb, ldsfa, ldsfb, ldd, stream)


def gemm_mxfp8_variant(variant: int, A: int, B: int, SFA: int, SFB: int, D: int, M: int, N: int,
                       K: int, lda: int, ldb: int, ldsfa: int, ldsfb: int, ldd: int,
                       stream: int = 0) -> int:
    return load().gemm_mxfp8_variant(variant, A, B, SFA, SFB, D, M, N, K, lda, ldb, ldsfa, ldsfb,
                                     ldd, stream)


def gemm_mxfp8_tiled(variant: int, A: int, B: int, SFA: int, SFB: int, D: int, M: int, N: int,
                     K: int, lda: int, ldb: int, ldd: int, stream: int = 0) -> int:
    return load().gemm_mxfp8_tiled(variant, A, B, SFA, SFB, D, M, N, K, lda, ldb, ldd, stream)


def gemm_bf16_streamk(variant: int, A: int, B: int, D: int, M: int, N: int, K: int, lda: int,
                      ldb: int, ldd: int, workspace: int, workspace_bytes: int,
                      stream: int = 0) -> int:
    return load().gemm_bf16_streamk(variant, A, B, D, M, N, K, lda, ldb, ldd, workspace,
                                    workspace_bytes, stream)


def gemm_mxfp8_streamk(variant: int, A: int, B: int, SFA: int, SFB: int, D: int, M: int, N: int,
                       K: int, lda: int, ldb: int, ldsfa: int, ldsfb: int, ldd: int,
                       workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return load().gemm_mxfp8_streamk(variant, A, B, SFA, SFB, D, M, N, K, lda, ldb, ldsfa, ldsfb,
                                     ldd, workspace, workspace_bytes, stream)


def gemm_bf16_streamk_noalloc(variant: int, A: int, B: int, D: int, M: int, N: int, K: int,
                              lda: int, ldb: int, ldd: int, stream: int = 0) -> int:
    return load().gemm_bf16_streamk_noalloc(variant, A, B, D, M, N, K, lda, ldb, ldd, stream)


def gemm_streamk_workspace_bytes(mxfp8: bool, variant: int) -> int:
    return int(load().gemm_streamk_workspace_bytes(int(bool(mxfp8)), variant))


STREAMK_AUTO, STREAMK_ALWAYS, STREAMK_NEVER = 0, 1, 2


def gemm_set_streamk_mode(mode: int) -> int:
    return load().gemm_set_streamk_mode(mode)


def gemm_set_tail_split(enable: int) -> int:
    return load().gemm_set_tail_split(enable)


def gemm_set_edge_last(enable: int) -> int:
    return load().gemm_set_edge_last(enable)


def gemm_tail_split_plan(tiles: int, resident: int) -> int:
    return int(load().gemm_tail_split_plan(tiles, resident))


def gemm_bf16_fused(variant: int, A: int, B: int, D: int, M: int, N: int, K: int, lda: int,
                    ldb: int, ldd: int, epi: GemmEpilogue | None, stream: int = 0) -> int:
    return load().gemm_bf16_fused(variant, A, B, D, M, N, K, lda, ldb, ldd,
                                  None if epi is None else ctypes.byref(epi), stream)


def gemm_mxfp8_fused(variant: int, A: int, B: int, SFA: int, SFB: int, D: int, M: int, N: int,
                     K: int, lda: int, ldb: int, ldsfa: int, ldsfb: int, ldd: int,
                     epi: GemmEpilogue | None, stream: int = 0) -> int:
    return load().gemm_mxfp8_fused(variant, A, B, SFA, SFB, D, M, N, K, lda, ldb, ldsfa, ldsfb,
                                   ldd, None if epi is None else ctypes.byref(epi), stream)


_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU}


def make_epilogue(alpha=1.0, beta=0.0, C=None, bias=None, activation="none",
                  out_dtype=None) -> GemmEpilogue:
    """A GemmEpilogue from torch tensors: C [M, >=N] of the output dtype,
    bias [N] bf16 or float32, activation "none" | "relu" | "gelu"."""
    import torch
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be bfloat16 or float32")
    e = GemmEpilogue()
    e.alpha, e.beta = float(alpha), float(beta)
    e.out_dtype = DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16
    e.activation = _ACTS[activation]
    if C is not None:
        _check_2d(C, "C")
        if C.dtype != out_dtype:
            raise TypeError("C must have the output dtype")
        e.C, e.ldc = C.data_ptr(), C.stride(0)
    if bias is not None:
        if bias.dim() != 1 or bias.stride(0) != 1 or bias.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("bias must be a contiguous 1-D bfloat16 or float32 tensor")
        e.bias = bias.data_ptr()
        e.bias_dtype = DTYPE_F32 if bias.dtype == torch.float32 else DTYPE_BF16
    return e


def matmul_fused(A, B, SFA=None, SFB=None, *, alpha=1.0, beta=0.0, C=None, bias=None,
                 activation="none", out_dtype=None, out=None, variant: int = VARIANT_AUTO,
                 stream=None):
    """D = act(alpha A @ B.T + beta C + bias): bf16 A [M,K], B [N,K], or
    MXFP8 codes with SFA/SFB as in matmul_mxfp8; D of out_dtype (bf16 or fp32)."""
    import torch
    _check_2d(A, "A")
    _check_2d(B, "B")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out is None:
        out = _new((M, N), out_dtype, A.device, stream)
    _check_2d(out, "out")
    if out.dtype != out_dtype:
        raise TypeError("out must have out_dtype")
    e = make_epilogue(alpha, beta, C, bias, activation, out_dtype)
    if SFA is None:
        if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
            raise TypeError("A and B must be bfloat16 (or pass SFA/SFB for MXFP8)")
        rc = gemm_bf16_fused(variant, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                             A.stride(0), B.stride(0), out.stride(0), e, _stream_handle(stream))
    else:
        rc = gemm_mxfp8_fused(variant, A.data_ptr(), B.data_ptr(), SFA.data_ptr(), SFB.data_ptr(),
                              out.data_ptr(), M, N, K, A.stride(0), B.stride(0), SFA.stride(0),
                              SFB.stride(0), out.stride(0), e, _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "matmul_fused")
    return out


def gemm_streamk_plan(tiles: int, resident: int, k_tiles: int, unit: int,
                      mode: int = STREAMK_AUTO) -> dict:
    """The stream-K schedule for a tile count (host only)."""
    out = (ctypes.c_int64 * 3)()
    rc = load().gemm_streamk_plan(tiles, resident, k_tiles, unit, mode, out)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_streamk_plan")
    return {"dp_tiles": out[0], "sk_tiles": out[1], "clusters": out[2]}


def gemm_last_schedule() -> dict:
    """Schedule of this thread's last persistent-kernel launch."""
    out = (ctypes.c_int64 * 7)()
    rc = load().gemm_last_schedule(out)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_last_schedule")
    return {"clusters": out[0], "ctas_per_cluster": out[1], "dp_tiles": out[2],
            "sk_tiles": out[3], "sk_unit": out[4], "half_tiles": out[5], "edge_last": out[6]}


def streamk_workspace(mxfp8: bool = False, variant: int = VARIANT_AUTO, device=None):
    """A zeroed device buffer sized for the stream-K entry points (one per
    stream: calls sharing a workspace must not overlap on the GPU)."""
    import torch
    n = gemm_streamk_workspace_bytes(mxfp8, variant)
    if n < 0:
        raise GemmError(n, "gemm_streamk_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def gemm_mxfp8_quantize(X: int, rows: int, K: int, ldx: int, Q: int, ldq: int, SF: int,
                        ldsf: int, stream: int = 0) -> int:
    return load().gemm_mxfp8_quantize(X, rows, K, ldx, Q, ldq, SF, ldsf, stream)


def gemm_mxfp8_quantize_tiled(X: int, rows: int, K: int, ldx: int, Q: int, ldq: int, SF: int,
                              stream: int = 0) -> int:
    return load().gemm_mxfp8_quantize_tiled(X, rows, K, ldx, Q, ldq, SF, stream)


MAX_GROUPS = 1024


def gemm_bf16_grouped(A: int, B: int, D: int, offsets: int, groups: int, M: int, N: int, K: int,
                      lda: int, ldb: int, stride_b: int, ldd: int, out_dtype: int = DTYPE_BF16,
                      stream: int = 0) -> int:
    return load().gemm_bf16_grouped(A, B, D, offsets, groups, M, N, K, lda, ldb, stride_b, ldd,
                                    out_dtype, stream)


def gemm_bf16_grouped_dgrad(dD: int, B: int, dA: int, offsets: int, groups: int, M: int, N: int,
                            K: int, ldd: int, ldb: int, stride_b: int, lda: int,
                            out_dtype: int = DTYPE_BF16, stream: int = 0) -> int:
    return load().gemm_bf16_grouped_dgrad(dD, B, dA, offsets, groups, M, N, K, ldd, ldb, stride_b,
                                          lda, out_dtype, stream)


def gemm_bf16_grouped_wgrad(dD: int, A: int, dB: int, offsets: int, groups: int, M: int, N: int,
                            K: int, ldd: int, lda: int, ldb: int, stride_b: int,
                            out_dtype: int = DTYPE_BF16, accumulate: int = 0,
                            stream: int = 0) -> int:
    return load().gemm_bf16_grouped_wgrad(dD, A, dB, offsets, groups, M, N, K, ldd, lda, ldb,
                                          stride_b, out_dtype, accumulate, stream)


# Muon's published quintic, whose steps bring singular values of [0.003, 1] to about [0.7, 1.2] in five.
NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def gemm_newton_schulz_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(load().gemm_newton_schulz_workspace_bytes(batch, rows, cols))


def gemm_newton_schulz(G: int, O: int, batch: int, rows: int, cols: int, ldg: int, stride_g: int,
                       ldo: int, stride_o: int, in_dtype: int, out_dtype: int, steps: int,
                       a: float, b: float, c: float, eps: float, workspace: int,
                       workspace_bytes: int, stream: int = 0) -> int:
    return load().gemm_newton_schulz(G, O, batch, rows, cols, ldg, stride_g, ldo, stride_o,
                                     in_dtype, out_dtype, steps, a, b, c, eps, workspace,
                                     workspace_bytes, stream)


INDEX_I32, INDEX_I64 = 0, 1
MAX_TOP = 1024


def gemm_bf16_cross_entropy_workspace_bytes(M: int, N: int, K: int, grad: int) -> int:
    return int(load().gemm_bf16_cross_entropy_workspace_bytes(M, N, K, grad))


def gemm_bf16_cross_entropy(A: int, B: int, targets: int, loss: int, lse: int, M: int, N: int, K: int,
                            lda: int, ldb: int, target_dtype: int, scale: float, smoothing: float,
                            z_loss: float, workspace: int, workspace_bytes: int,
                            stream: int = 0) -> int:
    return load().gemm_bf16_cross_entropy(A, B, targets, loss, lse, M, N, K, lda, ldb, target_dtype,
                                          scale, smoothing, z_loss, workspace, workspace_bytes, stream)


def gemm_bf16_cross_entropy_grad(dloss: int, A: int, B: int, targets: int, lse: int, dA: int, dB: int,
                                 M: int, N: int, K: int, inc_dloss: int, lda: int, ldb: int,
                                 ld_da: int, ld_db: int, target_dtype: int, da_dtype: int,
                                 db_dtype: int, scale: float, smoothing: float, z_loss: float,
                                 accumulate: int, workspace: int, workspace_bytes: int,
                                 stream: int = 0) -> int:
    return load().gemm_bf16_cross_entropy_grad(dloss, A, B, targets, lse, dA, dB, M, N, K, inc_dloss,
                                               lda, ldb, ld_da, ld_db, target_dtype, da_dtype,
                                               db_dtype, scale, smoothing, z_loss, accumulate,
                                               workspace, workspace_bytes, stream)


def gemm_bf16_distill_workspace_bytes(M: int, N: int, K: int, top: int, grad: int) -> int:
    return int(load().gemm_bf16_distill_workspace_bytes(M, N, K, top, grad))


def gemm_bf16_distill(A: int, B: int, teacher: int, ids: int, loss: int, lse: int, M: int, N: int,
                      K: int, top: int, lda: int, ldb: int, ld_teacher: int, ld_ids: int,
                      teacher_dtype: int, id_dtype: int, temperature: float, workspace: int,
                      workspace_bytes: int, stream: int = 0) -> int:
    return load().gemm_bf16_distill(A, B, teacher, ids, loss, lse, M, N, K, top, lda, ldb, ld_teacher,
                                    ld_ids, teacher_dtype, id_dtype, temperature, workspace,
                                    workspace_bytes, stream)


def gemm_bf16_distill_grad(dloss: int, A: int, B: int, teacher: int, ids: int, lse: int, dA: int,
                           dB: int, M: int, N: int, K: int, top: int, inc_dloss: int, lda: int,
                           ldb: int, ld_teacher: int, ld_ids: int, ld_da: int, ld_db: int,
                           teacher_dtype: int, id_dtype: int, da_dtype: int, db_dtype: int,
                           temperature: float, accumulate: int, workspace: int,
                           workspace_bytes: int, stream: int = 0) -> int:
    return load().gemm_bf16_distill_grad(dloss, A, B, teacher, ids, lse, dA, dB, M, N, K, top,
                                         inc_dloss, lda, ldb, ld_teacher, ld_ids, ld_da, ld_db,
                                         teacher_dtype, id_dtype, da_dtype, db_dtype, temperature,
                                         accumulate, workspace, workspace_bytes, stream)


def gemm_last_status(stream: int = 0) -> int:
    return load().gemm_last_status(stream)


def gemm_last_status_word(stream: int = 0) -> int:
    return int(load().gemm_last_status_word(stream))


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(status).decode()


def gemm_last_cuda_error() -> int:
    return int(load().gemm_last_cuda_error())


def gemm_debug_stall_next_launch(k_iteration: int) -> int:
    return int(load().gemm_debug_stall_next_launch(k_iteration))


def gemm_set_watchdog_ms(ms: int) -> int:
    return int(load().gemm_set_watchdog_ms(ms))


def gemm_kernel_plan(mxfp8, variant: int) -> dict:
    """mxfp8: False/0 bf16, True/1 MXFP8, 2 MXFP8 with tiled scales."""
    vals = [ctypes.c_int32() for _ in range(7)]
    rc = load().gemm_kernel_plan(int(mxfp8), variant, *[ctypes.byref(v) for v in vals])
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_kernel_plan")
    keys = ("stages", "smem_bytes", "tmem_cols", "threads", "cluster", "tile_m", "tile_n")
    return {k: v.value for k, v in zip(keys, vals)}


# ------------------------------------------------------- torch conveniences

def _stream_handle(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _new(shape, dtype, device, stream, zeroed=False):
    """A tensor that a call on `stream` writes.  On another stream than torch's
    current one it comes from that stream's memory: the current stream's could
    still be in use by what is queued there.  Either may use the result, so its
    memory is not given away before both are past its release."""
    import torch
    make = torch.zeros if zeroed else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream()
    if stream.cuda_stream == current.cuda_stream:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream))
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    if t.is_cuda:
        t.record_stream(current)
    return t


def _check_2d(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def matmul_bf16(A, B, out=None, variant: int = VARIANT_AUTO, stream=None, workspace=None):
    """D = A @ B.T for bf16 CUDA tensors A [M,K], B [N,K]; returns D [M,N] bf16.
    With `workspace` (from streamk_workspace) the stream-K schedule is used."""
    import torch
    _check_2d(A, "A")
    _check_2d(B, "B")
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    if out is None:
        out = _new((M, N), torch.bfloat16, A.device, stream)
    _check_2d(out, "out")
    if workspace is None:
        rc = gemm_bf16_variant(variant, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                               A.stride(0), B.stride(0), out.stride(0), _stream_handle(stream))
    else:
        rc = gemm_bf16_streamk(variant, A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K,
                               A.stride(0), B.stride(0), out.stride(0), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(),
                               _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16")
    return out


def matmul_mxfp8(A, SFA, B, SFB, out=None, variant: int = VARIANT_AUTO, stream=None,
                 workspace=None):
    """Block-scaled D = A @ B.T: A [M,K], B [N,K] E4M3 codes (uint8 or
    float8_e4m3fn), SFA [M,>=ceil(K/32)], SFB [N,>=ceil(K/32)] UE8M0 bytes.
    With `workspace` (from streamk_workspace) the stream-K schedule is used."""
    import torch
    for t, n in ((A, "A"), (B, "B"), (SFA, "SFA"), (SFB, "SFB")):
        _check_2d(t, n)
        if t.element_size() != 1:
            raise TypeError(f"{n} must hold one byte per element")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    if out is None:
        out = _new((M, N), torch.bfloat16, A.device, stream)
    _check_2d(out, "out")
    if workspace is None:
        rc = gemm_mxfp8_variant(variant, A.data_ptr(), B.data_ptr(), SFA.data_ptr(),
                                SFB.data_ptr(), out.data_ptr(), M, N, K, A.stride(0), B.stride(0),
                                SFA.stride(0), SFB.stride(0), out.stride(0),
                                _stream_handle(stream))
    else:
        rc = gemm_mxfp8_streamk(variant, A.data_ptr(), B.data_ptr(), SFA.data_ptr(),
                                SFB.data_ptr(), out.data_ptr(), M, N, K, A.stride(0), B.stride(0),
                                SFA.stride(0), SFB.stride(0), out.stride(0), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(),
                                _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_mxfp8")
    return out


def quantize_mxfp8_tiled(X, stream=None):
    """MXFP8-encode a float32 CUDA tensor X [rows, K]: returns (Q uint8 [rows, K],
    SF uint8, flat, in the tiled layout of gemm_mxfp8_tiled)."""
    import torch
    _check_2d(X, "X")
    if X.dtype != torch.float32:
        raise TypeError("X must be float32")
    rows, K = X.shape
    n = (rows + 127) // 128 * (((K + 31) // 32 + 3) // 4) * 512
    Q = _new((rows, K), torch.uint8, X.device, stream)
    SF = _new((n,), torch.uint8, X.device, stream)
    rc = gemm_mxfp8_quantize_tiled(X.data_ptr(), rows, K, X.stride(0), Q.data_ptr(), Q.stride(0),
                                   SF.data_ptr(), _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_mxfp8_quantize_tiled")
    return Q, SF


def matmul_mxfp8_tiled(A, SFA, B, SFB, out=None, variant: int = VARIANT_AUTO, stream=None):
    """Block-scaled D = A @ B.T with the scale matrices in the tiled layout of
    gemm_mxfp8_tiled (1-D byte tensors, e.g. from gemm_inputs.tile_scales)."""
    import torch
    for t, n in ((A, "A"), (B, "B")):
        _check_2d(t, n)
        if t.element_size() != 1:
            raise TypeError(f"{n} must hold one byte per element")
    for t, n in ((SFA, "SFA"), (SFB, "SFB")):
        if not t.is_cuda or t.element_size() != 1 or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous CUDA byte tensor")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    kt = (K + 127) // 128
    for t, n, R in ((SFA, "SFA", M), (SFB, "SFB", N)):
        if t.numel() < (R + 127) // 128 * kt * 512:
            raise ValueError(f"{n} is smaller than the tiled layout of {R} rows")
    if out is None:
        out = _new((M, N), torch.bfloat16, A.device, stream)
    _check_2d(out, "out")
    rc = gemm_mxfp8_tiled(variant, A.data_ptr(), B.data_ptr(), SFA.data_ptr(), SFB.data_ptr(),
                          out.data_ptr(), M, N, K, A.stride(0), B.stride(0), out.stride(0),
                          _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_mxfp8_tiled")
    return out


def quantize_mxfp8(X, stream=None):
    """MXFP8-encode a float32 CUDA tensor X [rows, K]: returns (Q uint8
    [rows, K], SF uint8 [rows, pitch]) with the scale pitch padded to a
    multiple of 16 bytes (the pitch gemm_mxfp8 requires), padding zeroed."""
    import torch
    _check_2d(X, "X")
    if X.dtype != torch.float32:
        raise TypeError("X must be float32")
    rows, K = X.shape
    pitch = max(16, ((K + 31) // 32 + 15) // 16 * 16)
    Q = _new((rows, K), torch.uint8, X.device, stream)
    SF = _new((rows, pitch), torch.uint8, X.device, stream, zeroed=True)
    rc = gemm_mxfp8_quantize(X.data_ptr(), rows, K, X.stride(0), Q.data_ptr(), Q.stride(0),
                             SF.data_ptr(), SF.stride(0), _stream_handle(stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_mxfp8_quantize")
    return Q, SF


# --------------------------------------------------- expert-training operators
#
# A decoding step makes these calls with a few microseconds of GPU work each,
# so the checks are one expression on the way to the call; what was wrong is
# worked out only once something is.

def _raw_stream(stream, device_index) -> int:
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device_index)
    return int(stream.cuda_stream)


def _out_code(dtype):
    import torch
    if dtype is torch.bfloat16:
        return DTYPE_BF16
    if dtype is torch.float32:
        return DTYPE_F32
    raise TypeError("the output dtype must be bfloat16 or float32")


def _check_3d(t, name):
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError(f"{name} must be a 3-D tensor with unit column stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _matrices(t, name):
    """(batch, rows, cols, row pitch, matrix stride) of a matrix or a batch of them."""
    if t.dim() == 2:
        (rows, cols), (ld, unit) = t.shape, t.stride()
        batch = stride = 1
    elif t.dim() == 3:
        (batch, rows, cols), (stride, ld, unit) = t.shape, t.stride()
    else:
        unit = 0
    if unit != 1 or not t.is_cuda:
        _check_3d(t if t.dim() == 3 else t.unsqueeze(0), name)
    return batch, rows, cols, ld, stride


def _refuse_grouped(rc, entry, x, x_name, B, B_name, offsets, groups, out):
    """Raises for what is wrong with a grouped product's tensors, else `rc`."""
    import torch
    for t, name in ((x, x_name), (B, B_name), (out, "out")):
        (_check_3d if t.dim() == 3 else _check_2d)(t, name)
    if x.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("the operands must be bfloat16")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous 1-D int32 tensor")
    if not offsets.is_cuda:
        raise ValueError("offsets must be a CUDA tensor")
    if offsets.numel() != groups + 1:
        raise ValueError(f"offsets must hold one value more than the {groups} groups")
    raise GemmError(rc, entry)


def _output(out, shape, dtype, device, stream):
    import torch
    if out is None:
        return _new(shape, torch.bfloat16 if dtype is None else dtype, device, stream)
    if out.shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}")
    if dtype is not None and out.dtype != dtype:
        raise TypeError("out must have out_dtype")
    return out


def _grouped_rows(entry, x, x_name, B, offsets, dgrad, out, out_dtype, stream):
    import torch
    M, reduced = x.shape
    groups, N, K = B.shape
    if reduced != (N if dgrad else K):
        raise ValueError(f"{x_name} and B disagree on {'N' if dgrad else 'K'}")
    out = _output(out, (M, K if dgrad else N), out_dtype, x.device, stream)
    ldx, x1 = x.stride()
    sb, ldb, b1 = B.stride()
    ldo, o1 = out.stride()
    bf16 = torch.bfloat16
    rc = GEMM_ERR_INVALID_ARG
    # (what is not on the GPU the call itself refuses)
    if (x.dtype is bf16 and B.dtype is bf16 and offsets.dtype is torch.int32 and x1 == b1 == o1 == 1
            and offsets.shape == (groups + 1,) and offsets.is_contiguous()):
        rc = getattr(_lib or load(), entry)(
            x.data_ptr(), B.data_ptr(), out.data_ptr(), offsets.data_ptr(), groups, M, N, K,
            ldx, ldb, sb, ldo, _out_code(out.dtype), _raw_stream(stream, x.get_device()))
    if rc != GEMM_OK:
        _refuse_grouped(rc, entry, x, x_name, B, "B", offsets, groups, out)
    return out


def matmul_grouped(A, B, offsets, out=None, out_dtype=None, stream=None):
    """D[r] = A[r] @ B[e].T for the rows offsets[e] <= r < offsets[e + 1] of
    A [M,K] bf16, B [groups,N,K] bf16, offsets [groups+1] int32, all on the
    GPU; returns D [M,N] of out_dtype (bfloat16 or float32).  Rows that belong
    to no group are not written.  No autograd graph is recorded: the gradients
    are matmul_grouped_dgrad and matmul_grouped_wgrad, whose dD needs a pitch
    that is a multiple of 8 like every operand."""
    return _grouped_rows("gemm_bf16_grouped", A, "A", B, offsets, False, out, out_dtype, stream)


def matmul_grouped_dgrad(dD, B, offsets, out=None, out_dtype=None, stream=None):
    """The gradient of matmul_grouped to A: dA[r] = dD[r] @ B[e], dD [M,N]
    bf16; returns dA [M,K] of out_dtype (bfloat16 or float32)."""
    return _grouped_rows("gemm_bf16_grouped_dgrad", dD, "dD", B, offsets, True, out, out_dtype,
                         stream)


def matmul_grouped_wgrad(dD, A, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """The gradient of matmul_grouped to B: dB[e] = dD[rows of e].T @ A[rows of
    e]; returns dB [groups,N,K] of out_dtype (bfloat16 or float32).  With
    accumulate, adds to `out` instead."""
    import torch
    M, N = dD.shape
    MA, K = A.shape
    if MA != M:
        raise ValueError("dD and A disagree on M")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    groups = max(0, offsets.numel() - 1)
    out = _output(out, (groups, N, K), out_dtype, A.device, stream)
    ldd, d1 = dD.stride()
    lda, a1 = A.stride()
    sb, ldb, o1 = out.stride()
    bf16 = torch.bfloat16
    rc = GEMM_ERR_INVALID_ARG
    if (dD.dtype is bf16 and A.dtype is bf16 and offsets.dtype is torch.int32
            and d1 == a1 == o1 == 1 and offsets.shape == (groups + 1,) and offsets.is_contiguous()):
        rc = (_lib or load()).gemm_bf16_grouped_wgrad(
            dD.data_ptr(), A.data_ptr(), out.data_ptr(), offsets.data_ptr(), groups, M, N, K,
            ldd, lda, ldb, sb, _out_code(out.dtype), 1 if accumulate else 0,
            _raw_stream(stream, A.get_device()))
    if rc != GEMM_OK:
        _refuse_grouped(rc, "gemm_bf16_grouped_wgrad", dD, "dD", A, "A", offsets, groups, out)
    return out


def newton_schulz_workspace(batch: int, rows: int, cols: int, device=None):
    """A workspace for newton_schulz on a batch of rows x cols matrices (one
    per stream: calls sharing a workspace must not overlap on the GPU)."""
    import torch
    n = gemm_newton_schulz_workspace_bytes(batch, rows, cols)
    if n < 0:
        raise GemmError(n, "gemm_newton_schulz_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def newton_schulz(G, steps: int = 5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps: float = 1e-7,
                  out=None, out_dtype=None, workspace=None, stream=None):
    """Newton-Schulz orthogonalisation of a matrix [rows,cols] or a batch
    [batch,rows,cols] (bfloat16 or float32): X = G / (|G| + eps), then `steps`
    times X <- a X + b (X X^T) X + c (X X^T)^2 X on the smaller side; returns X
    in out_dtype (bfloat16 or float32).  Without `workspace` (from
    newton_schulz_workspace) one is allocated for the call on torch's current
    stream."""
    import torch
    batch, rows, cols, ldg, stride_g = _matrices(G, "G")
    if G.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("G must be bfloat16 or float32")
    out = _output(out, G.shape, out_dtype, G.device, stream)
    _, _, _, ldo, stride_o = _matrices(out, "out")
    a, b, c = coefficients
    if workspace is None:
        if stream is not None and stream != torch.cuda.current_stream():
            raise ValueError("a call on another stream needs its own workspace")
        workspace = newton_schulz_workspace(batch, rows, cols, G.device)
    rc = gemm_newton_schulz(G.data_ptr(), out.data_ptr(), batch, rows, cols, ldg, stride_g, ldo, stride_o,
                            _out_code(G.dtype), _out_code(out.dtype), steps, a, b, c, eps,
                            workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, G.get_device()))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_newton_schulz")
    return out


# -------------------------------------------------- losses over a vocabulary
#
# A few rows' losses take the GPU little longer than a launch, so these calls
# too check in one expression on the way, and work out what was wrong only once
# something is.

def _index_code(dtype):
    import torch
    if dtype is torch.int64:
        return INDEX_I64
    if dtype is torch.int32:
        return INDEX_I32
    raise TypeError("targets and ids must be int32 or int64")


def _row_values(t, name, M, dtype=None, strided=False):
    """Checks a value per row: 1-D of M, contiguous unless `strided`."""
    if t.dim() != 1 or t.shape[0] != M:
        raise ValueError(f"{name} must be a 1-D tensor with a value for each of the {M} rows")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}")
    if not strided and M > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")


def _refuse_loss(rc, entry, A, B, of_rows, lists, outputs):
    """Raises for what is wrong with a loss's tensors, else `rc`: of_rows are
    (tensor, name, dtype, strided) with a value per row."""
    import torch
    _check_2d(A, "A")
    _check_2d(B, "B")
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    M, K = A.shape
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    for t, name in lists:
        _check_2d(t, name)
        if t.shape != lists[0][0].shape or t.shape[0] != M:
            raise ValueError(f"teacher and ids must both have shape ({M}, top)")
    for t, name, dtype, strided in of_rows:
        _row_values(t, name, M, dtype, strided)
    for t, name in outputs:
        if t is not None:
            _check_2d(t, name)
    raise GemmError(rc, entry)


@functools.lru_cache(maxsize=1024)
def _loss_bytes(entry, *sizes):
    n = getattr(load(), entry)(*sizes)
    if n < 0:
        raise GemmError(n, entry)
    return n


_CE_BYTES, _KD_BYTES = "gemm_bf16_cross_entropy_workspace_bytes", "gemm_bf16_distill_workspace_bytes"


def cross_entropy_workspace(M: int, N: int, K: int, grad: bool = False, device=None):
    """A workspace for matmul_cross_entropy (grad: for its gradient) on M rows
    of width K and a vocabulary of N (one per stream: calls sharing a workspace
    must not overlap on the GPU)."""
    import torch
    return torch.empty(_loss_bytes(_CE_BYTES, M, N, K, int(grad)), dtype=torch.uint8, device=device or "cuda")


def distill_workspace(M: int, N: int, K: int, top: int, grad: bool = False, device=None):
    """The same for matmul_distill with lists of `top` entries."""
    import torch
    return torch.empty(_loss_bytes(_KD_BYTES, M, N, K, top, int(grad)), dtype=torch.uint8, device=device or "cuda")


def _foreign(stream):
    """Refuses to allocate a workspace for a call on another stream than torch's current one."""
    import torch
    if stream is not None and stream != torch.cuda.current_stream():
        raise ValueError("a call on another stream needs its own workspace")


def _gradient(t, like, needed, out_dtype, stream):
    """(a gradient's tensor or None, pointer, pitch, its columns' stride, type code)."""
    if t is None:
        if not needed:
            return None, 0, 0, 1, DTYPE_BF16
        t = _output(None, like.shape, out_dtype, like.device, stream)
    elif t.shape != like.shape:
        raise ValueError(f"a gradient given must have shape {tuple(like.shape)}")
    ld, unit = t.stride() if t.dim() == 2 else (0, 0)
    return t, t.data_ptr(), ld, unit, _out_code(t.dtype)


def matmul_cross_entropy(A, B, targets, scale: float = 1.0, label_smoothing: float = 0.0, z_loss: float = 0.0,
                         out=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits z = scale * A @ B.T, which are never
    stored: A [M,K] and B [N,K] bf16, targets [M] int32 or int64; returns (loss
    [M], lse [M]), both float32 (into out=(loss, lse) if given), with
        loss = lse - (1 - label_smoothing) z[target] - label_smoothing mean(z) + z_loss lse**2.
    Rows with a negative target are left out: their loss and lse are 0.  A
    target of N or more makes its row's loss NaN.  No autograd graph is
    recorded: the gradients are matmul_cross_entropy_grad.  Without `workspace`
    (from cross_entropy_workspace) one is allocated for the call on torch's
    current stream."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    rc, loss, lse = GEMM_ERR_INVALID_ARG, None, None
    code = INDEX_I64 if targets.dtype is torch.int64 else _index_code(targets.dtype)
    if A.dim() == B.dim() == 2:
        (M, K), (N, KB) = A.shape, B.shape
        (lda, a1), (ldb, b1) = A.stride(), B.stride()
        device = A.device
        if out is not None:
            loss, lse = out
        elif stream is None:
            loss, lse = torch.empty(M, dtype=f32, device=device), torch.empty(M, dtype=f32, device=device)
        else:
            loss, lse = _new((M,), f32, device, stream), _new((M,), f32, device, stream)
        if (K == KB and a1 == b1 == 1 and A.dtype is bf16 and B.dtype is bf16 and A.is_cuda
                and targets.shape == loss.shape == lse.shape == (M,) and loss.dtype is f32 and lse.dtype is f32
                and targets.is_contiguous() and loss.is_contiguous() and lse.is_contiguous()):
            if workspace is None:
                if stream is not None:
                    _foreign(stream)
                workspace = torch.empty(_loss_bytes(_CE_BYTES, M, N, K, 0), dtype=torch.uint8, device=device)
            rc = (_lib or load()).gemm_bf16_cross_entropy(
                A.data_ptr(), B.data_ptr(), targets.data_ptr(), loss.data_ptr(), lse.data_ptr(), M, N, K, lda, ldb, code,
                scale, label_smoothing, z_loss, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, A.get_device()))
    if rc != GEMM_OK:
        outputs = () if loss is None else ((loss, "out[0]", f32, False), (lse, "out[1]", f32, False))
        _refuse_loss(rc, "gemm_bf16_cross_entropy", A, B, ((targets, "targets", None, False), *outputs), (), ())
    return loss, lse


def matmul_cross_entropy_grad(dloss, A, B, targets, lse, scale: float = 1.0, label_smoothing: float = 0.0,
                              z_loss: float = 0.0, dA=None, dB=None, need_dA: bool = True, need_dB: bool = True,
                              out_dtype=None, accumulate: bool = False, workspace=None, stream=None):
    """The gradients of matmul_cross_entropy to A and B, from the losses' own,
    dloss [M] float32 (any stride, an expanded one too), and the lse that it
    returned; returns (dA [M,K], dB [N,K]), into dA and dB if given (bfloat16 or
    float32 each), else of out_dtype; None for one that is neither given nor
    needed.  With accumulate, adds to dB.  Rows left out get zeros in dA and add
    nothing to dB, whatever A holds there.  The logits' gradient is rounded to
    bfloat16 before the products with it (up to 128 rows keep a second term), so
    float32 gradients of more rows are about 1.5e-3 off, as bfloat16 ones are
    2.4e-3.  Without `workspace` (from cross_entropy_workspace with grad=True)
    one is allocated for the call: 512 MiB of the logits' gradient at most, or
    4096 of its columns, and a few times A's size."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    if accumulate and dB is None:
        raise ValueError("accumulate needs dB")
    rc = GEMM_ERR_INVALID_ARG
    code = INDEX_I64 if targets.dtype is torch.int64 else _index_code(targets.dtype)
    if A.dim() == B.dim() == 2:
        (M, K), (N, KB) = A.shape, B.shape
        (lda, a1), (ldb, b1) = A.stride(), B.stride()
        dA, pa, ld_da, da1, ca = _gradient(dA, A, need_dA, out_dtype, stream)
        dB, pb, ld_db, db1, cb = _gradient(dB, B, need_dB, out_dtype, stream)
        if (K == KB and a1 == b1 == da1 == db1 == 1 and A.dtype is bf16 and B.dtype is bf16 and A.is_cuda
                and targets.shape == dloss.shape == lse.shape == (M,) and dloss.dtype is f32 and lse.dtype is f32
                and targets.is_contiguous() and lse.is_contiguous()):
            if workspace is None:
                if stream is not None:
                    _foreign(stream)
                workspace = torch.empty(_loss_bytes(_CE_BYTES, M, N, K, 1), dtype=torch.uint8, device=A.device)
            rc = (_lib or load()).gemm_bf16_cross_entropy_grad(
                dloss.data_ptr(), A.data_ptr(), B.data_ptr(), targets.data_ptr(), lse.data_ptr(), pa, pb, M, N, K,
                dloss.stride(0), lda, ldb, ld_da, ld_db, code, ca, cb, scale, label_smoothing, z_loss,
                1 if accumulate else 0, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, A.get_device()))
    if rc != GEMM_OK:
        _refuse_loss(rc, "gemm_bf16_cross_entropy_grad", A, B,
                     ((targets, "targets", None, False), (dloss, "dloss", f32, True), (lse, "lse", f32, False)), (),
                     ((dA, "dA"), (dB, "dB")))
    return dA, dB


def matmul_distill(A, B, teacher, ids, temperature: float = 1.0, out=None, workspace=None, stream=None):
    """Distillation from a teacher's top logits: teacher [M,top] (bfloat16 or
    float32) are its logits of the tokens ids [M,top] (int32 or int64, any
    order), p = softmax(teacher / temperature) over a row's entries; the
    student's logits z = A @ B.T / temperature, A [M,K] and B [N,K] bf16, are
    never stored; returns (loss [M], lse [M]), both float32 (into out=(loss,
    lse) if given), with loss = sum_j p_j (log p_j - z[ids_j] + lse).  Entries
    with a negative id or a logit of -inf are not there; rows without any are
    left out: their loss and lse are 0.  An id of N or more makes its row's loss
    NaN.  No autograd graph is recorded: the gradients are matmul_distill_grad.
    Without `workspace` (from distill_workspace) one is allocated for the call
    on torch's current stream."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    rc, loss, lse = GEMM_ERR_INVALID_ARG, None, None
    ct, ci = _out_code(teacher.dtype), _index_code(ids.dtype)
    if A.dim() == B.dim() == teacher.dim() == ids.dim() == 2:
        (M, K), (N, KB) = A.shape, B.shape
        (lda, a1), (ldb, b1), (ldt, t1), (ldi, i1) = A.stride(), B.stride(), teacher.stride(), ids.stride()
        top = ids.shape[1]
        device = A.device
        if out is not None:
            loss, lse = out
        elif stream is None:
            loss, lse = torch.empty(M, dtype=f32, device=device), torch.empty(M, dtype=f32, device=device)
        else:
            loss, lse = _new((M,), f32, device, stream), _new((M,), f32, device, stream)
        if (K == KB and a1 == b1 == t1 == i1 == 1 and A.dtype is bf16 and B.dtype is bf16 and A.is_cuda
                and teacher.shape == ids.shape == (M, top) and loss.shape == lse.shape == (M,) and loss.dtype is f32
                and lse.dtype is f32 and loss.is_contiguous() and lse.is_contiguous() and 1 <= top <= MAX_TOP):
            if workspace is None:
                if stream is not None:
                    _foreign(stream)
                workspace = torch.empty(_loss_bytes(_KD_BYTES, M, N, K, top, 0), dtype=torch.uint8, device=device)
            rc = (_lib or load()).gemm_bf16_distill(
                A.data_ptr(), B.data_ptr(), teacher.data_ptr(), ids.data_ptr(), loss.data_ptr(), lse.data_ptr(), M, N, K, top,
                lda, ldb, ldt, ldi, ct, ci, temperature, workspace.data_ptr(), workspace.nbytes,
                _raw_stream(stream, A.get_device()))
    if rc != GEMM_OK:
        outputs = () if loss is None else ((loss, "out[0]", f32, False), (lse, "out[1]", f32, False))
        _refuse_loss(rc, "gemm_bf16_distill", A, B, outputs, ((teacher, "teacher"), (ids, "ids")), ())
    return loss, lse


def matmul_distill_grad(dloss, A, B, teacher, ids, lse, temperature: float = 1.0, dA=None, dB=None, need_dA: bool = True,
                        need_dB: bool = True, out_dtype=None, accumulate: bool = False, workspace=None, stream=None):
    """The gradients of matmul_distill to A and B (not to the teacher), from the
    losses' own, dloss [M] float32, and the lse that it returned; arguments and
    results as in matmul_cross_entropy_grad."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    if accumulate and dB is None:
        raise ValueError("accumulate needs dB")
    rc = GEMM_ERR_INVALID_ARG
    ct, ci = _out_code(teacher.dtype), _index_code(ids.dtype)
    if A.dim() == B.dim() == teacher.dim() == ids.dim() == 2:
        (M, K), (N, KB) = A.shape, B.shape
        (lda, a1), (ldb, b1), (ldt, t1), (ldi, i1) = A.stride(), B.stride(), teacher.stride(), ids.stride()
        top = ids.shape[1]
        dA, pa, ld_da, da1, ca = _gradient(dA, A, need_dA, out_dtype, stream)
        dB, pb, ld_db, db1, cb = _gradient(dB, B, need_dB, out_dtype, stream)
        if (K == KB and a1 == b1 == t1 == i1 == da1 == db1 == 1 and A.dtype is bf16 and B.dtype is bf16 and A.is_cuda
                and teacher.shape == ids.shape == (M, top) and dloss.shape == lse.shape == (M,) and dloss.dtype is f32
                and lse.dtype is f32 and lse.is_contiguous() and 1 <= top <= MAX_TOP):
            if workspace is None:
                if stream is not None:
                    _foreign(stream)
                workspace = torch.empty(_loss_bytes(_KD_BYTES, M, N, K, top, 1), dtype=torch.uint8, device=A.device)
            rc = (_lib or load()).gemm_bf16_distill_grad(
                dloss.data_ptr(), A.data_ptr(), B.data_ptr(), teacher.data_ptr(), ids.data_ptr(), lse.data_ptr(), pa, pb, M, N,
                K, top, dloss.stride(0), lda, ldb, ldt, ldi, ld_da, ld_db, ct, ci, ca, cb, temperature,
                1 if accumulate else 0, workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, A.get_device()))
    if rc != GEMM_OK:
        _refuse_loss(rc, "gemm_bf16_distill_grad", A, B, ((dloss, "dloss", f32, True), (lse, "lse", f32, False)),
                     ((teacher, "teacher"), (ids, "ids")), ((dA, "dA"), (dB, "dB")))
    return dA, dB
