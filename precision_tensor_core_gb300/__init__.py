"""Python binding of libptc, the GB300 (sm_103a) tensor-core GEMM library.

Dense matrix products C = A.B in the three precisions of "Hand-Written PTX
Tensor-Core GEMM Kernels: A Multi-Precision Study on NVIDIA L4"
(Borowski & Osinski): FP16 -> FP32, INT8 -> INT32 and packed INT4 -> INT32.

Two layers, both argument marshalling only (every arithmetic step runs in the
library's CUDA kernels):

* ``gemm_f16``, ``gemm_f16_f16acc``, ``gemm_s8``, ``gemm_s4``, ``gemm_s8_scaled``, ``gemm_s4_scaled``,
  ``gemm_s8_noalloc``, ``gemm_s8_b_rowmajor``, ``gemm_status_string``,
  ``gemm_poll_device_error``, ``ptc_kernel_launch_count``, ``ptc_last_launch``, ``ptc_last_fp4_launch``, ``ptc_last_conversion``, ``ptc_plan_shape``,
  ``ptc_debug_set_wait_limit``, ``ptc_set_tuning``, ``gemm_fp4``, ``gemm_a16_fp4``, ``ptc_dropout``,
  ``ptc_dropout_to``, ``ptc_quantize_fp4``, ``ptc_dequantize_fp4``, ``gemm_a16_s4``, ``gemm_a16_s4_workspace``, ``ptc_moe_a16_s4``,
  ``ptc_moe_a16_s4_workspace``, ``ptc_rms_norm``, ``ptc_rms_norm_s8``,
  ``ptc_rms_norm_backward``, ``ptc_rms_norm_backward_workspace``: the C ABI of
  ``include/ptc.h`` under the same names, taking integers (sizes, leading
  dimensions, device addresses, a cudaStream_t handle).  A nonzero status
  raises :class:`PtcError`.
* ``matmul_f16``, ``matmul_f16_f16acc``, ``matmul_s8``, ``matmul_s4``, ``matmul_s8_scaled``,
  ``matmul_s4_scaled``: the same calls on torch tensors.  Device tensors run
  on the current CUDA stream; host (CPU) tensors of ``matmul_f16`` /
  ``matmul_s8`` / ``matmul_s4`` go through the host-buffer entry points
  (``gemm_*_host``), which pipeline the copies inside the library.
* ``dropout``, ``quantize_fp4``, ``dequantize_fp4``, ``matmul_fp4``, ``matmul_a16_fp4`` and
  :class:`Fp4Matrix`: counter-based dropout and microscaled 4-bit matrices on
  torch tensors of the device; :mod:`precision_tensor_core_gb300.fp4_linear`
  puts them together as a linear layer's training and decoding steps.
* ``matmul_a16_s4``, ``moe_a16_s4`` and :class:`S4Matrix`: a few tokens with 4-bit integer
  weights that have group scales, in one matrix or as a mixture of experts.
* ``rms_norm``, ``rms_norm_s8``, ``rms_norm_backward``: the norm before a product, also as
  the 8-bit operand of ``matmul_s8_scaled``.

There is no CPU fallback: if ``libptc.so`` has not been built the first call
raises, and on a machine without a compute-capability 10.3 GPU every GEMM call
raises ``PtcError`` with status ``PTC_ERR_DEVICE``.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libptc.so")

PTC_OK = 0
PTC_ERR_INVALID = 1
PTC_ERR_ALIGN = 2
PTC_ERR_OVERLAP = 3
PTC_ERR_DEVICE = 4
PTC_ERR_LAUNCH = 5
PTC_ERR_TIMEOUT = 6
PTC_ERR_ALLOC = 7

PTC_BASELINE_F16_WMMA = 0
PTC_BASELINE_F16_MMA = 1
PTC_BASELINE_S8_WMMA = 2
PTC_BASELINE_S8_MMA = 3
PTC_BASELINE_S4_WMMA = 4
PTC_BASELINE_S4_MMA = 5
PTC_BASELINE_F16_LDMATRIX = 6
PTC_BASELINE_S8_LDMATRIX = 7
PTC_BASELINE_S4_LDMATRIX = 8

PTC_OUT_F32 = 0
PTC_OUT_BF16 = 1
PTC_OUT_F16 = 2

PTC_FP4_MX = 0
PTC_FP4_NV = 1
PTC_ROUND_NEAREST = 0
PTC_ROUND_STOCHASTIC = 1

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_lib = None


class PtcError(RuntimeError):
    """A libptc call returned a nonzero status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libptc.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libptc.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name in ("gemm_f16", "gemm_f16_f16acc", "gemm_s8", "gemm_s4", "gemm_s8_noalloc",
                     "gemm_s8_b_rowmajor", "gemm_f16_host", "gemm_s8_host", "gemm_s4_host"):
            fn = getattr(L, name)
            fn.restype = ctypes.c_int
            fn.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
        for name in ("gemm_s8_scaled", "gemm_s4_scaled"):
            fn = getattr(L, name)
            fn.restype = ctypes.c_int
            fn.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, ctypes.c_int, _vp]
        _int, _u64, _f64, _f32 = ctypes.c_int, ctypes.c_uint64, ctypes.c_double, ctypes.c_float
        for name, args in (
                ("ptc_dropout", [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _f64, _u64, _u64, _vp]),
                ("ptc_dropout_to", [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _int, _f64, _u64, _u64, _vp]),
                ("ptc_quantize_fp4", [_i64, _i64, _vp, _i64, _int, _int, _int, _vp, _vp, _i64, _vp, _vp, _i64, _vp,
                                      _f64, _u64, _u64, _vp]),
                ("ptc_dequantize_fp4", [_i64, _i64, _vp, _i64, _vp, _int, _vp, _vp, _i64, _int, _vp]),
                ("gemm_fp4", [_i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _int,
                              _vp]),
                ("gemm_a16_fp4", [_i64, _i64, _i64, _int, _vp, _i64, _int, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
                ("gemm_a16_s4", [_i64, _i64, _i64, _int, _vp, _i64, _vp, _i64, _i64, _int, _vp, _vp, _vp, _i64, _vp, _i64,
                                 _vp]),
                ("ptc_moe_a16_s4", [_i64] * 5 + [_int, _int, _vp, _i64, _vp, _i64, _int, _i64, _int]
                 + [_vp, _i64, _i64, _vp, _vp] * 2 + [_vp, _i64, _vp, _vp, _vp, _i64, _vp]),
                ("ptc_rms_norm", [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _int, _f32, _vp, _i64, _vp]),
                ("ptc_rms_norm_s8", [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _int, _f32, _vp, _i64, _vp,
                                     _vp]),
                ("ptc_rms_norm_backward", [_i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _vp, _int, _f32, _vp, _i64,
                                           _vp, _vp, _i64, _vp])):
            fn = getattr(L, name)
            fn.restype = ctypes.c_int
            fn.argtypes = args
        L.gemm_a16_s4_workspace.restype = _i64
        L.gemm_a16_s4_workspace.argtypes = [_i64, _i64]
        L.ptc_moe_a16_s4_workspace.restype = _i64
        L.ptc_moe_a16_s4_workspace.argtypes = [_i64] * 5
        L.ptc_rms_norm_backward_workspace.restype = _i64
        L.ptc_rms_norm_backward_workspace.argtypes = [_i64, _i64]
        L.gemm_baseline.restype = ctypes.c_int
        L.gemm_baseline.argtypes = [ctypes.c_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
        L.gemm_status_string.restype = ctypes.c_char_p
        L.gemm_status_string.argtypes = [ctypes.c_int]
        L.gemm_poll_device_error.restype = ctypes.c_int
        L.gemm_poll_device_error.argtypes = []
        L.ptc_kernel_launch_count.restype = ctypes.c_uint64
        L.ptc_kernel_launch_count.argtypes = []
        L.ptc_debug_set_wait_limit.restype = ctypes.c_int
        L.ptc_debug_set_wait_limit.argtypes = [ctypes.c_uint64, _i64]
        L.ptc_set_tuning.restype = ctypes.c_int
        L.ptc_set_tuning.argtypes = [ctypes.c_char_p, _i64]
        _ip = ctypes.POINTER(ctypes.c_int)
        L.ptc_last_launch.restype = ctypes.c_int
        L.ptc_last_launch.argtypes = [_ip, _ip, _ip, _ip]
        L.ptc_last_fp4_launch.restype = ctypes.c_int
        L.ptc_last_fp4_launch.argtypes = [ctypes.POINTER(_i64), _ip, _ip, _ip]
        L.ptc_last_conversion.restype = ctypes.c_int
        L.ptc_last_conversion.argtypes = [_ip]
        _u64p = ctypes.POINTER(ctypes.c_uint64)
        L.ptc_clock_probe_read.restype = ctypes.c_int
        L.ptc_clock_probe_read.argtypes = [_u64p, _u64p, _u64p]
        L.ptc_plan_shape.restype = ctypes.c_int
        L.ptc_plan_shape.argtypes = [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, _ip, _ip, _ip, _ip]
        _lib = L
    return _lib


def _check(status: int) -> int:
    if status != PTC_OK:
        raise PtcError(status, gemm_status_string(status))
    return status


def gemm_status_string(status: int) -> str:
    return lib().gemm_status_string(int(status)).decode()


# ---------------------------------------------------------------- C ABI layer
def gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C[MxN] f32 = A[MxK] f16 (row-major) . B[KxN] f16 (row-major); device addresses."""
    return _check(lib().gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_f16_f16acc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C[MxN] f16 = A[MxK] f16 . B[KxN] f16 with FP16 accumulators; device addresses."""
    return _check(lib().gemm_f16_f16acc(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s8(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C[MxN] s32 = A[MxK] s8 (row-major) . B[KxN] s8 (column-major); device addresses."""
    return _check(lib().gemm_s8(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s8_b_rowmajor(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C[MxN] s32 = A[MxK] s8 (row-major) . B[KxN] s8 (row-major, ldb >= N); device addresses."""
    return _check(lib().gemm_s8_b_rowmajor(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s4(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """C[MxN] s32 = A[MxK] packed s4 . B[KxN] packed s4 (column-major); lda/ldb in nibbles."""
    return _check(lib().gemm_s4(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s8_scaled(M, N, K, A, lda, B, ldb, scale_a, scale_b, C, ldc, out_type, stream=0) -> int:
    """C = out(rn(rn(float(sum_k A_ik B_kj) * scale_a[i]) * scale_b[j])), INT8 operands."""
    return _check(lib().gemm_s8_scaled(M, N, K, A, lda, B, ldb, scale_a, scale_b, C, ldc, out_type, stream))


def gemm_s4_scaled(M, N, K, A, lda, B, ldb, scale_a, scale_b, C, ldc, out_type, stream=0) -> int:
    """As gemm_s8_scaled with packed INT4 operands (lda, ldb in nibbles)."""
    return _check(lib().gemm_s4_scaled(M, N, K, A, lda, B, ldb, scale_a, scale_b, C, ldc, out_type, stream))


def gemm_s8_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """gemm_s8 that allocates nothing: its workspace is a fixed 32 MiB device
    array shared by all calls, for callers that cannot allow a library to
    allocate device memory.  Overlapping calls race; see include/ptc.h."""
    return _check(lib().gemm_s8_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_f16_host(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """gemm_f16 with host-resident A, B, C (asynchronous on `stream`; see include/ptc.h)."""
    return _check(lib().gemm_f16_host(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s8_host(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """gemm_s8 with host-resident A, B, C (asynchronous on `stream`)."""
    return _check(lib().gemm_s8_host(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_s4_host(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """gemm_s4 with host-resident A, B, C (asynchronous on `stream`)."""
    return _check(lib().gemm_s4_host(M, N, K, A, lda, B, ldb, C, ldc, stream))


def gemm_baseline(variant, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """The paper's WMMA / mma.sync kernel families on GB300 (PTC_BASELINE_*); see include/ptc.h."""
    return _check(lib().gemm_baseline(variant, M, N, K, A, lda, B, ldb, C, ldc, stream))


def ptc_dropout(rows, cols, x, ldx, residual, ldr, y, ldy, type, p, seed, offset, stream=0) -> int:
    """y = dropout(x) (+ residual), mask from (seed, offset); device addresses."""
    return _check(lib().ptc_dropout(rows, cols, x, ldx, residual, ldr, y, ldy, type, p, seed, offset, stream))


def ptc_dropout_to(rows, cols, x, ldx, type, residual, ldr, y, ldy, out_type, p, seed, offset, stream=0) -> int:
    """ptc_dropout with a type of its own for y; device addresses."""
    return _check(lib().ptc_dropout_to(rows, cols, x, ldx, type, residual, ldr, y, ldy, out_type, p, seed, offset,
                                       stream))


def ptc_quantize_fp4(rows, cols, x, ldx, type, format, rounding, matrix_scale, codes, pitch, scales, codes_t, pitch_t,
                     scales_t, p, seed, offset, stream=0) -> int:
    """x to microscaled 4-bit rows and / or columns; see include/ptc.h."""
    return _check(lib().ptc_quantize_fp4(rows, cols, x, ldx, type, format, rounding, matrix_scale, codes, pitch,
                                         scales, codes_t, pitch_t, scales_t, p, seed, offset, stream))


def ptc_dequantize_fp4(rows, cols, codes, pitch, scales, format, matrix_scale, y, ldy, type, stream=0) -> int:
    """Values of a microscaled 4-bit matrix; device addresses."""
    return _check(lib().ptc_dequantize_fp4(rows, cols, codes, pitch, scales, format, matrix_scale, y, ldy, type,
                                           stream))


def gemm_fp4(M, N, K, format, A, lda, SA, GA, B, ldb, SB, GB, C, ldc, out_type, stream=0) -> int:
    """C[MxN] = A[MxK] . B[NxK]^T of two microscaled 4-bit matrices (code pitches in bytes)."""
    return _check(lib().gemm_fp4(M, N, K, format, A, lda, SA, GA, B, ldb, SB, GB, C, ldc, out_type, stream))


def gemm_a16_fp4(M, N, K, type, X, ldx, format, W, ldw, SW, GW, C, ldc, stream=0) -> int:
    """C[MxN] = X[MxK] (bfloat16 / binary16) . W[NxK]^T, W microscaled 4-bit."""
    return _check(lib().gemm_a16_fp4(M, N, K, type, X, ldx, format, W, ldw, SW, GW, C, ldc, stream))


def gemm_a16_s4_workspace(M, K) -> int:
    """Bytes of workspace with which gemm_a16_s4 is fastest."""
    return lib().gemm_a16_s4_workspace(M, K)


def gemm_a16_s4(M, N, K, type, X, ldx, W, ldw, group, scale_type, scales, zeros, C, ldc, workspace=None,
                workspace_bytes=0, stream=0) -> int:
    """Few 16-bit tokens times 4-bit integer weights with group scales (include/ptc.h)."""
    return _check(lib().gemm_a16_s4(M, N, K, type, X, ldx, W, ldw, group, scale_type, scales, zeros, C, ldc, workspace,
                                    workspace_bytes, stream))


def ptc_moe_a16_s4_workspace(tokens, hidden, inner, experts, top_k) -> int:
    """Bytes of workspace that ptc_moe_a16_s4 takes; 0 for sizes that it refuses."""
    return lib().ptc_moe_a16_s4_workspace(tokens, hidden, inner, experts, top_k)


def ptc_moe_a16_s4(tokens, hidden, inner, experts, top_k, renormalize, type, X, ldx, router, ldr, router_type, group,
                   scale_type, gate_up, ld_gate_up, expert_gate_up, gate_up_scales, gate_up_zeros, down, ld_down,
                   expert_down, down_scales, down_zeros, Y, ldy, ids, weights, workspace, workspace_bytes, stream=0) -> int:
    """A mixture-of-experts layer for a few tokens (include/ptc.h)."""
    return _check(lib().ptc_moe_a16_s4(tokens, hidden, inner, experts, top_k, renormalize, type, X, ldx, router, ldr,
                                       router_type, group, scale_type, gate_up, ld_gate_up, expert_gate_up, gate_up_scales,
                                       gate_up_zeros, down, ld_down, expert_down, down_scales, down_zeros, Y, ldy, ids,
                                       weights, workspace, workspace_bytes, stream))


def ptc_rms_norm(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type, eps, y, ldy, stream=0) -> int:
    """Root-mean-square norm of rows, with the residual's addition (include/ptc.h)."""
    return _check(lib().ptc_rms_norm(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type, eps, y, ldy,
                                     stream))


def ptc_rms_norm_s8(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type, eps, codes, ldc, scale,
                    stream=0) -> int:
    """The same as 8-bit codes with a scale per row (include/ptc.h)."""
    return _check(lib().ptc_rms_norm_s8(rows, cols, x, ldx, type, residual, ldr, sum, lds, weight, weight_type, eps, codes,
                                        ldc, scale, stream))


def ptc_rms_norm_backward_workspace(rows, cols) -> int:
    """Bytes of workspace that ptc_rms_norm_backward takes."""
    return lib().ptc_rms_norm_backward_workspace(rows, cols)


def ptc_rms_norm_backward(rows, cols, dy, lddy, s, lds, type, ds, ldds, weight, weight_type, eps, dx, lddx, dweight,
                          workspace, workspace_bytes, stream=0) -> int:
    """Gradients of the norm (include/ptc.h)."""
    return _check(lib().ptc_rms_norm_backward(rows, cols, dy, lddy, s, lds, type, ds, ldds, weight, weight_type, eps, dx,
                                              lddx, dweight, workspace, workspace_bytes, stream))


def gemm_poll_device_error() -> int:
    """Status of the device error word (read and cleared); synchronises the device."""
    return int(lib().gemm_poll_device_error())


def ptc_kernel_launch_count() -> int:
    return int(lib().ptc_kernel_launch_count())


def ptc_clock_probe_read():
    """Clock record of the GEMM kernels launched with the "clock_probe" knob
    set, per family (FP16, INT8 route, INT4 route): lists of SM cycles,
    nanoseconds and CTAs summed over CTAs.  Read and cleared; synchronous."""
    cyc, ns, ctas = (ctypes.c_uint64 * 3)(), (ctypes.c_uint64 * 3)(), (ctypes.c_uint64 * 3)()
    _check(lib().ptc_clock_probe_read(cyc, ns, ctas))
    return list(cyc), list(ns), list(ctas)


def ptc_debug_set_wait_limit(timeout_ns: int, stall_tile: int = -1) -> int:
    return _check(lib().ptc_debug_set_wait_limit(int(timeout_ns), int(stall_tile)))


def ptc_set_tuning(key: str, value: int) -> int:
    return _check(lib().ptc_set_tuning(key.encode(), int(value)))


def ptc_plan_shape(M: int, N: int, K: int, prec: int, sms: int = 152,
                   caps: tuple[int, int, int] = (76, 36, 15), with_ring: bool = False):
    """(CTAs per tile, tile width, CTAs per tile's K range) the library would
    launch for an M x N x K product of precision `prec` (0 FP16, 1 INT8,
    2 INT4) on a device of `sms` SMs with cluster capacities `caps` (clusters
    of 2, 4, 8 one-CTA tiles that fit at once), under the current knobs; with
    `with_ring`, a fourth item: whether the integer operands are converted
    inside the GEMM kernel.  Host arithmetic only; the defaults are a GB300's
    figures."""
    c, n, k, r = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().ptc_plan_shape(int(M), int(N), int(K), int(prec), int(sms), int(caps[0]), int(caps[1]),
                                int(caps[2]), ctypes.byref(c), ctypes.byref(n), ctypes.byref(k), ctypes.byref(r)))
    if with_ring:
        return c.value, n.value, k.value, bool(r.value)
    return c.value, n.value, k.value


def ptc_last_launch() -> tuple[int, int, int, int]:
    """(grid CTAs, CTAs per cluster, CTAs sharing a tile's K range, tile
    width) of the calling thread's last GEMM kernel launch."""
    g, c, k, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().ptc_last_launch(ctypes.byref(g), ctypes.byref(c), ctypes.byref(k), ctypes.byref(n)))
    return g.value, c.value, k.value, n.value


def ptc_last_fp4_launch() -> tuple[int, int, int, int]:
    """(grid CTAs, CTAs per cluster, CTAs sharing K, tile columns of gemm_fp4 or
    weight rows per CTA of gemm_a16_fp4) of the calling thread's last 4-bit product."""
    g, c, k, n = _i64(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().ptc_last_fp4_launch(ctypes.byref(g), ctypes.byref(c), ctypes.byref(k), ctypes.byref(n)))
    return g.value, c.value, k.value, n.value


def ptc_last_conversion() -> int:
    """Operand conversion of the calling thread's last GEMM call: 0 none, 1 a
    separate pass into a workspace, 2 inside the GEMM kernel."""
    m = ctypes.c_int(0)
    _check(lib().ptc_last_conversion(ctypes.byref(m)))
    return m.value


# ---------------------------------------------------------------- torch layer
def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _rowmajor(t, name):
    """Row pitch in elements of a 2-D tensor with unit column stride.  A single
    row has no pitch; the smallest one that meets every alignment rule is used."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if t.shape[0] > 1:
        return t.stride(0)
    return max(32, (t.shape[1] + 31) // 32 * 32)


_HOST_FN = {}


def _run(fn, A, B, out, out_shape, out_dtype, M, N, K, lda_scale, stream, sync=True):
    """Device tensors: the device entry point on `stream`.  Host tensors: the
    host entry point (pipelined copies inside the library); the result is
    ready on return unless sync=False, in which case `stream` must be
    synchronised before `out` is read and A, B must be kept alive (and
    unchanged) until then."""
    import torch
    host = A.device.type == "cpu"
    if host != (B.device.type == "cpu"):
        raise ValueError("A and B must both be on the host or both on the device")
    if host:
        hfn = _HOST_FN.get(fn)
        if hfn is None:
            raise ValueError("this product has no host-buffer entry point")
        C = out if out is not None else torch.empty(out_shape, dtype=out_dtype, pin_memory=True)
        if C.device.type != "cpu":
            raise ValueError("host operands need a host result tensor")
        st = _stream(stream)
        hfn(M, N, K, A.data_ptr(), _rowmajor(A, "A") * lda_scale, B.data_ptr(), _rowmajor(B, "B") * lda_scale,
            C.data_ptr(), _rowmajor(C, "C"), st)
        if sync:
            torch.cuda.ExternalStream(st).synchronize() if st else torch.cuda.synchronize()
        return C
    C = out if out is not None else torch.empty(out_shape, dtype=out_dtype, device=A.device)
    fn(M, N, K, A.data_ptr(), _rowmajor(A, "A") * lda_scale, B.data_ptr(), _rowmajor(B, "B") * lda_scale,
       C.data_ptr(), _rowmajor(C, "C"), _stream(stream))
    return C


def matmul_f16(A, B, out=None, stream=None, sync=True):
    """FP16 A (M,K) @ B (K,N) -> float32 (M,N) on the tensor cores (device or host tensors)."""
    import torch
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("matmul_f16 takes float16 operands")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    return _run(gemm_f16, A, B, out, (M, N), torch.float32, M, N, K, 1, stream, sync)


def matmul_f16_f16acc(A, B, out=None, stream=None):
    """FP16 A (M,K) @ B (K,N) -> float16 (M,N), accumulated in FP16 on the tensor cores."""
    import torch
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("matmul_f16_f16acc takes float16 operands")
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    return _run(gemm_f16_f16acc, A, B, out, (M, N), torch.float16, M, N, K, 1, stream)


def matmul_s8(A, Bt, out=None, stream=None, sync=True):
    """INT8 A (M,K) @ B where B (K,N) is column-major, given as Bt (N,K) -> int32 (M,N)."""
    import torch
    if A.dtype != torch.int8 or Bt.dtype != torch.int8:
        raise TypeError("matmul_s8 takes int8 operands")
    M, K = A.shape
    N, K2 = Bt.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    return _run(gemm_s8, A, Bt, out, (M, N), torch.int32, M, N, K, 1, stream, sync)


def matmul_s4(A, Bt, K, out=None, stream=None, sync=True):
    """Packed INT4 A (M, >=K/2 bytes) @ B, B column-major given as Bt (N, >=K/2 bytes),
    two values per byte with the low nibble first -> int32 (M,N)."""
    import torch
    if A.dtype != torch.uint8 or Bt.dtype != torch.uint8:
        raise TypeError("matmul_s4 takes packed uint8 operands")
    M, N = A.shape[0], Bt.shape[0]
    return _run(gemm_s4, A, Bt, out, (M, N), torch.int32, M, N, int(K), 2, stream, sync)


def _out_type(dtype):
    import torch
    table = {torch.float32: PTC_OUT_F32, torch.bfloat16: PTC_OUT_BF16, torch.float16: PTC_OUT_F16}
    if dtype not in table:
        raise TypeError("scaled outputs are float32, bfloat16 or float16")
    return table[dtype]


def _scaled(fn, A, Bt, K, scale_a, scale_b, out_dtype, out, stream, lda_scale):
    import torch
    M, N = A.shape[0], Bt.shape[0]
    if A.device.type == "cpu" or Bt.device.type == "cpu":
        raise ValueError("scaled products take device tensors")
    C = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=A.device)
    for v, n, name in ((scale_a, M, "scale_a"), (scale_b, N, "scale_b")):
        if v is not None and (v.dtype != torch.float32 or v.numel() != n or not v.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 vector of {n} elements")
    fn(M, N, K, A.data_ptr(), _rowmajor(A, "A") * lda_scale, Bt.data_ptr(), _rowmajor(Bt, "B") * lda_scale,
       None if scale_a is None else scale_a.data_ptr(), None if scale_b is None else scale_b.data_ptr(),
       C.data_ptr(), _rowmajor(C, "C"), _out_type(C.dtype), _stream(stream))
    return C


def matmul_s8_scaled(A, Bt, scale_a=None, scale_b=None, out_dtype=None, out=None, stream=None):
    """(A (M,K) int8 @ B, B column-major as Bt (N,K) int8) * scale_a[:,None] * scale_b[None,:]
    -> float32 / bfloat16 / float16 (M,N), with the rounding order of gemm_s8_scaled."""
    import torch
    if A.dtype != torch.int8 or Bt.dtype != torch.int8:
        raise TypeError("matmul_s8_scaled takes int8 operands")
    if A.shape[1] != Bt.shape[1]:
        raise ValueError("inner dimensions differ")
    dt = out.dtype if out is not None else (out_dtype or torch.float32)
    return _scaled(gemm_s8_scaled, A, Bt, A.shape[1], scale_a, scale_b, dt, out, stream, 1)


def matmul_s4_scaled(A, Bt, K, scale_a=None, scale_b=None, out_dtype=None, out=None, stream=None):
    """As matmul_s8_scaled with packed INT4 operands (two per byte, low nibble first)."""
    import torch
    if A.dtype != torch.uint8 or Bt.dtype != torch.uint8:
        raise TypeError("matmul_s4_scaled takes packed uint8 operands")
    dt = out.dtype if out is not None else (out_dtype or torch.float32)
    return _scaled(gemm_s4_scaled, A, Bt, int(K), scale_a, scale_b, dt, out, stream, 2)


_HOST_FN.update({gemm_f16: gemm_f16_host, gemm_s8: gemm_s8_host, gemm_s4: gemm_s4_host})


# ---------------------------------------------------------------- 4-bit operators on tensors
# These calls are a few microseconds on the device at decoding sizes, so their
# marshalling is native: _native.so (csrc/binding.cpp) checks the tensors,
# allocates results and calls the C ABI.  With `stream` (a torch stream or a
# handle) a call runs as under torch.cuda.stream(stream): it is ordered after that
# stream's work alone, so the caller waits for its inputs and for the result.
# The tensors' memory needs no such care: results come from that stream's, and
# inputs and results may be released while it runs.  The operators are outside
# autograd: a tensor that requires grad is refused unless gradients are off.
_FP4 = {"mxfp4": (PTC_FP4_MX, 32), "nvfp4": (PTC_FP4_NV, 16)}
_ROUNDING = {"nearest": PTC_ROUND_NEAREST, "stochastic": PTC_ROUND_STOCHASTIC}
_native = None


def _load_native():
    """The native module, bound to libptc by the first call."""
    global _native
    import importlib
    import torch  # noqa: F401  (its libraries are what the module links against)
    path = os.path.join(_HERE, "_native.so")
    if not os.path.exists(path):
        raise RuntimeError(f"_native.so is not built ({path}); run __graft_entry__.build()")
    n = importlib.import_module(__name__ + "._native")
    L = lib()
    n.init(*(ctypes.cast(getattr(L, f), _vp).value for f in ("ptc_dropout_to", "ptc_quantize_fp4",
                                                             "ptc_dequantize_fp4", "gemm_fp4", "gemm_a16_fp4",
                                                             "gemm_a16_s4_workspace", "gemm_a16_s4", "ptc_moe_a16_s4_workspace",
                                                             "ptc_moe_a16_s4", "ptc_rms_norm", "ptc_rms_norm_s8",
                                                             "ptc_rms_norm_backward_workspace",
                                                             "ptc_rms_norm_backward")),
           _check, _stream, Fp4Matrix, S4Matrix)
    _native = n
    return n


def fp4_scale_bytes(rows: int, cols: int, fmt: str) -> int:
    """Bytes of the tiled scales of `rows` rows of `cols` values."""
    blocks = -(-cols // _FP4[fmt][1])
    return -(-rows // 128) * -(-blocks // 4) * 512


class Fp4Matrix:
    """A microscaled 4-bit matrix of ``codes.shape[0]`` rows of ``K`` values.

    codes: uint8 (rows, >= 16 * ceil(K / 32)) with unit column stride, a row pitch
        that is a multiple of 16 bytes, and zeros past K
    scales: contiguous uint8 of ``fp4_scale_bytes(rows, K, fmt)`` bytes in the
        tiled layout of include/ptc.h (:meth:`tile_scales` makes it from rows)
    fmt: "mxfp4" or "nvfp4"; tensor_scale: None, or (nvfp4) a float32 device
        tensor of one element, 0 .. 2^100, that scales the whole matrix.
    """

    __slots__ = ("_codes", "_scales", "_K", "_fmt", "_ts")

    def __init__(self, codes, scales, K, fmt="mxfp4", tensor_scale=None):
        (_native or _load_native()).check_matrix(codes, scales, K, fmt, tensor_scale)
        self._codes, self._scales, self._K, self._fmt, self._ts = codes, scales, K, fmt, tensor_scale

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    tensor_scale = property(lambda self: self._ts)
    K = property(lambda self: self._K)
    fmt = property(lambda self: self._fmt)
    shape = property(lambda self: (self._codes.shape[0], self._K))
    device = property(lambda self: self._codes.device)

    def record_stream(self, stream):
        """As torch.Tensor.record_stream, for every tensor of the matrix."""
        for t in (self._codes, self._scales, self._ts):
            if t is not None:
                t.record_stream(stream)

    @staticmethod
    def tile_scales(scales):
        """Row-major scale bytes (rows, blocks) to the tiled layout (laid out once, e.g. when weights are loaded)."""
        import torch
        r, b = scales.shape
        if r == 0 or b == 0:
            return scales.reshape(-1)
        s = torch.nn.functional.pad(scales, (0, -b % 4, 0, -r % 128))
        return s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)

    def row_scales(self):
        """Row-major scale bytes (rows, blocks)."""
        r, b = self._codes.shape[0], -(-self._K // _FP4[self._fmt][1])
        rt, kt = -(-r // 128), -(-b // 4)
        s = self._scales.view(-1)[:fp4_scale_bytes(r, self._K, self._fmt)].view(rt, kt, 32, 4, 4)
        return s.permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:r, :b]


def dropout(x, p, seed, offset=0, residual=None, out=None, stream=None, out_dtype=None):
    """``x`` with each element dropped with probability ``p`` (kept ones scaled so
    that the expectation is x's), plus ``residual`` if given; float32, bfloat16
    or float16 (rows, cols).  The mask is a function of (seed, offset, row,
    column) and is never stored: the backward pass is the same call on the
    gradient (made by the caller: autograd does not see this call, and ``x`` must
    not require grad while gradients are on).  ``out`` may be ``x`` or ``residual``.  ``out_dtype`` is x's dtype;
    float32 x without a residual may also give bfloat16 or float16, rounded once."""
    return (_native or _load_native()).dropout(x, p, seed, offset, residual, out, stream, out_dtype)


def quantize_fp4(x, fmt="mxfp4", transposed=False, rounding="nearest", tensor_scale=None, p=0.0, seed=0, offset=0,
                 stream=None):
    """``x`` (rows, cols) as a microscaled 4-bit :class:`Fp4Matrix`.

    transposed: False for blocks along the rows of x; True for the matrix of
        x's columns (cols, rows), which a product that contracts over x's rows
        takes; "both" for the pair (one pass over x).
    rounding: "nearest" (ties to even) or "stochastic" (16 bits per element from seed
        and offset: the mean is the value, down to 2^-16 of the gap between codes).
    tensor_scale: see :class:`Fp4Matrix`; the largest magnitude / 2688 uses the
        whole range, and 0 (that of zeros) gives zeros.  With p > 0 the largest
        magnitude is that of the kept values, 1 / (1 - p) times x's: with x's own
        the largest blocks saturate.
    p: with p > 0 the values are ``dropout(x, p, seed, offset)`` in float32.
    """
    how = _ROUNDING.get(rounding)
    if how is None:
        raise ValueError("rounding is 'nearest' or 'stochastic'")
    which = 0 if transposed is False else 1 if transposed is True else 2
    if which == 2 and transposed != "both":
        raise ValueError("transposed is False, True or 'both'")
    return (_native or _load_native()).quantize(x, fmt, which, how, tensor_scale, p, seed, offset, stream)


def dequantize_fp4(q, dtype=None, out=None, stream=None):
    """The values of an :class:`Fp4Matrix` as float32, bfloat16 (default) or float16."""
    return (_native or _load_native()).dequantize(q, dtype, out, stream)


def matmul_fp4(A, Bt, out_dtype=None, out=None, stream=None):
    """A (M,K) @ B with B given as Bt (N,K), both :class:`Fp4Matrix` of one format
    -> float32, bfloat16 (default) or float16 (M,N), summed in FP32 on the
    block-scaled tensor cores."""
    return (_native or _load_native()).matmul(A, Bt, out_dtype, out, stream)


def matmul_a16_fp4(x, Wt, out=None, stream=None):
    """x (M,K) bfloat16 or float16 @ W given as Wt (N,K) :class:`Fp4Matrix` -> x's
    dtype (M,N), summed in FP32: the product of a decoding step, for M up to 16
    rows (more are taken 16 at a time; quantise x and use :func:`matmul_fp4`
    for many)."""
    return (_native or _load_native()).matmul_a16(x, Wt, out, stream)


# ---------------------------------------------------------------- grouped 4-bit integer weights
class S4Matrix:
    """A matrix of rows of ``K`` weights (c - z) s: 4-bit integer codes c with a scale s,
    and a zero z if given, per row and group of ``group`` codes; or several such matrices
    of one size (the experts of :func:`moe_a16_s4`).

    codes: uint8 (rows, >= ceil(K / 2)) or (experts, rows, >= ceil(K / 2)), the packed INT4
        of :func:`matmul_s4`: two's complement, two per byte, the low nibble first, unit
        column stride, rows (and experts) a multiple of 16 bytes apart
    scales: contiguous bfloat16 or float16 in tiles of 16 rows (:meth:`tile_scales` makes
        them from (rows, groups))
    group: 32, 64 or a multiple of 128; at least K for one scale per row
    zeros: None, or like the scales
    """

    __slots__ = ("_codes", "_scales", "_K", "_group", "_zeros")

    def __init__(self, codes, scales, K, group=128, zeros=None):
        (_native or _load_native()).check_s4(codes, scales, K, group, zeros)
        self._codes, self._scales, self._K, self._group, self._zeros = codes, scales, K, group, zeros

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    zeros = property(lambda self: self._zeros)
    K = property(lambda self: self._K)
    group = property(lambda self: self._group)
    shape = property(lambda self: (*self._codes.shape[:-1], self._K))
    device = property(lambda self: self._codes.device)

    def record_stream(self, stream):
        """As torch.Tensor.record_stream, for every tensor of the matrix."""
        for t in (self._codes, self._scales, self._zeros):
            if t is not None:
                t.record_stream(stream)

    @staticmethod
    def tile_scales(scales):
        """(..., rows, groups) to the tiled layout (laid out once, e.g. when weights are loaded)."""
        import torch
        r, n = scales.shape[-2:]
        if scales.numel() == 0:
            return scales.reshape(-1)
        t = torch.nn.functional.pad(scales, (0, 0, 0, -r % 16))
        return t.reshape(*scales.shape[:-2], -1, 16, n).transpose(-1, -2).reshape(-1).contiguous()

    @classmethod
    def quantize(cls, w, group=128, zeros=False, dtype=None):
        """Weights (rows, K) or (experts, rows, K) rounded to nearest, when they are loaded: scales
        max |w| / 7 of a group, or with zeros (max - min) / 15 about a whole zero.  ``dtype`` of
        the scales: w's, or bfloat16 for float32."""
        import torch
        dtype = dtype or (w.dtype if w.dtype in (torch.bfloat16, torch.float16) else torch.bfloat16)
        K, groups = w.shape[-1], -(-w.shape[-1] // group)
        v = torch.nn.functional.pad(w.detach().float(), (0, groups * group - K))
        v = v.reshape(*w.shape[:-1], groups, group)
        if zeros:
            low, high = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
            scale = ((high - low) / 15).to(dtype)
            zero = torch.where(scale > 0, -8 - low / scale.float(), 0.0).round().clamp(-8, 7).to(dtype)
        else:
            scale, zero = (v.abs().amax(-1) / 7).to(dtype), None
        code = torch.where(scale.float().unsqueeze(-1) > 0, v / scale.float().unsqueeze(-1), 0.0)
        code = code if zero is None else code + zero.float().unsqueeze(-1)
        code = code.round().clamp(-8, 7).to(torch.int8).reshape(*w.shape[:-1], -1)[..., :K].view(torch.uint8) & 15
        code = torch.nn.functional.pad(code, (0, -K % 32))
        return cls((code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), cls.tile_scales(scale), K, group,
                   None if zero is None else cls.tile_scales(zero))


def matmul_a16_s4(x, Wt, out=None, stream=None):
    """x (M,K) bfloat16 or float16 @ W given as Wt (N,K) :class:`S4Matrix` -> x's dtype (M,N),
    summed in FP32: the product of a decoding step, for M up to 16 rows (more are taken 16
    at a time)."""
    return (_native or _load_native()).matmul_a16_s4(x, Wt, out, stream)


def moe_a16_s4(x, router, gate_up, down, top_k, renormalize=True, out=None, return_routing=False, stream=None):
    """A mixture-of-experts layer for up to 64 tokens x (tokens, hidden) bfloat16 or float16
    -> x's dtype: each token's ``top_k`` experts of the largest logits x router^T, their
    weights p the softmax over the chosen (``renormalize``) or over all experts, and the
    sum of p * down(silu(gate(x)) * up(x)).

    router: (experts, hidden), x's dtype or float32
    gate_up: :class:`S4Matrix` of (experts, 2 inner, hidden), the gate's rows first; down: of
        (experts, hidden, inner), with the same group and scales' dtype
    return_routing: also give the chosen experts (tokens, top_k) int32, in falling order
        of their logits (equal ones: the lowest first), and their weights p in float32

    tokens * top_k is at most 512.  Outside autograd, as the other products."""
    return (_native or _load_native()).moe_a16_s4(x, router, gate_up, down, top_k, renormalize, out, return_routing, stream)


# ---------------------------------------------------------------- norms on tensors
def rms_norm(x, weight=None, eps=1e-6, residual=None, out=None, sum_out=None, stream=None):
    """``s / sqrt(mean(s^2) + eps) * weight`` of every row of x (rows, cols) float32,
    bfloat16 or float16, computed in float32 and rounded once; s is x, or with a
    ``residual`` x + residual rounded to x's dtype.  Returns y, or with a residual (y,
    s).  ``weight`` (cols,): x's dtype or float32, None for ones.  ``out`` or
    ``sum_out`` may be x or the residual.  Outside autograd, as the 4-bit operators;
    :func:`rms_norm_backward` is the backward pass."""
    return (_native or _load_native()).rms_norm(x, weight, eps, residual, out, sum_out, stream)


def rms_norm_s8(x, weight=None, eps=1e-6, residual=None, sum_out=None, stream=None):
    """:func:`rms_norm` as int8 codes (rows, cols) with a float32 scale per row, what
    :func:`matmul_s8_scaled` takes as A and scale_a (the codes' rows are a multiple of
    16 bytes apart).  Returns (codes, scale), or with a residual (codes, scale, s).  A
    row with an infinity or NaN has codes 0 and scale NaN."""
    return (_native or _load_native()).rms_norm_s8(x, weight, eps, residual, sum_out, stream)


def rms_norm_backward(dy, s, weight=None, eps=1e-6, dsum=None, out=None, stream=None):
    """(dx, dweight) of :func:`rms_norm` from the gradient dy of y and the s that was
    normalised (x, or the returned sum).  ``dsum`` is the gradient that reaches s from
    elsewhere (the residual stream's) and is added to dx, which is the gradient of x
    and of the residual; dweight is float32 (cols,), added over the rows in a fixed
    order.  ``out`` may be dy, s or dsum."""
    return (_native or _load_native()).rms_norm_backward(dy, s, weight, eps, dsum, out, stream)
