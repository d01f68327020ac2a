"""Python binding of ``libswiglu_mlp.so`` (C ABI in ``include/swiglu_mlp.h``).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  There is no fallback of any kind; if the shared
library has not been built this module raises on first use.  (ctypes, but for
the ``*_into`` helpers of the expert MLP, which go through the CPython module
``_binding``.)

Functions with the C names take the C arguments (pointers may be given as
ints or as tensors, whose ``data_ptr()`` is used; ``stream`` may be a
``torch.cuda.Stream``, a raw handle, or None for the current torch stream).
Each raises :class:`SwgError` when the library returns a non-zero status.
The ``*_into`` helpers derive sizes and strides from row-major torch tensors.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "SwgError", "OP_N", "OP_T", "F16_F32OUT", "BF16", "F16", "BF16_F32OUT", "E4M3_BF16OUT",
    "E4M3_F32OUT", "swiglu_mlp_fp8",
    "gemm", "gemm_ex", "gemm_splitk_noalloc", "swiglu_mlp", "swiglu_mlp_dual", "swiglu_mlp_forward", "swiglu_interleave", "status_string",
    "get_device_error", "debug_workspace_guards", "launch_count", "shutdown", "gemm_into", "selftest_wait_timeout",
    "swiglu_mlp_into", "interleave_weights", "library_path", "load",
    "MXFP4", "NVFP4", "TYPE_F16", "TYPE_BF16", "TYPE_F32", "MAX_GROUPS",
    "gemm_grouped", "gemm_grouped_wgrad", "swiglu_grouped", "swiglu_grouped_grad",
    "mx4_scale_bytes", "mx4_quantize", "mx4_dequantize", "gemm_mx4", "swiglu_mx4",
    "gemm_grouped_into", "gemm_grouped_wgrad_into", "swiglu_grouped_into",
    "swiglu_grouped_grad_into", "mx4_alloc", "mx4_quantize_into", "mx4_dequantize_into",
    "gemm_mx4_into", "swiglu_mx4_into",
    "SOFTMAX", "SIGMOID", "MAX_EXPERTS", "MAX_TOP", "MAX_EXPERT_GROUPS",
    "expert_route", "expert_sort", "expert_route_grad", "expert_dispatch", "expert_combine",
    "expert_combine_grad", "w4_quantize", "w4_dequantize", "gemm_w4", "swiglu_w4",
    "expert_plan_alloc", "expert_route_into", "expert_sort_into", "expert_route_grad_into",
    "expert_dispatch_into", "expert_combine_into", "expert_combine_grad_into", "w4_alloc",
    "w4_quantize_into", "w4_dequantize_into", "gemm_w4_into", "swiglu_w4_into",
]

OP_N, OP_T = 0, 1
F16_F32OUT, BF16, F16, BF16_F32OUT, E4M3_BF16OUT, E4M3_F32OUT = 0, 1, 2, 3, 4, 5
MXFP4, NVFP4 = 0, 1
TYPE_F16, TYPE_BF16, TYPE_F32 = 0, 1, 2
MAX_GROUPS = 1024
SOFTMAX, SIGMOID = 0, 1
MAX_EXPERTS, MAX_TOP, MAX_EXPERT_GROUPS = 1024, 32, 32
STATUS = {0: "SWG_OK", 1: "SWG_ERR_INVALID_ARG", 2: "SWG_ERR_MISALIGNED",
          3: "SWG_ERR_UNSUPPORTED", 4: "SWG_ERR_CUDA", 5: "SWG_ERR_NO_MEMORY",
          6: "SWG_ERR_DEVICE_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libswiglu_mlp.so")
_lock = threading.Lock()
_lib = None


class SwgError(RuntimeError):
    """A non-zero status from the C ABI; for SWG_ERR_CUDA the message also
    names the CUDA error behind it (swg_last_cuda_error)."""

    def __init__(self, status: int, where: str, cuda_error: int = 0, cuda_name: str = ""):
        self.status = int(status)
        self.cuda_error = int(cuda_error)
        msg = f"{where}: {STATUS.get(self.status, 'SWG_ERR_UNKNOWN')} ({self.status})"
        if self.cuda_error:
            msg += f" [CUDA {self.cuda_error}: {cuda_name}]"
        super().__init__(msg)


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads the shared library (once).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(_LIB_PATH)
        i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        lib.gemm.argtypes = [i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, i32, vp]
        lib.gemm.restype = i32
        lib.gemm_ex.argtypes = [i32, i32, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, i32,
                                i32, vp]
        lib.gemm_ex.restype = i32
        lib.gemm_splitk_noalloc.argtypes = [i32, i32, i64, i64, i64, f32, vp, i64, vp, i64,
                                            f32, vp, i64, i32, i32, vp]
        lib.gemm_splitk_noalloc.restype = i32
        lib.swiglu_mlp.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        lib.swiglu_mlp.restype = i32
        lib.swiglu_mlp_fp8.argtypes = [vp, vp, vp, i64, i64, i64, f32, vp]
        lib.swiglu_mlp_fp8.restype = i32
        lib.swiglu_mlp_dual.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        lib.swiglu_mlp_dual.restype = i32
        lib.swiglu_mlp_forward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, f32, vp]
        lib.swiglu_mlp_forward.restype = i32
        lib.swiglu_interleave.argtypes = [vp, vp, vp, i64, i64, vp]
        lib.swiglu_interleave.restype = i32
        lib.swg_status_string.argtypes = [i32]
        lib.swg_status_string.restype = ctypes.c_char_p
        lib.swg_get_device_error.argtypes = [vp]
        lib.swg_get_device_error.restype = i32
        lib.swg_selftest_wait_timeout.argtypes = [i64, vp]
        lib.swg_selftest_wait_timeout.restype = i32
        lib.swg_launch_count.argtypes = []
        lib.swg_launch_count.restype = ctypes.c_uint64
        lib.swg_shutdown.argtypes = []
        lib.swg_shutdown.restype = None
        lib.swg_last_cuda_error.argtypes = []
        lib.swg_last_cuda_error.restype = i32
        lib.swg_cuda_error_name.argtypes = [i32]
        lib.swg_cuda_error_name.restype = ctypes.c_char_p
        lib.swg_debug_workspace_guards.argtypes = [vp, ctypes.POINTER(i64)]
        lib.swg_debug_workspace_guards.restype = i32
        lib.gemm_grouped.argtypes = [i32, i64, i64, i64, i64, f32, vp, i64, vp, i64, i64, vp, f32,
                                     vp, i64, i32, vp]
        lib.gemm_grouped_wgrad.argtypes = [i64, i64, i64, i64, f32, vp, i64, vp, i64, vp, f32, vp,
                                           i64, i64, i32, vp]
        lib.swiglu_grouped.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, vp]
        lib.swiglu_grouped_grad.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp]
        lib.mx4_scale_bytes.argtypes = [i32, i64, i64, i64]
        lib.mx4_scale_bytes.restype = i64
        lib.mx4_quantize.argtypes = [i32, i64, i64, i64, vp, i64, i32, f32, vp, vp, i64, vp, vp]
        lib.mx4_dequantize.argtypes = [i32, i64, i64, i64, vp, i64, vp, f32, vp, vp, i64, i32, vp]
        lib.gemm_mx4.argtypes = [i32, i64, i64, i64, i64, f32, vp, i64, vp, vp, i64, i64, vp, vp,
                                 f32, vp, i64, i32, vp]
        lib.swiglu_mx4.argtypes = [i32, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, f32, vp]
        lib.expert_route.argtypes = [i32, i64, i64, i64, vp, i64, i32, vp, i64, i64, i32, i32, f32,
                                     vp, vp, vp, vp, vp, vp]
        lib.expert_sort.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp]
        lib.expert_route_grad.argtypes = [i32, i64, i64, i64, vp, i64, i32, vp, i32, f32, vp, vp,
                                          i64, vp]
        lib.expert_dispatch.argtypes = [i64, i64, i64, i64, vp, i64, i32, vp, vp, i64, vp]
        lib.expert_combine.argtypes = [i64, i64, i64, i64, vp, i64, i32, vp, vp, f32, vp, i64, i32,
                                       vp]
        lib.expert_combine_grad.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, i32, vp, vp, vp,
                                            i64, vp, vp]
        lib.w4_quantize.argtypes = [i64, i64, i64, vp, i64, i32, i64, vp, vp, vp, i64, i32, vp]
        lib.w4_dequantize.argtypes = [i64, i64, i64, vp, vp, vp, i64, i32, i64, vp, i64, i32, vp]
        lib.gemm_w4.argtypes = [i64, i64, i64, i64, f32, vp, i64, vp, vp, vp, i64, i64, vp, f32, vp,
                                i64, i32, i32, vp]
        lib.swiglu_w4.argtypes = [i64, i64, i64, i64, f32, vp, i64, vp, vp, vp, i64, i64, vp, vp,
                                  i64, i32, vp]
        for name in ("gemm_grouped", "gemm_grouped_wgrad", "swiglu_grouped",
                     "swiglu_grouped_grad", "mx4_quantize", "mx4_dequantize", "gemm_mx4",
                     "swiglu_mx4", "expert_route", "expert_sort", "expert_route_grad",
                     "expert_dispatch", "expert_combine", "expert_combine_grad", "w4_quantize",
                     "w4_dequantize", "gemm_w4", "swiglu_w4"):
            getattr(lib, name).restype = i32
        _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None    # torch's accessor of the current raw stream handle, once found
_device = None        # torch's accessor of the current device, once CUDA is initialised


def _current_stream():
    """The calling thread's current torch stream on the current device as a
    raw handle (None without CUDA).  torch's raw accessor is used when it has
    one: building a torch.cuda.Stream object per call costs several
    microseconds of host time."""
    global _raw_stream, _device
    if _device is None:
        import torch
        if not torch.cuda.is_available():
            return None
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = get if get is not None else (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        torch.cuda.current_device()       # initialises CUDA; the accessor alone does not
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_stream(_device())


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str) -> int:
    if rc != 0:
        code, name = 0, ""
        if rc == 4:                     # SWG_ERR_CUDA
            code = load().swg_last_cuda_error()
            name = load().swg_cuda_error_name(code).decode()
        raise SwgError(rc, where, code, name)
    return rc


def gemm(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype, stream=None):
    """D = alpha * op(A) op(B) + beta * C, in place over C (see the C header)."""
    return _check(load().gemm(int(transA), int(transB), int(M), int(N), int(K), float(alpha),
                              _ptr(A), int(lda), _ptr(B), int(ldb), float(beta), _ptr(C),
                              int(ldc), int(dtype), _stream(stream)), "gemm")


def gemm_ex(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype, split_k,
            stream=None):
    return _check(load().gemm_ex(int(transA), int(transB), int(M), int(N), int(K), float(alpha),
                                 _ptr(A), int(lda), _ptr(B), int(ldb), float(beta), _ptr(C),
                                 int(ldc), int(dtype), int(split_k), _stream(stream)), "gemm_ex")


def gemm_splitk_noalloc(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype,
                        split_k=0, stream=None):
    """Split-K GEMM that allocates no device memory: its partial sums live in
    a fixed array inside the library (see the C header for the size limit and
    the sharing rules)."""
    return _check(load().gemm_splitk_noalloc(int(transA), int(transB), int(M), int(N), int(K),
                                             float(alpha), _ptr(A), int(lda), _ptr(B), int(ldb),
                                             float(beta), _ptr(C), int(ldc), int(dtype),
                                             int(split_k), _stream(stream)),
                  "gemm_splitk_noalloc")


def swiglu_mlp(A, W_fused, Y, M, N, K, stream=None):
    """Y = SiLU(A W1) (.) (A W2) over the interleaved W_fused (see the C header)."""
    return _check(load().swiglu_mlp(_ptr(A), _ptr(W_fused), _ptr(Y), int(M), int(N), int(K),
                                    _stream(stream)), "swiglu_mlp")


def swiglu_mlp_fp8(A, W_fused_t, Y, M, N, K, scale, stream=None):
    """Y = SiLU(s A W1) (.) (s A W2) from e4m3 A [M, K] and the transposed
    interleaved e4m3 weight [2N, K] (see the C header)."""
    return _check(load().swiglu_mlp_fp8(_ptr(A), _ptr(W_fused_t), _ptr(Y), int(M), int(N),
                                        int(K), float(scale), _stream(stream)), "swiglu_mlp_fp8")


def swiglu_mlp_dual(A, W1, W2, Y, M, N, K, stream=None):
    """Y = SiLU(A W1) (.) (A W2) from separate K x N weights (see the C header)."""
    return _check(load().swiglu_mlp_dual(_ptr(A), _ptr(W1), _ptr(W2), _ptr(Y), int(M), int(N),
                                         int(K), _stream(stream)), "swiglu_mlp_dual")


def swiglu_mlp_forward(A, W_fused, W_down, Y, Out, M, N, K, beta=0.0, stream=None):
    """Out = (SiLU(A W1) (.) (A W2)) W_down + beta * Out (see the C header)."""
    return _check(load().swiglu_mlp_forward(_ptr(A), _ptr(W_fused), _ptr(W_down), _ptr(Y),
                                            _ptr(Out), int(M), int(N), int(K), float(beta),
                                            _stream(stream)), "swiglu_mlp_forward")


def swiglu_interleave(W1, W2, W_fused, K, N, stream=None):
    return _check(load().swiglu_interleave(_ptr(W1), _ptr(W2), _ptr(W_fused), int(K), int(N),
                                           _stream(stream)), "swiglu_interleave")


def gemm_grouped(transB, G, M, N, K, alpha, A, lda, B, ldb, strideB, offsets, beta, C, ldc,
                 dtype, stream=None):
    """C = alpha * A op(B_g) + beta * C for the rows of every group (see the C header)."""
    return _check(load().gemm_grouped(int(transB), int(G), int(M), int(N), int(K), float(alpha),
                                      _ptr(A), int(lda), _ptr(B), int(ldb), int(strideB),
                                      _ptr(offsets), float(beta), _ptr(C), int(ldc), int(dtype),
                                      _stream(stream)), "gemm_grouped")


def gemm_grouped_wgrad(G, M, N, K, alpha, A, lda, D, ldd, offsets, beta, C, ldc, strideC, dtype,
                       stream=None):
    """C_g = alpha * A_g^T D_g + beta * C_g (see the C header)."""
    return _check(load().gemm_grouped_wgrad(int(G), int(M), int(N), int(K), float(alpha), _ptr(A),
                                            int(lda), _ptr(D), int(ldd), _ptr(offsets),
                                            float(beta), _ptr(C), int(ldc), int(strideC),
                                            int(dtype), _stream(stream)), "gemm_grouped_wgrad")


def swiglu_grouped(A, W_fused, Y, offsets, G, M, N, K, stream=None):
    """Y = SiLU(A W1_g) (.) (A W2_g) for the rows of every group (see the C header)."""
    return _check(load().swiglu_grouped(_ptr(A), _ptr(W_fused), _ptr(Y), _ptr(offsets), int(G),
                                        int(M), int(N), int(K), _stream(stream)),
                  "swiglu_grouped")


def swiglu_grouped_grad(A, W_fused, dY, Y, dH, offsets, G, M, N, K, stream=None):
    """The gradient of swiglu_grouped in Gate and Up, and Y (see the C header)."""
    return _check(load().swiglu_grouped_grad(_ptr(A), _ptr(W_fused), _ptr(dY), _ptr(Y), _ptr(dH),
                                             _ptr(offsets), int(G), int(M), int(N), int(K),
                                             _stream(stream)), "swiglu_grouped_grad")


def mx4_scale_bytes(format, G, M, K) -> int:
    """Bytes of scale tiles that are enough for any offsets (see the C header)."""
    n = int(load().mx4_scale_bytes(int(format), int(G), int(M), int(K)))
    if n < 0:
        raise SwgError(1, "mx4_scale_bytes")
    return n


def mx4_quantize(format, G, M, K, X, ldx, xtype, scale, offsets, Q, ldq, S, stream=None):
    """X * scale to 4-bit codes and scale tiles (see the C header)."""
    return _check(load().mx4_quantize(int(format), int(G), int(M), int(K), _ptr(X), int(ldx),
                                      int(xtype), float(scale), _ptr(offsets), _ptr(Q), int(ldq),
                                      _ptr(S), _stream(stream)), "mx4_quantize")


def mx4_dequantize(format, G, M, K, Q, ldq, S, scale, offsets, X, ldx, xtype, stream=None):
    """The values of 4-bit codes and scale tiles, times scale (see the C header)."""
    return _check(load().mx4_dequantize(int(format), int(G), int(M), int(K), _ptr(Q), int(ldq),
                                        _ptr(S), float(scale), _ptr(offsets), _ptr(X), int(ldx),
                                        int(xtype), _stream(stream)), "mx4_dequantize")


def gemm_mx4(format, G, M, N, K, alpha, A, lda, SA, B, ldb, strideB, SB, offsets, beta, C, ldc,
             ctype, stream=None):
    """C = alpha * A B_g^T + beta * C with 4-bit A and B (see the C header)."""
    return _check(load().gemm_mx4(int(format), int(G), int(M), int(N), int(K), float(alpha),
                                  _ptr(A), int(lda), _ptr(SA), _ptr(B), int(ldb), int(strideB),
                                  _ptr(SB), _ptr(offsets), float(beta), _ptr(C), int(ldc),
                                  int(ctype), _stream(stream)), "gemm_mx4")


def swiglu_mx4(format, A, SA, W, SW, Y, offsets, G, M, N, K, alpha, stream=None):
    """Y = SiLU(alpha A W1_g) (.) (alpha A W2_g) with 4-bit A and W (see the C header)."""
    return _check(load().swiglu_mx4(int(format), _ptr(A), _ptr(SA), _ptr(W), _ptr(SW), _ptr(Y),
                                    _ptr(offsets), int(G), int(M), int(N), int(K), float(alpha),
                                    _stream(stream)), "swiglu_mx4")


def expert_route(score, T, E, top, logits, ldl, type, bias, groups, top_groups, group_sum, normalise,
                 scale, experts, weights, offsets, source, position, stream=None):
    """The experts of each token, their weights and the plan of rows (see the C header)."""
    return _check(load().expert_route(int(score), int(T), int(E), int(top), _ptr(logits), int(ldl),
                                      int(type), _ptr(bias), int(groups), int(top_groups),
                                      int(group_sum), int(normalise), float(scale), _ptr(experts),
                                      _ptr(weights), _ptr(offsets), _ptr(source), _ptr(position),
                                      _stream(stream)), "expert_route")


def expert_sort(T, E, top, experts, offsets, source, position, stream=None):
    """The plan of rows sorted by expert (see the C header)."""
    return _check(load().expert_sort(int(T), int(E), int(top), _ptr(experts), _ptr(offsets),
                                     _ptr(source), _ptr(position), _stream(stream)), "expert_sort")


def expert_route_grad(score, T, E, top, logits, ldl, type, experts, normalise, scale, d_weights,
                      d_logits, ldd, stream=None):
    """The gradient of the logits from that of the weights (see the C header)."""
    return _check(load().expert_route_grad(int(score), int(T), int(E), int(top), _ptr(logits),
                                           int(ldl), int(type), _ptr(experts), int(normalise),
                                           float(scale), _ptr(d_weights), _ptr(d_logits), int(ldd),
                                           _stream(stream)), "expert_route_grad")


def expert_dispatch(T, R, D, top, X, ldx, type, position, rows, ldr, stream=None):
    """rows[position[t, j]] = X[t] (see the C header)."""
    return _check(load().expert_dispatch(int(T), int(R), int(D), int(top), _ptr(X), int(ldx),
                                         int(type), _ptr(position), _ptr(rows), int(ldr),
                                         _stream(stream)), "expert_dispatch")


def expert_combine(T, R, D, top, rows, ldr, type, position, weights, beta, out, ldo, otype,
                   stream=None):
    """out[t] = sum_j weights[t, j] rows[position[t, j]] + beta out[t] (see the C header)."""
    return _check(load().expert_combine(int(T), int(R), int(D), int(top), _ptr(rows), int(ldr),
                                        int(type), _ptr(position), _ptr(weights), float(beta),
                                        _ptr(out), int(ldo), int(otype), _stream(stream)),
                  "expert_combine")


def expert_combine_grad(T, R, D, top, d_out, ldd, rows, ldr, type, position, weights, d_rows, lddr,
                        d_weights, stream=None):
    """The gradients of expert_combine in rows and weights (see the C header)."""
    return _check(load().expert_combine_grad(int(T), int(R), int(D), int(top), _ptr(d_out), int(ldd),
                                             _ptr(rows), int(ldr), int(type), _ptr(position),
                                             _ptr(weights), _ptr(d_rows), int(lddr),
                                             _ptr(d_weights), _stream(stream)),
                  "expert_combine_grad")


def w4_quantize(G, N, K, X, ldx, xtype, group, Q, S, Z, lds, stype, stream=None):
    """X to 4-bit codes, group scales and zero points (see the C header)."""
    return _check(load().w4_quantize(int(G), int(N), int(K), _ptr(X), int(ldx), int(xtype),
                                     int(group), _ptr(Q), _ptr(S), _ptr(Z), int(lds), int(stype),
                                     _stream(stream)), "w4_quantize")


def w4_dequantize(G, N, K, Q, S, Z, lds, stype, group, X, ldx, xtype, stream=None):
    """The values of 4-bit weights (see the C header)."""
    return _check(load().w4_dequantize(int(G), int(N), int(K), _ptr(Q), _ptr(S), _ptr(Z), int(lds),
                                       int(stype), int(group), _ptr(X), int(ldx), int(xtype),
                                       _stream(stream)), "w4_dequantize")


def gemm_w4(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, beta, C, ldc, type, ctype,
            stream=None):
    """C = alpha * A W_g^T + beta * C with weights of 4 bits (see the C header)."""
    return _check(load().gemm_w4(int(G), int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                 _ptr(Q), _ptr(S), _ptr(Z), int(lds), int(group), _ptr(offsets),
                                 float(beta), _ptr(C), int(ldc), int(type), int(ctype),
                                 _stream(stream)), "gemm_w4")


def swiglu_w4(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, Y, ldy, type, stream=None):
    """Y = SiLU(alpha A W1_g^T) (.) (alpha A W2_g^T), weights of 4 bits (see the C header)."""
    return _check(load().swiglu_w4(int(G), int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                                   _ptr(Q), _ptr(S), _ptr(Z), int(lds), int(group), _ptr(offsets),
                                   _ptr(Y), int(ldy), int(type), _stream(stream)), "swiglu_w4")


def status_string(status: int) -> str:
    return load().swg_status_string(int(status)).decode()


def get_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    return load().swg_get_device_error(_stream(stream))


def selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Runs a kernel whose bounded wait is made to run out (see the C header)."""
    return _check(load().swg_selftest_wait_timeout(int(limit_ns), _stream(stream)),
                  "swg_selftest_wait_timeout")


def debug_workspace_guards(stream=None) -> int:
    """Changed guard bytes around the current device's split-K workspaces
    (only those created under SWG_TEST_WS_GUARD=1; see the C header)."""
    bad = ctypes.c_int64(0)
    _check(load().swg_debug_workspace_guards(_stream(stream), ctypes.byref(bad)),
           "swg_debug_workspace_guards")
    return int(bad.value)


def launch_count() -> int:
    return int(load().swg_launch_count())


def shutdown() -> None:
    load().swg_shutdown()


# ---------------------------------------------------------------- tensor helpers

_dtype_table = None


def _dtype_code(in_dtype, out_dtype) -> int:
    global _dtype_table
    if _dtype_table is None:
        import torch
        _dtype_table = {
            (torch.float16, torch.float32): F16_F32OUT, (torch.bfloat16, torch.bfloat16): BF16,
            (torch.float16, torch.float16): F16, (torch.bfloat16, torch.float32): BF16_F32OUT}
    try:
        return _dtype_table[(in_dtype, out_dtype)]
    except KeyError:
        raise SwgError(3, f"gemm_into: unsupported dtypes {in_dtype} -> {out_dtype}") from None


def _row_major_ld(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise SwgError(1, f"{name} must be a 2-D row-major tensor (unit column stride)")
    return t.stride(0)


def gemm_into(C, A, B, transA=0, transB=0, alpha=1.0, beta=0.0, split_k=None, stream=None):
    """C <- alpha * op(A) op(B) + beta * C for 2-D row-major tensors."""
    M = A.shape[1] if transA else A.shape[0]
    K = A.shape[0] if transA else A.shape[1]
    N = B.shape[0] if transB else B.shape[1]
    Kb = B.shape[1] if transB else B.shape[0]
    if Kb != K or tuple(C.shape) != (M, N) or A.dtype != B.dtype:
        raise SwgError(1, "gemm_into: inconsistent shapes or dtypes")
    code = _dtype_code(A.dtype, C.dtype)
    args = (transA, transB, M, N, K, alpha, A, _row_major_ld(A, "A"), B, _row_major_ld(B, "B"),
            beta, C, _row_major_ld(C, "C"), code)
    if split_k is None:
        gemm(*args, stream=stream)
    else:
        gemm_ex(*args, split_k, stream=stream)
    return C


def swiglu_mlp_into(Y, A, W_fused, stream=None):
    """Y <- SiLU(A W1) (.) (A W2) with W_fused the interleaved [K, 2N] weight."""
    M, K = A.shape
    N = W_fused.shape[1] // 2
    if W_fused.shape[0] != K or tuple(Y.shape) != (M, N):
        raise SwgError(1, "swiglu_mlp_into: inconsistent shapes")
    for t, n in ((A, "A"), (W_fused, "W_fused"), (Y, "Y")):
        if not t.is_contiguous():
            raise SwgError(1, f"swiglu_mlp_into: {n} must be contiguous")
    swiglu_mlp(A, W_fused, Y, M, N, K, stream=stream)
    return Y


def interleave_weights(W1, W2, stream=None):
    """W_fused[K, 2N] with even columns W1 (Gate) and odd columns W2 (Up)."""
    import torch
    K, N = W1.shape
    if tuple(W2.shape) != (K, N) or not (W1.is_contiguous() and W2.is_contiguous()):
        raise SwgError(1, "interleave_weights: W1, W2 must be contiguous and the same shape")
    Wf = torch.empty((K, 2 * N), dtype=W1.dtype, device=W1.device)
    swiglu_interleave(W1, W2, Wf, K, N, stream=stream)
    return Wf


# ------------------------------------------------- tensor helpers, expert MLP
#
# These run once per call of operators that take a few microseconds on the
# GPU, so each tensor's shape and strides are fetched once and the refusals'
# messages are only built when one is raised.

_torch = None
_bound = None         # the CPython module of the C functions these helpers call


def _fast():
    """torch, loaded with the library and its binding on the first call."""
    global _torch, _bound
    load()
    import importlib

    import torch
    _bound = importlib.import_module("._binding", __name__)
    _torch = torch
    return torch


def _refuse(where, why, status=1):
    raise SwgError(status, f"{where}: {why}")


def _place(stream):
    """The handle of the call's stream, and the device that its tensors have to
    be on: the current one (-2, that of no tensor, without CUDA)."""
    if _device is None:
        _current_stream()
    dev = _device() if _device is not None else -2
    return (_raw_stream(dev) if stream is None and dev >= 0 else _stream(stream)), dev


def _failed(rc, where, name):
    if rc < 0:            # the binding's: nothing was called
        _refuse(where, "every tensor must be on the current CUDA device")
    _check(rc, name)


def _groups(offsets, where):
    """G of an int32 offsets tensor, or of none."""
    if offsets is None:
        return 1
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 1 or offsets.dtype is not _torch.int32 \
            or not offsets.is_contiguous():
        _refuse(where, "offsets must be a contiguous 1-D int32 tensor of G + 1 values")
    return shape[0] - 1


def _one_row(cols):
    """The row stride of a matrix of one row, which torch leaves open (it may be
    less than a row): one that every rule of alignment allows."""
    return (cols + 15) & ~15


def _matrices(t, name, where, G):
    """(rows, columns, row stride, group stride) of a [G, rows, columns]
    tensor, or with G = 1 also of a [rows, columns] one."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        g, rows, cols = shape
        sg, sr, sc = stride
    elif len(shape) == 2:
        (rows, cols), (sr, sc), g, sg = shape, stride, 1, 0
    else:
        g = sg = sr = sc = rows = cols = -1
    if sc != 1 or g != G:
        _refuse(where, f"{name} must hold one row-major matrix for each of {G} groups")
    return rows, cols, sr if rows > 1 else _one_row(cols), sg


def _matrix(t, name, where):
    """(rows, columns, row stride) of a 2-D row-major tensor."""
    try:
        (rows, cols), (ld, unit) = t.shape, t.stride()
    except ValueError:
        unit = 0
    if unit != 1:
        _refuse(where, f"{name} must be a 2-D row-major tensor (unit column stride)")
    return rows, cols, ld if rows > 1 else _one_row(cols)


def _type_code(dtype, where) -> int:
    if dtype is _torch.bfloat16:
        return TYPE_BF16
    if dtype is _torch.float16:
        return TYPE_F16
    if dtype is _torch.float32:
        return TYPE_F32
    _refuse(where, f"unsupported dtype {dtype}", 3)


def _output(w, name, t, rows, cols, dtype):
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 2 or shape[0] != rows or shape[1] != cols \
            or not t.is_contiguous():
        _refuse(w, f"{name} must be a contiguous [{rows}, {cols}] {dtype} tensor")


def gemm_grouped_into(C, A, B, offsets, transB=0, alpha=1.0, beta=0.0, stream=None):
    """C[M, N] <- alpha * A[M, K] op(B_g) + beta * C for the rows of each group;
    B is [G, K, N] (transB = 0) or [G, N, K], offsets int32 [G + 1] on the GPU."""
    w = "gemm_grouped_into"
    _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    rows, cols, ldb, stride = _matrices(B, "B", w, G)
    N, Kb = (rows, cols) if transB else (cols, rows)
    M, K, lda = _matrix(A, "A", w)
    Mc, Nc, ldc = _matrix(C, "C", w)
    if Kb != K or Mc != M or Nc != N or A.dtype is not B.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = lib.gemm_grouped(int(transB), G, M, N, K, alpha, A, lda, B, ldb, stride, offsets, beta, C,
                          ldc, _dtype_code(A.dtype, C.dtype), s, dev)
    if rc:
        _failed(rc, w, "gemm_grouped")
    return C


def gemm_grouped_wgrad_into(C, A, D, offsets, alpha=1.0, beta=0.0, stream=None):
    """C[G, K, N] <- alpha * A_g^T D_g + beta * C_g from A[M, K] and D[M, N]."""
    w = "gemm_grouped_wgrad_into"
    _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    rows, cols, ldc, stride = _matrices(C, "C", w, G)
    M, K, lda = _matrix(A, "A", w)
    Md, N, ldd = _matrix(D, "D", w)
    if Md != M or rows != K or cols != N or A.dtype is not D.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = lib.gemm_grouped_wgrad(G, M, N, K, alpha, A, lda, D, ldd, offsets, beta, C, ldc, stride,
                                _dtype_code(A.dtype, C.dtype), s, dev)
    if rc:
        _failed(rc, w, "gemm_grouped_wgrad")
    return C


def _swiglu_shapes(w, A, W_fused, G, bf16):
    rows, cols, _, _ = _matrices(W_fused, "W_fused", w, G)
    M, K, _ = _matrix(A, "A", w)
    if rows != K or cols % 2 or A.dtype is not bf16 or W_fused.dtype is not bf16 \
            or not A.is_contiguous() or not W_fused.is_contiguous():
        _refuse(w, "A [M, K] and W_fused [G, K, 2N] must be contiguous bfloat16")
    return M, cols // 2, K


def swiglu_grouped_into(Y, A, W_fused, offsets, stream=None):
    """Y[M, N] <- SiLU(A W1_g) (.) (A W2_g), W_fused [G, K, 2N] interleaved."""
    w = "swiglu_grouped_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M, N, K = _swiglu_shapes(w, A, W_fused, G, torch.bfloat16)
    _output(w, "Y", Y, M, N, torch.bfloat16)
    s, dev = _place(stream)
    rc = lib.swiglu_grouped(A, W_fused, Y, offsets, G, M, N, K, s, dev)
    if rc:
        _failed(rc, w, "swiglu_grouped")
    return Y


def swiglu_grouped_grad_into(dH, A, W_fused, dY, offsets, Y=None, stream=None):
    """dH[M, 2N] <- the gradient of swiglu_grouped in the interleaved Gate and
    Up, from dY[M, N]; Y, when given, receives swiglu_grouped's result."""
    w = "swiglu_grouped_grad_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M, N, K = _swiglu_shapes(w, A, W_fused, G, torch.bfloat16)
    _output(w, "dH", dH, M, 2 * N, torch.bfloat16)
    _output(w, "dY", dY, M, N, torch.bfloat16)
    if Y is not None:
        _output(w, "Y", Y, M, N, torch.bfloat16)
    s, dev = _place(stream)
    rc = lib.swiglu_grouped_grad(A, W_fused, dY, Y, dH, offsets, G, M, N, K, s, dev)
    if rc:
        _failed(rc, w, "swiglu_grouped_grad")
    return dH


def mx4_alloc(M, K, format, groups=1, device="cuda"):
    """(Q, S) for mx4_quantize_into: codes [M, 16 * ceil(K / 32)] and scale tiles."""
    import torch
    return (torch.empty((M, -(-K // 32) * 16), dtype=torch.uint8, device=device),
            torch.empty(mx4_scale_bytes(format, groups, M, K), dtype=torch.uint8, device=device))


def _mx4_rows(w, Q, S, format, G, M, K, torch):
    """Row stride of the codes Q of an M x K matrix whose scale tiles are S."""
    rows, width, ldq = _matrix(Q, "Q", w)
    if rows != M or width < -(-K // 32) * 16 or Q.dtype is not torch.uint8:
        _refuse(w, "Q must be M uint8 rows of at least 16 * ceil(K / 32) bytes")
    block = 64 if format == NVFP4 else 128
    if S.dtype is not torch.uint8 or not S.is_contiguous() \
            or S.numel() < 512 * -(-K // block) * (M // 128 + G):
        _refuse(w, "S must be contiguous uint8 scale tiles of mx4_scale_bytes")
    return ldq


def mx4_quantize_into(Q, S, X, format, scale=1.0, offsets=None, stream=None):
    """Q, S <- X[M, K] * scale in 4 bits (Q uint8 rows of codes, S scale tiles)."""
    w = "mx4_quantize_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M, K, ldx = _matrix(X, "X", w)
    ldq = _mx4_rows(w, Q, S, format, G, M, K, torch)
    s, dev = _place(stream)
    rc = lib.mx4_quantize(format, G, M, K, X, ldx, _type_code(X.dtype, w), scale, offsets, Q, ldq,
                          S, s, dev)
    if rc:
        _failed(rc, w, "mx4_quantize")
    return Q, S


def mx4_dequantize_into(X, Q, S, format, scale=1.0, offsets=None, stream=None):
    """X[M, K] <- scale * the values of the 4-bit rows (Q, S)."""
    w = "mx4_dequantize_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M, K, ldx = _matrix(X, "X", w)
    ldq = _mx4_rows(w, Q, S, format, G, M, K, torch)
    s, dev = _place(stream)
    rc = lib.mx4_dequantize(format, G, M, K, Q, ldq, S, scale, offsets, X, ldx,
                            _type_code(X.dtype, w), s, dev)
    if rc:
        _failed(rc, w, "mx4_dequantize")
    return X


def _mx4_weights(w, W, SW, format, G, K, torch):
    """(N, row stride, group stride) of weights W with scale tiles SW."""
    N, width, ldb, stride = _matrices(W, "W", w, G)
    if width < -(-K // 32) * 16 or W.dtype is not torch.uint8:
        _refuse(w, "W must hold uint8 rows of at least 16 * ceil(K / 32) bytes")
    block = 64 if format == NVFP4 else 128
    if SW.dtype is not torch.uint8 or not SW.is_contiguous() \
            or SW.numel() < 512 * -(-K // block) * -(-N // 128) * G:
        _refuse(w, "SW must be the weights' contiguous uint8 scale tiles")
    return N, ldb, stride


def gemm_mx4_into(C, Q, S, W, SW, K, format, alpha=1.0, beta=0.0, offsets=None, stream=None):
    """C[M, N] <- alpha * A W_g^T + beta * C with 4-bit A = (Q, S) of K columns
    and weights (W [N, bytes] or [G, N, bytes], SW)."""
    w = "gemm_mx4_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M, Nc, ldc = _matrix(C, "C", w)
    lda = _mx4_rows(w, Q, S, format, G, M, K, torch)
    N, ldb, stride = _mx4_weights(w, W, SW, format, G, K, torch)
    if Nc != N:
        _refuse(w, "inconsistent shapes")
    s, dev = _place(stream)
    rc = lib.gemm_mx4(format, G, M, N, K, alpha, Q, lda, S, W, ldb, stride, SW, offsets, beta, C,
                      ldc, _type_code(C.dtype, w), s, dev)
    if rc:
        _failed(rc, w, "gemm_mx4")
    return C


def swiglu_mx4_into(Y, Q, S, W, SW, K, format, alpha=1.0, offsets=None, stream=None):
    """Y[M, N] <- SiLU(alpha A W1_g^T) (.) (alpha A W2_g^T), W [2N, bytes] or
    [G, 2N, bytes] with Gate in even and Up in odd rows."""
    w = "swiglu_mx4_into"
    torch = _torch or _fast()
    lib = _bound
    G = _groups(offsets, w)
    M = Q.shape[0]
    lda = _mx4_rows(w, Q, S, format, G, M, K, torch)
    N2, ldb, stride = _mx4_weights(w, W, SW, format, G, K, torch)
    row = -(-K // 32) * 16
    if N2 % 2 or K > 0 and ((lda != row and M > 1) or ldb != row or (stride != N2 * row and G > 1)):
        _refuse(w, "Q and W must be contiguous rows of 16 * ceil(K / 32) bytes, W of 2N of them")
    _output(w, "Y", Y, M, N2 // 2, torch.bfloat16)
    s, dev = _place(stream)
    rc = lib.swiglu_mx4(format, Q, S, W, SW, Y, offsets, G, M, N2 // 2, K, alpha, s, dev)
    if rc:
        _failed(rc, w, "swiglu_mx4")
    return Y


# ------------------------------------------------------ tensor helpers, routing

def expert_plan_alloc(T, E, top, device="cuda"):
    """(offsets, source, position) for expert_route_into and expert_sort_into."""
    import torch
    return tuple(torch.empty(n, dtype=torch.int32, device=device) for n in (E + 1, T * top, (T, top)))


def _slots(w, name, t, T, top, dtype):
    """A contiguous [T, top] tensor of slots."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 2 or shape[0] != T or shape[1] != top \
            or not t.is_contiguous():
        _refuse(w, f"{name} must be a contiguous [{T}, {top}] {dtype} tensor")


def _plan(w, plan, T, E, top, int32):
    offsets, source, position = plan
    if offsets.dtype is not int32 or len(offsets.shape) != 1 or not offsets.is_contiguous() \
            or (offsets.shape[0] != E + 1 if E is not None else offsets.shape[0] < 2):
        _refuse(w, "offsets must be a contiguous 1-D int32 tensor of E + 1 values")
    if source.dtype is not int32 or len(source.shape) != 1 or source.shape[0] != T * top \
            or not source.is_contiguous():
        _refuse(w, f"source must be a contiguous [{T * top}] int32 tensor")
    _slots(w, "position", position, T, top, int32)
    return offsets, source, position


def _pair(w, name, t):
    """(T, top) of a tensor of slots."""
    shape = t.shape
    if len(shape) != 2:
        _refuse(w, f"{name} must be a [T, top] tensor")
    return shape[0], shape[1]


def expert_route_into(experts, weights, logits, score=SOFTMAX, bias=None, groups=1, top_groups=None,
                      group_sum=1, normalise=True, scale=1.0, plan=None, stream=None):
    """experts int32 [T, top], weights float32 [T, top] <- the router's choice for
    logits [T, E], best first (-1 and 0 where a slot has no expert); plan, when
    given (expert_plan_alloc), receives the rows sorted by expert.  top_groups:
    all of them by default."""
    w = "expert_route_into"
    torch = _torch or _fast()
    lib = _bound
    T, E, ld = _matrix(logits, "logits", w)
    Te, top = _pair(w, "experts", experts)
    _slots(w, "experts", experts, T, top, torch.int32)
    _slots(w, "weights", weights, T, top, torch.float32)
    if bias is not None and (bias.dtype is not torch.float32 or bias.dim() != 1 or bias.shape[0] != E
                             or not bias.is_contiguous()):
        _refuse(w, f"bias must be a contiguous [{E}] float32 tensor")
    offsets = source = position = None
    if plan is not None:
        offsets, source, position = _plan(w, plan, T, E, top, torch.int32)
    s, dev = _place(stream)
    rc = lib.expert_route(score, T, E, top, logits, ld, _type_code(logits.dtype, w), bias, groups,
                          groups if top_groups is None else top_groups, group_sum, bool(normalise),
                          scale, experts, weights, offsets, source, position, s, dev)
    if rc:
        _failed(rc, w, "expert_route")
    return experts, weights


def expert_sort_into(plan, experts, stream=None):
    """plan (expert_plan_alloc) <- rows sorted by expert, for experts int32 [T, top]."""
    w = "expert_sort_into"
    torch = _torch or _fast()
    lib = _bound
    T, top = _pair(w, "experts", experts)
    _slots(w, "experts", experts, T, top, torch.int32)
    offsets, source, position = _plan(w, plan, T, None, top, torch.int32)
    s, dev = _place(stream)
    rc = lib.expert_sort(T, offsets.shape[0] - 1, top, experts, offsets, source, position, s, dev)
    if rc:
        _failed(rc, w, "expert_sort")
    return plan


def expert_route_grad_into(d_logits, d_weights, logits, experts, score=SOFTMAX, normalise=True,
                           scale=1.0, stream=None):
    """d_logits [T, E] <- the gradient of expert_route_into's weights in the logits,
    from d_weights float32 [T, top]."""
    w = "expert_route_grad_into"
    torch = _torch or _fast()
    lib = _bound
    T, E, ld = _matrix(logits, "logits", w)
    Td, Ed, ldd = _matrix(d_logits, "d_logits", w)
    Te, top = _pair(w, "experts", experts)
    _slots(w, "experts", experts, T, top, torch.int32)
    _slots(w, "d_weights", d_weights, T, top, torch.float32)
    if Td != T or Ed != E or d_logits.dtype is not logits.dtype:
        _refuse(w, "d_logits must have the shape and type of logits")
    s, dev = _place(stream)
    rc = lib.expert_route_grad(score, T, E, top, logits, ld, _type_code(logits.dtype, w), experts,
                               bool(normalise), scale, d_weights, d_logits, ldd, s, dev)
    if rc:
        _failed(rc, w, "expert_route_grad")
    return d_logits


def _weights_of(w, weights, T, top, float32):
    if weights is not None:
        _slots(w, "weights", weights, T, top, float32)


def expert_dispatch_into(rows, X, position, stream=None):
    """rows[position[t, j]] <- X[t] for every slot with a row (position int32
    [T, top], -1 where a slot has none); other rows keep their values."""
    w = "expert_dispatch_into"
    torch = _torch or _fast()
    lib = _bound
    T, D, ldx = _matrix(X, "X", w)
    R, Dr, ldr = _matrix(rows, "rows", w)
    Tp, top = _pair(w, "position", position)
    _slots(w, "position", position, T, top, torch.int32)
    if Dr != D or rows.dtype is not X.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = lib.expert_dispatch(T, R, D, top, X, ldx, _type_code(X.dtype, w), position, rows, ldr, s, dev)
    if rc:
        _failed(rc, w, "expert_dispatch")
    return rows


def expert_combine_into(out, rows, position, weights=None, beta=0.0, stream=None):
    """out[t] <- sum_j weights[t, j] * rows[position[t, j]] + beta * out[t] (weights
    float32 [T, top]; None: ones).  out is of the rows' type; of float32 rows also
    16-bit."""
    w = "expert_combine_into"
    torch = _torch or _fast()
    lib = _bound
    T, D, ldo = _matrix(out, "out", w)
    R, Dr, ldr = _matrix(rows, "rows", w)
    Tp, top = _pair(w, "position", position)
    _slots(w, "position", position, T, top, torch.int32)
    _weights_of(w, weights, T, top, torch.float32)
    if Dr != D or (rows.dtype is not out.dtype and rows.dtype is not torch.float32):
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = lib.expert_combine(T, R, D, top, rows, ldr, _type_code(rows.dtype, w), position, weights,
                            beta, out, ldo, _type_code(out.dtype, w), s, dev)
    if rc:
        _failed(rc, w, "expert_combine")
    return out


def expert_combine_grad_into(d_rows, d_weights, d_out, rows, position, weights=None, stream=None):
    """d_rows[position[t, j]] <- weights[t, j] * d_out[t] and d_weights[t, j] <-
    <rows[position[t, j]], d_out[t]> (d_weights None: not computed, and rows may be
    None).  All of the rows' type: of float32 rows summed into 16 bits d_out is float32."""
    w = "expert_combine_grad_into"
    torch = _torch or _fast()
    lib = _bound
    T, D, ldd = _matrix(d_out, "d_out", w)
    R, Dr, lddr = _matrix(d_rows, "d_rows", w)
    Tp, top = _pair(w, "position", position)
    _slots(w, "position", position, T, top, torch.int32)
    _weights_of(w, weights, T, top, torch.float32)
    ldr = 0
    if d_weights is not None:
        _slots(w, "d_weights", d_weights, T, top, torch.float32)
        Rr, Dx, ldr = _matrix(rows, "rows", w)
        if Rr != R or Dx != D or rows.dtype is not d_out.dtype:
            _refuse(w, "inconsistent shapes or dtypes")
    else:
        rows = None
    if Dr != D or d_rows.dtype is not d_out.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = lib.expert_combine_grad(T, R, D, top, d_out, ldd, rows, ldr, _type_code(d_out.dtype, w),
                                 position, weights, d_rows, lddr, d_weights, s, dev)
    if rc:
        _failed(rc, w, "expert_combine_grad")
    return d_rows, d_weights


# ------------------------- tensor helpers, 4-bit weights with group scales

def w4_alloc(N, K, group, dtype, zeros=False, experts=None, device="cuda"):
    """(Q, S, Z) of a weight [N, K], or of [experts, N, K]: codes, scales of dtype
    (float16 or bfloat16) and zero points (None without `zeros`)."""
    import torch
    lead = () if experts is None else (experts,)
    shape = lead + (-(-K // group), -(-N // 16) * 16)
    return (torch.empty(lead + (N, -(-K // 32) * 16), dtype=torch.uint8, device=device),
            torch.empty(shape, dtype=dtype, device=device),
            torch.empty(shape, dtype=torch.uint8, device=device) if zeros else None)


def _w4_weight(w, Q, S, Z, group, G, K, torch):
    """(rows of each weight, the scales' row length)."""
    shape = Q.shape
    if len(shape) == 2:
        shape = (1, *shape)
    if len(shape) != 3 or shape[0] != G or shape[2] != -(-K // 32) * 16 or Q.dtype is not torch.uint8 \
            or not Q.is_contiguous():
        _refuse(w, f"Q must be contiguous uint8 [{G}, N, {-(-K // 32) * 16}]")
    if group not in (32, 64, 128):
        _refuse(w, "scales are kept for 32, 64 or 128 columns", 3)
    blocks = -(-K // group)
    for name, t, dtype in (("S", S, None), ("Z", Z, torch.uint8)):
        if t is None and dtype is not None:
            continue
        of = t.shape
        if len(of) == 2:
            of = (1, *of)
        if len(of) != 3 or of[0] != G or of[1] != blocks or of[2] < shape[1] or of[2] % 16 \
                or of[2] != S.shape[-1] or not t.is_contiguous() \
                or (t.dtype is not dtype if dtype else t.dtype not in (torch.float16, torch.bfloat16)):
            _refuse(w, f"{name} must be contiguous [{G}, {blocks}, at least N, a multiple of 16], S of "
                       "float16 or bfloat16, Z of uint8")
    return shape[1], S.shape[-1]


def _w4_matrix(w, X):
    """(G, rows, columns, row stride) of [rows, columns] or [G, rows, columns], whose
    rows follow one another at one stride."""
    shape, stride = X.shape, X.stride()
    if len(shape) == 2:
        rows, cols, ld = _matrix(X, "W", w)
        return 1, rows, cols, ld
    if len(shape) != 3 or stride[2] != 1:
        _refuse(w, "W must hold row-major matrices")
    G, rows, cols = shape
    ld = stride[1] if rows > 1 else stride[0] if G > 1 else _one_row(cols)
    if G > 1 and rows > 1 and stride[0] != rows * ld:
        _refuse(w, "the matrices of W must follow one another")
    return G, rows, cols, ld


def _w4_convert(w, W, Q, S, Z, group):
    torch = _torch or _fast()
    G, N, K, ld = _w4_matrix(w, W)
    rows, lds = _w4_weight(w, Q, S, Z, group, G, K, torch)
    if rows != N:
        _refuse(w, "inconsistent shapes")
    return G, N, K, ld, _type_code(W.dtype, w), lds, _type_code(S.dtype, w)


def w4_quantize_into(Q, S, Z, W, group, stream=None):
    """Q, S, Z (w4_alloc; Z None: symmetric) <- W [N, K] or [G, N, K] in 4 bits."""
    w = "w4_quantize_into"
    G, N, K, ld, xtype, lds, stype = _w4_convert(w, W, Q, S, Z, group)
    s, dev = _place(stream)
    rc = _bound.w4_quantize(G, N, K, W, ld, xtype, group, Q, S, Z, lds, stype, s, dev)
    if rc:
        _failed(rc, w, "w4_quantize")
    return Q, S, Z


def w4_dequantize_into(W, Q, S, Z, group, stream=None):
    """W [N, K] or [G, N, K] <- the values of the 4-bit weight (Q, S, Z)."""
    w = "w4_dequantize_into"
    G, N, K, ld, xtype, lds, stype = _w4_convert(w, W, Q, S, Z, group)
    s, dev = _place(stream)
    rc = _bound.w4_dequantize(G, N, K, Q, S, Z, lds, stype, group, W, ld, xtype, s, dev)
    if rc:
        _failed(rc, w, "w4_dequantize")
    return W


def gemm_w4_into(C, A, Q, S, Z, group, alpha=1.0, beta=0.0, offsets=None, stream=None):
    """C[M, N] <- alpha * A[M, K] W_g^T + beta * C with a 4-bit weight (Q, S, Z) of
    A's type, [N, K] or [G, N, K]; offsets int32 [G + 1] on the GPU, or None."""
    w = "gemm_w4_into"
    torch = _torch or _fast()
    G = _groups(offsets, w)
    M, K, lda = _matrix(A, "A", w)
    Mc, Nc, ldc = _matrix(C, "C", w)
    N, lds = _w4_weight(w, Q, S, Z, group, G, K, torch)
    if Mc != M or Nc != N or S.dtype is not A.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = _bound.gemm_w4(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, beta, C, ldc,
                        _type_code(A.dtype, w), _type_code(C.dtype, w), s, dev)
    if rc:
        _failed(rc, w, "gemm_w4")
    return C


def swiglu_w4_into(Y, A, Q, S, Z, group, alpha=1.0, offsets=None, stream=None):
    """Y[M, N] <- SiLU(alpha A W1_g^T) (.) (alpha A W2_g^T), the weight's 2N rows W1's
    and W2's in turn; Y and A of one type."""
    w = "swiglu_w4_into"
    torch = _torch or _fast()
    G = _groups(offsets, w)
    M, K, lda = _matrix(A, "A", w)
    My, N, ldy = _matrix(Y, "Y", w)
    rows, lds = _w4_weight(w, Q, S, Z, group, G, K, torch)
    if My != M or rows != 2 * N or S.dtype is not A.dtype or Y.dtype is not A.dtype:
        _refuse(w, "inconsistent shapes or dtypes")
    s, dev = _place(stream)
    rc = _bound.swiglu_w4(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, Y, ldy,
                          _type_code(A.dtype, w), s, dev)
    if rc:
        _failed(rc, w, "swiglu_w4")
    return Y
