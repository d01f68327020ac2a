"""Refusals of the expert-MLP entry points: every bad argument is answered
before any CUDA call, so these run without a GPU."""
import os
import subprocess

import pytest
import torch

import swiglu_mlp_gb300 as swg
from swiglu_mlp_gb300 import build as swg_build
from test_abi_host import INVALID, MISALIGNED, OK, P, UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    swg_build.build()
    return swg.load()


def call(fn, names, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*(a[n] for n in names.split()), None)


def test_gemm_grouped(lib):
    d = dict(t=0, G=4, M=128, N=64, K=72, alpha=1.0, A=P, lda=72, B=P, ldb=64, sB=72 * 64, off=P, beta=0.0,
             C=P, ldc=64, dt=1)

    def f(**kw):
        return call(lib.gemm_grouped, "t G M N K alpha A lda B ldb sB off beta C ldc dt", d, **kw)

    assert f(t=2) == INVALID and f(G=-1) == INVALID and f(M=-1) == INVALID and f(N=-1) == INVALID
    assert f(K=-1) == INVALID and f(A=None) == INVALID and f(B=None) == INVALID and f(C=None) == INVALID
    assert f(off=None) == INVALID                       # more than one group needs offsets
    assert f(lda=64) == INVALID and f(ldb=56) == INVALID and f(ldc=56) == INVALID
    assert f(t=1, ldb=64) == INVALID                    # op T: ldb >= K
    assert f(sB=64 * 8) == INVALID                      # groups would overlap
    assert f(dt=4) == UNSUPPORTED and f(dt=9) == UNSUPPORTED and f(G=1025) == UNSUPPORTED
    assert f(M=2 ** 31) == UNSUPPORTED
    assert f(A=P + 8) == MISALIGNED and f(lda=76) == MISALIGNED and f(ldb=68, sB=72 * 72) == MISALIGNED
    assert f(sB=72 * 64 + 4) == MISALIGNED and f(C=P + 2) == MISALIGNED and f(ldc=68) == MISALIGNED
    assert f(off=P + 2) == MISALIGNED
    assert f(M=0) == OK and f(N=0) == OK and f(G=0) == OK


def test_gemm_grouped_wgrad(lib):
    d = dict(G=4, M=128, N=64, K=72, alpha=1.0, A=P, lda=72, D=P, ldd=64, off=P, beta=0.0, C=P, ldc=64,
             sC=72 * 64, dt=1)

    def f(**kw):
        return call(lib.gemm_grouped_wgrad, "G M N K alpha A lda D ldd off beta C ldc sC dt", d, **kw)

    assert f(G=-1) == INVALID and f(M=-1) == INVALID and f(A=None) == INVALID and f(D=None) == INVALID
    assert f(C=None) == INVALID and f(off=None) == INVALID and f(lda=64) == INVALID and f(ldd=56) == INVALID
    assert f(ldc=56) == INVALID and f(sC=64) == INVALID
    assert f(dt=5) == UNSUPPORTED and f(G=1025) == UNSUPPORTED
    assert f(A=P + 4) == MISALIGNED and f(ldd=68) == MISALIGNED and f(sC=72 * 64 + 2) == MISALIGNED
    assert f(N=0) == OK and f(K=0) == OK and f(G=0) == OK


def test_swiglu_grouped(lib):
    d = dict(A=P, W=P, Y=P, off=P, G=4, M=128, N=64, K=72)

    def f(**kw):
        return call(lib.swiglu_grouped, "A W Y off G M N K", d, **kw)

    def h(**kw):
        return call(lib.swiglu_grouped_grad, "A W dY Y dH off G M N K", dict(d, dY=P, dH=P), **kw)

    for c in (f, h):
        assert c(M=-1) == INVALID and c(A=None) == INVALID and c(W=None) == INVALID and c(off=None) == INVALID
        assert c(N=60) == MISALIGNED and c(K=68) == MISALIGNED and c(A=P + 8) == MISALIGNED
        assert c(G=1025) == UNSUPPORTED and c(N=2 ** 30) == UNSUPPORTED
        assert c(M=0) == OK and c(N=0) == OK and c(G=0) == OK
    assert f(Y=None) == INVALID and h(dY=None) == INVALID and h(dH=None) == INVALID
    assert h(dY=P + 2) == MISALIGNED and h(Y=P + 2) == MISALIGNED


def test_mx4(lib):
    d = dict(fmt=0, G=4, M=128, N=64, K=72, X=P, ldx=72, type=1, scale=1.0, off=P, Q=P, ldq=48, S=P)

    def f(**kw):
        return call(lib.mx4_quantize, "fmt G M K X ldx type scale off Q ldq S", d, **kw)

    def b(**kw):
        return call(lib.mx4_dequantize, "fmt G M K Q ldq S scale off X ldx type", d, **kw)

    for c in (f, b):
        assert c(fmt=2) == UNSUPPORTED and c(type=3) == UNSUPPORTED and c(G=1025) == UNSUPPORTED
        assert c(M=-1) == INVALID and c(K=-1) == INVALID and c(X=None) == INVALID and c(Q=None) == INVALID
        assert c(S=None) == INVALID and c(off=None) == INVALID and c(ldx=64) == INVALID and c(ldq=32) == INVALID
        assert c(scale=0.0) == INVALID and c(scale=float("inf")) == INVALID and c(scale=float("nan")) == INVALID
        assert c(X=P + 2) == MISALIGNED and c(ldx=76) == MISALIGNED and c(ldq=56) == MISALIGNED
        assert c(S=P + 8) == MISALIGNED
        assert c(M=0) == OK and c(K=0) == OK and c(G=0) == OK
    assert lib.mx4_scale_bytes(0, 1, 300, 1000) == 512 * 8 * 3
    assert lib.mx4_scale_bytes(1, 5, 300, 1000) == 512 * 16 * 7
    assert lib.mx4_scale_bytes(2, 1, 1, 1) == -1 and lib.mx4_scale_bytes(0, -1, 1, 1) == -1


def test_gemm_mx4(lib):
    d = dict(fmt=1, G=4, M=128, N=64, K=72, alpha=1.0, A=P, lda=48, SA=P, B=P, ldb=48, sB=64 * 48, SB=P, off=P,
             beta=0.0, C=P, ldc=64, type=1)

    def f(**kw):
        return call(lib.gemm_mx4, "fmt G M N K alpha A lda SA B ldb sB SB off beta C ldc type", d, **kw)

    assert f(fmt=7) == UNSUPPORTED and f(type=9) == UNSUPPORTED and f(G=1025) == UNSUPPORTED
    assert f(M=-1) == INVALID and f(off=None) == INVALID and f(lda=32) == INVALID and f(ldb=32) == INVALID
    assert f(sB=48) == INVALID and f(ldc=56) == INVALID
    for name in ("A", "SA", "B", "SB", "C"):
        assert f(**{name: None}) == INVALID
        assert f(**{name: P + 8}) == MISALIGNED
    assert f(lda=56) == MISALIGNED and f(sB=64 * 48 + 8) == MISALIGNED and f(ldc=68) == MISALIGNED
    assert f(M=0) == OK and f(N=0) == OK and f(G=0) == OK

    d = dict(fmt=0, A=P, SA=P, W=P, SW=P, Y=P, off=P, G=4, M=128, N=64, K=72, alpha=1.0)

    def h(**kw):
        return call(lib.swiglu_mx4, "fmt A SA W SW Y off G M N K alpha", d, **kw)

    assert h(fmt=7) == UNSUPPORTED and h(N=2 ** 30) == UNSUPPORTED
    assert h(N=-8) == INVALID and h(off=None) == INVALID
    for name in ("A", "SA", "W", "SW", "Y"):
        assert h(**{name: None}) == INVALID
        assert h(**{name: P + 8}) == MISALIGNED
    assert h(N=60) == MISALIGNED
    assert h(M=0) == OK and h(N=0) == OK and h(G=0) == OK


def test_tensor_helpers_refuse():
    """The *_into helpers check shapes, types and strides of their tensors."""
    t = torch.zeros
    off = t(3, dtype=torch.int32)
    A, B, C = t(8, 16).half(), t(2, 16, 24).half(), t(8, 24).half()
    bad = [
        lambda: swg.gemm_grouped_into(C, A, B, off.long()),
        lambda: swg.gemm_grouped_into(C, A, B, t(4, dtype=torch.int32)),
        lambda: swg.gemm_grouped_into(C, A, B.transpose(1, 2), off),
        lambda: swg.gemm_grouped_into(C, A, B.float(), off),
        lambda: swg.gemm_grouped_into(t(7, 24).half(), A, B, off),
        lambda: swg.gemm_grouped_wgrad_into(B, A, t(7, 24).half(), off),
        lambda: swg.gemm_grouped_wgrad_into(B[0], A, C, off),
        lambda: swg.swiglu_grouped_into(t(8, 12).half(), A, B, off),
        lambda: swg.swiglu_grouped_grad_into(t(8, 24).bfloat16(), A.bfloat16(), B.bfloat16(), t(8, 11).bfloat16(), off),
        lambda: swg.mx4_quantize_into(t(8, 16), t(4096, dtype=torch.uint8), A, swg.MXFP4),
        lambda: swg.mx4_quantize_into(t(8, 8, dtype=torch.uint8), t(4096, dtype=torch.uint8), A, swg.MXFP4),
        lambda: swg.mx4_quantize_into(t(8, 16, dtype=torch.uint8), t(100, dtype=torch.uint8), A, swg.MXFP4),
        lambda: swg.mx4_quantize_into(t(8, 16, dtype=torch.uint8), t(4096, dtype=torch.uint8), A.double(), swg.MXFP4),
        lambda: swg.gemm_mx4_into(C, t(8, 16, dtype=torch.uint8), t(512, dtype=torch.uint8),
                                  t(24, 16, dtype=torch.uint8), t(100, dtype=torch.uint8), 16, swg.MXFP4),
        lambda: swg.swiglu_mx4_into(C.bfloat16(), t(8, 16, dtype=torch.uint8), t(512, dtype=torch.uint8),
                                    t(24, 16, dtype=torch.uint8), t(512, dtype=torch.uint8), 16, swg.MXFP4),
    ]
    for f in bad:
        with pytest.raises(swg.SwgError):
            f()


def test_sizes_that_round_up_past_32_bits(lib):
    """Rows and columns are rounded up to whole tiles in 32 bits, so sizes end
    1023 before 2^31."""
    top = 2 ** 31 - 1023
    ld = 2 ** 31 - 8                                   # strides may be larger
    d = dict(t=0, G=1, M=128, N=64, K=72, alpha=1.0, A=P, lda=ld, B=P, ldb=ld, sB=0, off=P, beta=0.0, C=P,
             ldc=ld, dt=1, D=P, ldd=ld, sC=0, fmt=0, X=P, ldx=ld, type=1, scale=1.0, Q=P, ldq=2 ** 31 - 16, S=P,
             SA=P, SB=P, W=P, SW=P, Y=P, dY=P, dH=P)
    for f, names, sizes in (
            (lib.gemm_grouped, "t G M N K alpha A lda B ldb sB off beta C ldc dt", "MNK"),
            (lib.gemm_grouped_wgrad, "G M N K alpha A lda D ldd off beta C ldc sC dt", "MNK"),
            (lib.swiglu_grouped, "A W Y off G M N K", "MK"),
            (lib.swiglu_grouped_grad, "A W dY Y dH off G M N K", "MK"),
            (lib.mx4_quantize, "fmt G M K X ldx type scale off Q ldq S", "MK"),
            (lib.mx4_dequantize, "fmt G M K Q ldq S scale off X ldx type", "MK"),
            (lib.gemm_mx4, "fmt G M N K alpha A lda SA B ldb sB SB off beta C ldc type", "MNK"),
            (lib.swiglu_mx4, "fmt A SA W SW Y off G M N K alpha", "MK")):
        for name in sizes:
            assert call(f, names, d, **{name: top}) == UNSUPPORTED, (f, name)
    assert call(lib.swiglu_grouped, "A W Y off G M N K", d, N=(top + 7) // 2) == UNSUPPORTED


@pytest.mark.parametrize("extra", [8, 64])
def test_sizes_whose_products_pass_64_bits(lib, extra):
    """2N of a SwiGLU, or a group stride, may pass 2^63: refused all the same."""
    big = 2 ** 62 + extra
    d = dict(A=P, W=P, Y=P, dY=P, dH=P, SA=P, SW=P, off=P, G=2, M=128, N=big, K=72, fmt=0, alpha=1.0)
    assert call(lib.swiglu_grouped, "A W Y off G M N K", d) == UNSUPPORTED
    assert call(lib.swiglu_grouped_grad, "A W dY Y dH off G M N K", d) == UNSUPPORTED
    assert call(lib.swiglu_mx4, "fmt A SA W SW Y off G M N K alpha", d) == UNSUPPORTED
    d = dict(t=0, G=2, M=128, N=64, K=big, alpha=1.0, A=P, lda=big, B=P, ldb=64, sB=2 ** 62, off=P, beta=0.0,
             C=P, ldc=64, dt=1, D=P, ldd=64, sC=2 ** 62, fmt=0, SA=P, SB=P, type=1)
    assert call(lib.gemm_grouped, "t G M N K alpha A lda B ldb sB off beta C ldc dt", d) == UNSUPPORTED
    assert call(lib.gemm_grouped_wgrad, "G M N K alpha A lda D ldd off beta C ldc sC dt", d) == UNSUPPORTED
    assert call(lib.gemm_mx4, "fmt G M N K alpha A lda SA B ldb sB SB off beta C ldc type", d) == UNSUPPORTED


@pytest.mark.parametrize("extra", [8, 64])
def test_dense_swiglu_widths_that_pass_64_bits(lib, extra):
    big = 2 ** 62 + extra
    assert lib.swiglu_mlp(P, P, P, 128, big, 72, None) == UNSUPPORTED
    assert lib.swiglu_mlp_fp8(P, P, P, 128, big, 128, 1.0, None) == UNSUPPORTED
    assert lib.swiglu_mlp_dual(P, P, P, P, 128, big, 72, None) == UNSUPPORTED
    assert lib.swiglu_mlp_forward(P, P, P, P, P, 128, big, 72, 0.0, None) == UNSUPPORTED
    assert lib.swiglu_interleave(P, P, P, 72, big, None) == UNSUPPORTED


def expert_calls():
    """Each *_into helper with arguments that fit, as (function, tensors, the rest)."""
    off = torch.tensor([0, 3, 8], dtype=torch.int32)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    q, s = z(8, 16, t=torch.uint8), z(1024, t=torch.uint8)
    w, sw = z(2, 32, 16, t=torch.uint8), z(1024, t=torch.uint8)
    return [
        (swg.gemm_grouped_into, dict(C=z(8, 24), A=z(8, 16), B=z(2, 16, 24), offsets=off), {}),
        (swg.gemm_grouped_wgrad_into, dict(C=z(2, 16, 24), A=z(8, 16), D=z(8, 24), offsets=off), {}),
        (swg.swiglu_grouped_into, dict(Y=z(8, 16), A=z(8, 16), W_fused=z(2, 16, 32), offsets=off), {}),
        (swg.swiglu_grouped_grad_into, dict(dH=z(8, 32), A=z(8, 16), W_fused=z(2, 16, 32), dY=z(8, 16),
                                            offsets=off, Y=z(8, 16)), {}),
        (swg.mx4_quantize_into, dict(Q=q, S=s, X=z(8, 32), offsets=off), dict(format=swg.MXFP4)),
        (swg.mx4_dequantize_into, dict(Q=q, S=s, X=z(8, 32), offsets=off), dict(format=swg.MXFP4)),
        (swg.gemm_mx4_into, dict(C=z(8, 32), Q=q, S=s, W=w, SW=sw, offsets=off), dict(K=32, format=swg.MXFP4)),
        (swg.swiglu_mx4_into, dict(Y=z(8, 16), Q=q, S=s, W=w, SW=sw, offsets=off), dict(K=32, format=swg.MXFP4)),
    ]


@pytest.mark.parametrize("i", range(8))
def test_tensors_on_the_host_are_refused(i):
    f, tensors, rest = expert_calls()[i]
    with pytest.raises(swg.SwgError, match="current CUDA device") as e:
        f(**tensors, **rest)
    assert e.value.status == INVALID


def test_binding_keeps_to_the_stable_abi(lib):
    """Another interpreter than the one that built it may find it and load it."""
    import importlib
    module = importlib.import_module("swiglu_mlp_gb300._binding")
    assert os.path.samefile(module.__file__, swg_build.BINDING) and module.__file__.endswith(".abi3.so")
    needed = subprocess.run(["nm", "-D", "--undefined-only", module.__file__], capture_output=True, text=True).stdout
    names = [line.split()[-1].split("@")[0] for line in needed.splitlines()]
    assert any(n.startswith("Py") for n in names)
    # private names are in no stable ABI, but for these
    assert {n for n in names if n.startswith("_Py")} <= {"_Py_Dealloc", "_Py_IncRef", "_Py_DecRef", "_Py_NoneStruct"}


def test_build_without_python_headers(lib, monkeypatch, tmp_path):
    """The library is there and the error names the compiler that failed."""
    monkeypatch.setattr(swg_build, "BINDING", str(tmp_path / "_binding.abi3.so"))
    monkeypatch.setattr(swg_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.raises(RuntimeError, match="^gcc failed"):
        swg_build.build()
    assert os.path.exists(swg_build.LIB)
