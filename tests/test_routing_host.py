"""Refusals of the routing and 4-bit-weight entry points: every bad argument is
answered before any CUDA call, so these run without a GPU."""
import pytest
import torch

import swiglu_mlp_gb300 as swg
from swiglu_mlp_gb300 import build as swg_build
from test_abi_host import INVALID, MISALIGNED, OK, P, UNSUPPORTED
from test_experts_host import call


@pytest.fixture(scope="module")
def lib():
    swg_build.build()
    return swg.load()


def test_expert_route(lib):
    d = dict(score=0, T=128, E=64, top=4, l=P, ldl=64, type=1, bias=P, groups=8, tg=4, gs=2, norm=1, scale=1.0,
             ex=P, we=P, off=P, src=P, pos=P)

    def f(**kw):
        return call(lib.expert_route, "score T E top l ldl type bias groups tg gs norm scale ex we off src pos", d, **kw)

    assert f(type=3) == UNSUPPORTED and f(score=2) == UNSUPPORTED and f(score=-1) == UNSUPPORTED
    assert f(T=-1) == INVALID and f(top=0) == INVALID and f(E=0) == INVALID
    assert f(top=33) == UNSUPPORTED and f(T=2 ** 31) == UNSUPPORTED and f(T=2 ** 29, top=4) == UNSUPPORTED
    assert f(E=1025, groups=1, tg=1, ldl=1025) == UNSUPPORTED
    assert f(E=64, groups=64, tg=64) == UNSUPPORTED                     # more groups than there may be
    assert f(top=5, E=4, groups=1, tg=1) == INVALID
    assert f(groups=0) == INVALID and f(groups=7) == INVALID and f(tg=0) == INVALID and f(tg=9) == INVALID
    assert f(tg=1, top=9) == INVALID                                    # eight experts in a group
    assert f(gs=0) == INVALID and f(gs=3) == INVALID
    for bad in (float("inf"), float("nan")):
        assert f(scale=bad) == INVALID
    for name in ("l", "ex", "we", "off", "src", "pos"):
        assert f(**{name: None}) == INVALID
    for name in ("bias", "ex", "we", "off", "src", "pos"):
        assert f(**{name: P + 2}) == MISALIGNED
    assert f(l=P + 1) == MISALIGNED and f(type=2, l=P + 2) == MISALIGNED
    assert f(ldl=63) == INVALID and f(ldl=2 ** 31) == UNSUPPORTED
    assert f(T=0, off=None, src=None, pos=None, l=None, ex=None, we=None) == OK


def test_expert_sort(lib):
    d = dict(T=128, E=64, top=4, ex=P, off=P, src=P, pos=P)

    def f(**kw):
        return call(lib.expert_sort, "T E top ex off src pos", d, **kw)

    assert f(T=-1) == INVALID and f(E=0) == INVALID and f(top=0) == INVALID
    assert f(E=1025) == UNSUPPORTED and f(top=33) == UNSUPPORTED and f(T=2 ** 30) == UNSUPPORTED
    for name in ("ex", "off", "src", "pos"):
        assert f(**{name: None}) == INVALID and f(**{name: P + 2}) == MISALIGNED


def test_expert_route_grad(lib):
    d = dict(score=0, T=128, E=64, top=4, l=P, ldl=64, type=1, ex=P, norm=1, scale=1.0, dw=P, dl=P, ldd=64)

    def f(**kw):
        return call(lib.expert_route_grad, "score T E top l ldl type ex norm scale dw dl ldd", d, **kw)

    assert f(type=3) == UNSUPPORTED and f(score=2) == UNSUPPORTED and f(E=1025, ldl=1025, ldd=1025) == UNSUPPORTED
    assert f(T=-1) == INVALID and f(top=0) == INVALID and f(top=33) == UNSUPPORTED and f(E=3) == INVALID
    assert f(scale=float("nan")) == INVALID and f(ldl=63) == INVALID and f(ldd=63) == INVALID
    for name in ("l", "ex", "dw", "dl"):
        assert f(**{name: None}) == INVALID and f(**{name: P + 1}) == MISALIGNED
    assert f(T=0) == OK


def test_moving_rows(lib):
    d = dict(T=128, R=512, D=64, top=4, X=P, ldx=64, type=1, pos=P, rows=P, ldr=64, we=P, beta=0.0, out=P, ldo=64, otype=1,
             dr=P, lddr=64, dw=P)
    calls = [(lib.expert_dispatch, "T R D top X ldx type pos rows ldr", ("X", "rows"), ("ldx", "ldr")),
             (lib.expert_combine, "T R D top rows ldr type pos we beta out ldo otype", ("rows", "out"), ("ldr", "ldo")),
             (lib.expert_combine_grad, "T R D top X ldx rows ldr type pos we dr lddr dw", ("X", "rows", "dr"),
              ("ldx", "ldr", "lddr"))]
    for fn, names, pointers, strides in calls:
        def f(**kw):
            return call(fn, names, d, **kw)
        assert f(type=3) == UNSUPPORTED and f(T=-1) == INVALID and f(R=-1) == INVALID and f(D=-1) == INVALID
        assert f(top=0) == INVALID and f(top=33) == UNSUPPORTED and f(T=2 ** 30) == UNSUPPORTED
        assert f(R=2 ** 31) == UNSUPPORTED and f(pos=None) == INVALID and f(pos=P + 2) == MISALIGNED
        assert f(T=2 ** 28, top=1, D=2 ** 20, ldx=2 ** 20, ldr=2 ** 20, ldo=2 ** 20, lddr=2 ** 20) == UNSUPPORTED
        for name in pointers:
            assert f(**{name: None}) == INVALID and f(**{name: P + 8}) == MISALIGNED
        for name in strides:
            assert f(**{name: 56}) == INVALID and f(**{name: 68}) == MISALIGNED
            assert f(**{name: 2 ** 31}) == UNSUPPORTED
        assert f(T=0) == OK
    assert call(lib.expert_combine, calls[1][1], d, we=P + 2) == MISALIGNED
    for bad in (0, 2, 3):                               # bfloat16 rows give bfloat16
        assert call(lib.expert_combine, calls[1][1], d, otype=bad) == UNSUPPORTED
    assert call(lib.expert_combine, calls[1][1], d, type=2, otype=3) == UNSUPPORTED
    assert call(lib.expert_combine, calls[1][1], d, type=2, otype=0, ldo=68) == MISALIGNED
    assert call(lib.expert_combine_grad, calls[2][1], d, dw=P + 2) == MISALIGNED


def test_w4_conversions(lib):
    d = dict(G=3, N=100, K=72, X=P, ldx=72, xtype=1, group=32, Q=P, S=P, Z=P, lds=112, stype=1)
    for fn, names in ((lib.w4_quantize, "G N K X ldx xtype group Q S Z lds stype"),
                      (lib.w4_dequantize, "G N K Q S Z lds stype group X ldx xtype")):
        def f(**kw):
            return call(fn, names, d, **kw)
        assert f(xtype=3) == UNSUPPORTED and f(stype=2) == UNSUPPORTED and f(group=16) == UNSUPPORTED
        assert f(G=-1) == INVALID and f(N=-1) == INVALID and f(K=-1) == INVALID and f(ldx=64) == INVALID
        assert f(lds=96) == INVALID and f(lds=104) == MISALIGNED and f(ldx=76) == MISALIGNED
        assert f(K=2 ** 24, ldx=2 ** 24) == UNSUPPORTED and f(N=2 ** 31, lds=2 ** 31) == UNSUPPORTED
        for name in ("X", "Q", "S"):
            assert f(**{name: None}) == INVALID
        for name in ("X", "Q", "S", "Z"):
            assert f(**{name: P + 8}) == MISALIGNED
        assert f(G=0) == OK and f(N=0) == OK and f(K=0) == OK


def test_w4_products(lib):
    d = dict(G=3, M=8, N=48, K=72, alpha=1.0, A=P, lda=72, Q=P, S=P, Z=P, lds=96, group=32, off=P, beta=0.0, C=P,
             ldc=48, type=1, ctype=1)
    for fn, names in ((lib.gemm_w4, "G M N K alpha A lda Q S Z lds group off beta C ldc type ctype"),
                      (lib.swiglu_w4, "G M N K alpha A lda Q S Z lds group off C ldc type")):
        def f(**kw):
            return call(fn, names, d, **kw)
        assert f(type=2) == UNSUPPORTED and f(group=48) == UNSUPPORTED and f(G=1025) == UNSUPPORTED
        assert f(G=-1) == INVALID and f(M=-1) == INVALID and f(N=-1) == INVALID and f(K=-1) == INVALID
        assert f(off=None) == INVALID and f(off=P + 2) == MISALIGNED and f(lda=64) == INVALID
        assert f(ldc=40) == INVALID and f(lds=32) == INVALID and f(lds=104) == MISALIGNED
        assert f(lda=76) == MISALIGNED and f(ldc=52) == MISALIGNED
        for name in ("A", "Q", "S", "C"):
            assert f(**{name: None}) == INVALID
        for name in ("A", "Q", "S", "Z", "C"):
            assert f(**{name: P + 8}) == MISALIGNED
        assert f(M=2 ** 31) == UNSUPPORTED and f(K=2 ** 31, lda=2 ** 31) == UNSUPPORTED
        assert f(M=2 ** 31 - 1024, N=2 ** 20, lds=2 ** 21, ldc=2 ** 20) == UNSUPPORTED     # more CTAs than a grid has
        assert f(M=0) == OK and f(N=0) == OK and f(G=0) == OK
    assert call(lib.gemm_w4, "G M N K alpha A lda Q S Z lds group off beta C ldc type ctype", d, ctype=3) == UNSUPPORTED
    assert call(lib.swiglu_w4, "G M N K alpha A lda Q S Z lds group off C ldc type", d, N=2 ** 30, lds=2 ** 31 - 16,
                ldc=2 ** 30) == UNSUPPORTED


def helper_calls():
    """Each *_into helper with arguments that fit, as (function, tensors, the rest)."""
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    off = torch.tensor([0, 3, 8], dtype=torch.int32)
    plan = (i(17), i(24), i(8, 3))
    Q, S, Z = swg.w4_alloc(32, 40, 32, torch.bfloat16, zeros=True, experts=2, device="cpu")
    return [
        (swg.expert_route_into, dict(experts=i(8, 3), weights=f(8, 3), logits=z(8, 16), bias=f(16)), dict(plan=plan)),
        (swg.expert_sort_into, dict(experts=i(8, 3)), dict(plan=plan)),
        (swg.expert_route_grad_into, dict(d_logits=z(8, 16), d_weights=f(8, 3), logits=z(8, 16), experts=i(8, 3)), {}),
        (swg.expert_dispatch_into, dict(rows=z(24, 16), X=z(8, 16), position=i(8, 3)), {}),
        (swg.expert_combine_into, dict(out=z(8, 16), rows=z(24, 16), position=i(8, 3), weights=f(8, 3)), {}),
        (swg.expert_combine_grad_into, dict(d_rows=z(24, 16), d_weights=f(8, 3), d_out=z(8, 16), rows=z(24, 16),
                                            position=i(8, 3), weights=f(8, 3)), {}),
        (swg.w4_quantize_into, dict(Q=Q, S=S, Z=Z, W=z(2, 32, 40)), dict(group=32)),
        (swg.w4_dequantize_into, dict(W=z(2, 32, 40), Q=Q, S=S, Z=Z), dict(group=32)),
        (swg.gemm_w4_into, dict(C=z(8, 32), A=z(8, 40), Q=Q, S=S, Z=Z, offsets=off), dict(group=32)),
        (swg.swiglu_w4_into, dict(Y=z(8, 16), A=z(8, 40), Q=Q, S=S, Z=Z, offsets=off), dict(group=32)),
    ]


@pytest.mark.parametrize("i", range(10))
def test_tensors_on_the_host_are_refused(lib, i):
    f, tensors, rest = helper_calls()[i]
    with pytest.raises(swg.SwgError, match="current CUDA device") as e:
        f(**tensors, **rest)
    assert e.value.status == INVALID


@pytest.mark.parametrize("i", range(10))
def test_helpers_check_shapes_and_types(lib, i):
    """Each tensor in turn of another type, with a row less, or transposed."""
    f, tensors, rest = helper_calls()[i]
    for name, t in tensors.items():
        other = t.double() if t.is_floating_point() else t.long()
        for bad in (other, t[:-1], t.unsqueeze(0).unsqueeze(0), t.flip(-1)[..., ::2]):
            with pytest.raises(swg.SwgError):
                f(**{**tensors, name: bad}, **rest)
    for k in range(3 if "plan" in rest else 0):
        plan = list(rest["plan"])
        plan[k] = plan[k].long()
        with pytest.raises(swg.SwgError):
            f(**tensors, plan=plan)
    if "group" in rest:
        with pytest.raises(swg.SwgError) as e:
            f(**tensors, group=48)
        assert e.value.status == UNSUPPORTED
