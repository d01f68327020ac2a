"""The router, the plan of rows, and rows to the experts and back, against their
64-bit forms (routing_plain.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from experts_plain import f64, fp32_sum_bound
from helpers import Guarded
from test_routing_host import helper_calls

pytestmark = pytest.mark.gpu

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SCORE = {"softmax": swg.SOFTMAX, "sigmoid": swg.SIGMOID}
INF = float("inf")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def logits_of(T, E, dtype, seed, ties=False):
    x = torch.randn((T, E), generator=gen(seed)) * 1.5
    return ((x * 4).round() / 4 if ties else x).to(TYPE[dtype])


def close(got, want, tol, what=""):
    got = f64(got)
    assert got.shape == want.shape
    same = (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
    assert same.all(), f"{what}: {(~same).sum()} of {same.size} off, e.g. {np.argwhere(~same)[:4].tolist()}, " \
        f"got {got[~same][:4]}, want {want[~same][:4]}, bound {np.broadcast_to(tol, same.shape)[~same][:4]}"


def check_plan(p, experts, E):
    for got, want, name in zip(p, plain.plan(experts, E), ("offsets", "source", "position")):
        assert np.array_equal(got.cpu().numpy(), want), name


def run_route(l, top, bias=None, score="softmax", groups=1, top_groups=None, group_sum=1, normalise=True, scale=1.0,
              planned=True, stream=None):
    """Routes l (on the CPU, any strides) and compares with the definition."""
    T, E = l.shape
    d = l.cuda()
    experts = torch.full((T, top), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((T, top), 7.0, device="cuda")
    p = swg.expert_plan_alloc(T, E, top) if planned else None
    torch.cuda.synchronize()
    swg.expert_route_into(experts, weights, d, SCORE[score], bias=None if bias is None else bias.cuda(), groups=groups,
                          top_groups=top_groups, group_sum=group_sum, normalise=normalise, scale=scale, plan=p, stream=stream)
    assert swg.get_device_error(stream) == 0
    l64 = f64(l)
    want, w = plain.route(l64, None if bias is None else f64(bias), top, score, groups, top_groups, group_sum, normalise, scale)
    got = experts.cpu().numpy()
    assert np.array_equal(got, want), f"{np.argwhere((got != want).any(1)).ravel()[:5]} {got[(got != want).any(1)][:3]} {want[(got != want).any(1)][:3]}"
    close(weights, w, plain.route_bound(l64, w, top), "weights")
    if planned:
        check_plan(p, want, E)
    return experts, weights, p


CHOICES = [dict(), dict(normalise=False), dict(score="sigmoid"), dict(score="sigmoid", normalise=False, scale=2.5)]


@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 33, 4), (64, 64, 8), (65, 64, 6), (200, 160, 6),
                                     (97, 256, 8), (33, 257, 3), (40, 512, 32), (20, 1000, 10), (70, 1024, 32)])
@pytest.mark.parametrize("how", range(4))
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_choices(T, E, top, how, dtype):
    kw = CHOICES[how]
    l = logits_of(T, E, dtype, T + E)
    run_route(l, top, **kw)
    bias = torch.randn(E, generator=gen(E)) * 0.05
    run_route(l, top, bias=bias, planned=False, **kw)


@pytest.mark.parametrize("E,groups,top_groups,top", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 8, 1, 8), (48, 4, 2, 3), (21, 7, 3, 5),
                                                     (32, 32, 5, 5), (1024, 32, 7, 9), (96, 3, 2, 6), (10, 2, 2, 4), (1000, 2, 1, 8)])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("how", range(4))
def test_groups(E, groups, top_groups, top, group_sum, how):
    l = logits_of(70, E, "f32", E + groups)
    kw = dict(groups=groups, top_groups=top_groups, group_sum=group_sum, **CHOICES[how])
    run_route(l, top, **kw)
    run_route(l, top, bias=torch.randn(E, generator=gen(3)) * 0.1, **kw)
    # bf16 logits on a coarse grid: many ties
    run_route(logits_of(70, E, "bf16", E, ties=True), top, **kw)
    run_route(logits_of(70, E, "bf16", E, ties=True), top, bias=torch.zeros(E), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 256, 1024])
def test_ties_go_to_the_lowest(score, E):
    run_route(torch.zeros(9, E), min(E, 8), score=score)
    run_route(torch.zeros(9, E), min(E, 8), score=score, bias=torch.zeros(E), groups=4, top_groups=2, group_sum=2)
    run_route(logits_of(300, E, "bf16", 5, ties=True), 6, score=score, bias=torch.zeros(E))
    l = torch.zeros(2, E)
    l[0, 1::2] = -0.0                                    # zeros are equal
    run_route(l, 4, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_choices_nearer_than_fp32_can_tell(score, groups):
    """Biases that make all choices of a token equal but for 1e-11 to 1e-8: the order is
    the exact one."""
    E = 64
    rng = np.random.default_rng(7)
    rows = []
    for t in range(100):
        l = rng.normal(size=E).astype(np.float32).astype(np.float64)
        s = plain.scores(l[None], score)[0]
        bias = (0.4 - s + rng.uniform(1e-11, 1e-8, E) * 10 ** rng.uniform(0, 3)).astype(np.float32)
        c = s + bias.astype(np.float64)
        if np.diff(np.sort(c)).min() > 1e-14:
            rows.append((l, bias))
    assert len(rows) > 50
    for l, bias in rows[:12]:
        run_route(torch.from_numpy(l[None]).float().repeat(3, 1), 7, bias=torch.from_numpy(bias), score=score, groups=groups,
                  top_groups=max(groups // 2, 1), group_sum=2)


def test_masked_experts_and_tokens():
    l = logits_of(80, 40, "f32", 11)
    l[3] = -INF                                          # nothing is left
    l[4, 1:] = -INF                                      # one is
    l[5, ::2] = -INF
    l[70:] = -INF                                        # padding at the end
    l[6] = torch.finfo(torch.float32).min                # the type's lowest is a logit like another
    l[7, :20] = torch.finfo(torch.float32).min
    for how in CHOICES:
        run_route(l, 6, **how)
        run_route(l, 6, groups=8, top_groups=2, group_sum=2, **how)
        bias = torch.zeros(40)
        bias[3] = -INF
        bias[4] = 100.0
        run_route(l, 6, bias=bias, **how)
        run_route(l, 6, bias=bias, groups=5, top_groups=1, **how)
    run_route(torch.full((100, 12), -INF), 3, bias=torch.ones(12))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    l = logits_of(8, 24, "f32", 12)
    l[0] = torch.linspace(-3e38, 3e38, 24, dtype=torch.float64).float()
    l[1] -= 200.0                                        # sigmoids below the smallest float
    l[2] += 200.0
    l[3, 5] = float("nan")
    l[4, 5] = INF
    l[5] = torch.linspace(-90, -39, 24)
    l[6] = torch.linspace(-60, 60, 24)
    for normalise in (True, False):
        run_route(l, 4, score=score, normalise=normalise)
        run_route(l, 4, score=score, normalise=normalise, bias=torch.linspace(0, 1, 24))
        run_route(l, 4, score=score, normalise=normalise, groups=4, top_groups=2, group_sum=2)


def test_strides_and_alignment():
    """Rows of any stride, from any element on."""
    for dtype in ("f32", "bf16"):
        big = logits_of(90, 150, dtype, 13).cuda()
        l = big[:, 7:7 + 101]
        experts = torch.empty((90, 5), dtype=torch.int32, device="cuda")
        weights = torch.empty((90, 5), device="cuda")
        swg.expert_route_into(experts, weights, l)
        assert np.array_equal(experts.cpu().numpy(), plain.route(f64(l), None, 5)[0])
        d = torch.full((90, 140), 9.0, dtype=TYPE[dtype], device="cuda")
        swg.expert_route_grad_into(d[:, 3:104], weights, l, experts)
        assert bool((d[:, :3] == 9).all()) and bool((d[:, 104:] == 9).all())
    one = torch.randn(1, 64, device="cuda")[:, ::1]
    run_route(one.cpu(), 3)


@pytest.mark.parametrize("T", [0, 1, 63, 64, 65, 1000, 5003])
def test_many_tokens(T):
    l = logits_of(T, 24, "bf16", T)
    if T > 10:
        l[-7:] = -INF
    run_route(l, 3)
    run_route(l, 3, planned=False)
    run_route(l, 3, score="sigmoid", bias=torch.randn(24, generator=gen(1)) * 0.02)


def test_repeats_bit_for_bit():
    l = logits_of(4000, 128, "f32", 21)
    a = run_route(l, 8, score="sigmoid", bias=torch.randn(128, generator=gen(2)) * 0.05, groups=8, top_groups=4, group_sum=2)
    b = run_route(l, 8, score="sigmoid", bias=torch.randn(128, generator=gen(2)) * 0.05, groups=8, top_groups=4, group_sum=2)
    assert all(torch.equal(x, y) for x, y in zip(a[:2] + a[2], b[:2] + b[2]))


# -------------------------------------------------------------------- plan

@pytest.mark.parametrize("T,E,top", [(0, 4, 2), (1, 1, 1), (5, 3, 2), (100, 64, 8), (512, 8, 8), (513, 8, 8), (3000, 200, 4),
                                     (700, 1024, 32), (40000, 16, 2), (4097, 1, 1), (2000, 600, 3)])
def test_sort(T, E, top):
    rng = np.random.default_rng(T + E)
    e = rng.integers(-1, E, (T, top)).astype(np.int32)
    for experts in (e, np.where(e > 0, 0, e), np.full_like(e, E - 1), np.full_like(e, -1)):
        p = swg.expert_plan_alloc(T, E, top)
        for x in p:
            x.fill_(99)
        swg.expert_sort_into(p, torch.from_numpy(experts).cuda())
        assert swg.get_device_error() == 0
        check_plan(p, experts, E)


@pytest.mark.parametrize("T", [20, 3000])
def test_sort_reports_wrong_experts(T):
    e = np.random.default_rng(1).integers(0, 10, (T, 4)).astype(np.int32)
    e[T // 2, 1], e[3, 2], e[T - 1, 3] = 10, -2, 2 ** 31 - 1
    p = swg.expert_plan_alloc(T, 10, 4)
    swg.expert_sort_into(p, torch.from_numpy(e).cuda())
    assert swg.get_device_error() == 1 and swg.get_device_error() == 0
    check_plan(p, np.where((e < 0) | (e >= 10), -1, e), 10)


# --------------------------------------------------------------- gradients

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("how", range(4))
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (9, 8, 2), (50, 33, 6), (17, 256, 8), (5, 1000, 32), (3, 512, 4)])
def test_route_grad(T, E, top, how, dtype):
    kw = dict(score="softmax", normalise=True, scale=1.0)
    kw.update(CHOICES[how])
    l = logits_of(T, E, dtype, T * E)
    experts, _ = plain.route(f64(l), None, top, **kw)
    rng = np.random.default_rng(E)
    experts[rng.random(experts.shape) < 0.1] = -1        # slots without an expert
    if T > 4:
        experts[1] = -1
        experts[2, -1] = experts[2, 0]                   # an expert twice
    dw = torch.randn((T, top), generator=gen(4))
    dw[torch.from_numpy(experts) < 0] = float("nan")     # which says nothing
    d = Guarded(T, E, TYPE[dtype], fill=5.0)
    swg.expert_route_grad_into(d.view, dw.cuda(), l.cuda(), torch.from_numpy(experts.astype(np.int32)).cuda(),
                               SCORE[kw["score"]], normalise=kw["normalise"], scale=kw["scale"])
    assert swg.get_device_error() == 0
    want, mags = plain.route_grad(f64(l), experts, f64(dw), **kw)
    close(d.cpu(), want, plain.grad_bound(f64(l), want, mags, top, dtype), "d_logits")


@pytest.mark.parametrize("how", range(4))
def test_route_grad_against_differences(how):
    kw = dict(score="softmax", normalise=True, scale=1.0)
    kw.update(CHOICES[how])
    T, E, top = 4, 12, 3
    l = logits_of(T, E, "f32", 31)
    x, dw = f64(l), np.random.default_rng(5).normal(size=(T, top))
    experts, _ = plain.route(x, None, top, **kw)

    def loss(x, t):
        s = plain.scores(x[t:t + 1], kw["score"])[0, experts[t]]
        return kw["scale"] * ((s / s.sum() if kw["normalise"] else s) * dw[t]).sum()

    want = np.empty((T, E))
    h = 1e-5                                             # differences are off by h^2 and 1e-16 / h
    for t in range(T):
        for e in range(E):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            want[t, e] = (loss(up, t) - loss(down, t)) / (2 * h)
    d = torch.empty((T, E), device="cuda")
    swg.expert_route_grad_into(d, torch.from_numpy(dw).float().cuda(), l.cuda(), torch.from_numpy(experts.astype(np.int32)).cuda(),
                               SCORE[kw["score"]], normalise=kw["normalise"], scale=kw["scale"])
    mags = plain.route_grad(x, experts, dw, **kw)[1]
    # dw was rounded to FP32: one more U of the magnitudes
    close(d, want, plain.grad_bound(x, want, mags, top, "f32") + plain.U * mags + 1e-9, "differences")


def test_route_grad_extremes():
    l = logits_of(6, 16, "f32", 41)
    l[0] -= 200.0
    l[1, 3:] = -INF
    l[2] = -INF
    l[3, 2] = -INF
    for how in range(4):
        kw = dict(score="softmax", normalise=True, scale=1.0)
        kw.update(CHOICES[how])
        experts, _ = plain.route(f64(l), None, 4, **kw)
        dw = torch.randn((6, 4), generator=gen(6))
        d = torch.full((6, 16), 3.0, device="cuda")
        swg.expert_route_grad_into(d, dw.cuda(), l.cuda(), torch.from_numpy(experts.astype(np.int32)).cuda(),
                                   SCORE[kw["score"]], normalise=kw["normalise"], scale=kw["scale"])
        want, mags = plain.route_grad(f64(l), experts, f64(dw), **kw)
        close(d, want, plain.grad_bound(f64(l), want, mags, 4, "f32"), f"{kw}")


def test_route_grad_reports_wrong_experts():
    l = logits_of(3, 8, "f32", 42)
    e = np.array([[0, 1], [2, 8], [-2, 3]], np.int32)
    dw = torch.ones(3, 2)
    d = torch.empty((3, 8), device="cuda")
    swg.expert_route_grad_into(d, dw.cuda(), l.cuda(), torch.from_numpy(e).cuda(), normalise=False)
    assert swg.get_device_error() == 1
    e = np.where((e < 0) | (e > 7), -1, e)
    want, mags = plain.route_grad(f64(l), e, f64(dw), "softmax", False, 1.0)
    close(d, want, plain.grad_bound(f64(l), want, mags, 2, "f32"))


# -------------------------------------------------------------- moving rows

def a_plan(T, E, top, seed, none=0.15):
    rng = np.random.default_rng(seed)
    e = np.stack([rng.permutation(max(E, top))[:top] for _ in range(T)]) if T else np.zeros((0, top), int)
    e = np.where((rng.random(e.shape) < none) | (e >= E), -1, e)
    return plain.plan(e, E)[2]


def padded(rows, cols, dtype, seed, std=1.0):
    """In storage with NaN behind each row's columns."""
    per = 4 if dtype == "f32" else 8
    t = torch.full((rows, -(-cols // per) * per + per), float("nan"), dtype=TYPE[dtype])
    t[:, :cols] = (torch.randn((rows, cols), generator=gen(seed)) * std).to(TYPE[dtype])
    return t.cuda()[:, :cols]


SHAPES = [(1, 1, 1, 1), (1, 4096, 8, 8), (5, 8, 4, 2), (33, 129, 16, 4), (64, 2051, 48, 6), (7, 8200, 9, 3), (300, 520, 8, 32),
          (2000, 264, 64, 2), (700, 4100, 4, 1), (3, 64, 2, 5),
          (2600, 1030, 64, 5), (5000, 20, 8, 2)]


@pytest.mark.parametrize("T,D,E,top", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dispatch(T, D, E, top, dtype):
    pos = a_plan(T, E, top, T + D)
    X = padded(T, D, dtype, 1)
    rows = Guarded(T * top, D, TYPE[dtype], fill=3.0)
    swg.expert_dispatch_into(rows.view, X, torch.from_numpy(pos.astype(np.int32)).cuda())
    assert swg.get_device_error() == 0
    want = np.full((T * top, D), 3.0)
    for t in range(T):
        for p in pos[t][pos[t] >= 0]:
            want[p] = f64(X)[t] if T < 50 else 0
    if T >= 50:
        x = f64(X)
        t, j = np.nonzero(pos >= 0)
        want[pos[t, j]] = x[t]
    assert np.array_equal(f64(rows.cpu("dispatch")), want)


@pytest.mark.parametrize("T,D,E,top", SHAPES)
@pytest.mark.parametrize("source,dtype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("weighted,beta", [(True, 0.0), (False, 1.0), (True, -0.5)])
def test_combine(T, D, E, top, source, dtype, weighted, beta):
    pos = a_plan(T, E, top, T + D)
    rows = padded(T * top, D, source, 2)
    used = pos[pos >= 0]
    idle = np.setdiff1d(np.arange(T * top), used)
    rows[torch.from_numpy(idle).cuda()] = float("nan")   # rows of no slot
    w = torch.randn((T, top), generator=gen(3)) if weighted else torch.ones(T, top)
    old = torch.randn((T, D), generator=gen(4)).to(TYPE[dtype])
    given = w.clone()
    given[torch.from_numpy(pos) < 0] = float("nan")
    out = Guarded(T, D, TYPE[dtype], init=old if beta else torch.full((T, D), float("nan"), dtype=TYPE[dtype]))
    swg.expert_combine_into(out.view, rows, torch.from_numpy(pos.astype(np.int32)).cuda(), given.cuda() if weighted else None,
                            beta=beta)
    assert swg.get_device_error() == 0
    want, tol = plain.combine(f64(rows), pos, f64(w), beta, f64(old) if beta else np.zeros((T, D)), dtype)
    close(out.cpu("combine"), want, tol, "combine")


@pytest.mark.parametrize("T,D,E,top", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(T, D, E, top, dtype, weighted):
    pos = a_plan(T, E, top, T + D)
    rows, d_out = padded(T * top, D, dtype, 5), padded(T, D, dtype, 6)
    w = torch.randn((T, top), generator=gen(7)) if weighted else torch.ones(T, top)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    d_rows = Guarded(T * top, D, TYPE[dtype], fill=3.0)
    d_w = torch.full((T, top), 9.0, device="cuda")
    swg.expert_combine_grad_into(d_rows.view, d_w, d_out, rows, p, w.cuda() if weighted else None)
    assert swg.get_device_error() == 0
    want, x, r = np.full((T * top, D), 3.0), f64(d_out), f64(rows)
    t, j = np.nonzero(pos >= 0)
    want[pos[t, j]] = f64(w)[t, j][:, None] * x[t]
    close(d_rows.cpu("d_rows"), want, plain.ROUND[dtype] * np.abs(want) + plain.TINY[dtype], "d_rows")
    dw, tol = np.zeros((T, top)), np.zeros((T, top))
    dw[t, j] = (r[pos[t, j]] * x[t]).sum(1)
    tol[t, j] = fp32_sum_bound(D, (np.abs(r[pos[t, j]]) * np.abs(x[t])).sum(1))
    close(d_w, dw, tol, "d_weights")
    # without the weights' gradient the rows are not needed
    again = Guarded(T * top, D, TYPE[dtype], fill=3.0)
    swg.expert_combine_grad_into(again.view, None, d_out, None, p, w.cuda() if weighted else None)
    assert torch.equal(again.cpu().nan_to_num(-7), d_rows.cpu().nan_to_num(-7))


def test_dispatch_and_combine_are_transposes():
    """<dispatch(x), y> = <x, combine(y)>: the gradient of dispatch is combine without weights."""
    pos = a_plan(40, 16, 4, 1)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    x, y = torch.randn(40, 100, generator=gen(1)).cuda(), torch.randn(160, 100, generator=gen(2)).cuda()
    rows = torch.zeros(160, 100, device="cuda")
    swg.expert_dispatch_into(rows, x, p)
    out = swg.expert_combine_into(torch.empty_like(x), y, p)
    a, b = (rows.double() * y.double()).sum(), (x.double() * out.double()).sum()
    # each out element is off by 5 roundings of at most 4 terms
    assert abs(float(a - b)) <= 5 * plain.U * float((x.double().abs() * swg.expert_combine_into(
        torch.empty_like(x), y.abs(), p).double()).sum())


def test_wrong_positions_are_reported():
    x, rows, out = torch.ones(3, 16, device="cuda"), torch.full((6, 16), 2.0, device="cuda"), torch.empty(3, 16, device="cuda")
    p = torch.tensor([[0, 6], [-1, 2], [-2, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    swg.expert_combine_into(out, rows, p)
    assert swg.get_device_error() == 1
    assert out[:, 0].tolist() == [2.0, 2.0, 0.0]
    swg.expert_dispatch_into(rows, x, p)
    assert swg.get_device_error() == 1
    assert rows[:, 0].tolist() == [1.0, 2.0, 1.0, 2.0, 2.0, 2.0]
    d_w = torch.full((3, 2), 9.0, device="cuda")
    swg.expert_combine_grad_into(rows, d_w, x, torch.ones(6, 16, device="cuda"), p, torch.full((3, 2), 5.0, device="cuda"))
    assert swg.get_device_error() == 1
    assert d_w.tolist() == [[16.0, 0.0], [0.0, 16.0], [0.0, 0.0]] and rows[:, 0].tolist() == [5.0, 2.0, 5.0, 2.0, 2.0, 2.0]


def test_no_tokens_no_rows_no_columns():
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    swg.expert_dispatch_into(f(0, 8), f(0, 8), i(0, 2))
    swg.expert_combine_into(f(0, 8), f(0, 8), i(0, 2))
    out = f(4, 8)
    swg.expert_combine_into(out, f(0, 8), i(4, 2) - 1)   # no rows: nothing to add
    assert float(out.abs().sum()) == 0
    out = f(4, 8)
    swg.expert_combine_into(out, f(0, 8), i(4, 2) - 1, beta=2.0)
    assert float(out.sum()) == 64
    d_w = f(4, 2)
    swg.expert_combine_grad_into(f(8, 0), d_w, f(4, 0), f(8, 0), i(4, 2))
    assert float(d_w.abs().sum()) == 0
    swg.expert_route_into(i(0, 2), f(0, 2), f(0, 8))
    assert swg.get_device_error() == 0


def test_offsets_beyond_32_bits():
    """Rows and columns numbered in 64 bits: 2.3 * 10^9 elements of rows."""
    D, R = 8192, 280000
    rows = torch.empty((R, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[R - 1, 0], [-1, R - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, D, generator=gen(1)).bfloat16().cuda()
    swg.expert_dispatch_into(rows, x, pos)
    assert torch.equal(rows[R - 1], x[0]) and torch.equal(rows[0], x[0]) and torch.equal(rows[R - 2], x[1])
    out = swg.expert_combine_into(torch.empty_like(x), rows, pos)
    assert torch.equal(out[1], x[1]) and torch.equal(out[0], x[0] + x[0])
    d_rows = rows.fill_(0)
    swg.expert_combine_grad_into(d_rows, None, x, None, pos)
    assert torch.equal(d_rows[R - 1], x[0]) and torch.equal(d_rows[R - 2], x[1]) and swg.get_device_error() == 0


# ------------------------------------------------------- streams and graphs

def test_on_another_stream():
    s = torch.cuda.Stream()
    run_route(logits_of(500, 64, "bf16", 3), 4, stream=s)


def test_two_graphs_and_their_stream():
    """A routed plan of many tokens, captured twice, replayed beside one another with
    new inputs: each keeps its counts in a workspace of its own."""
    T, E, top = 3000, 64, 4
    sets = []
    for k in range(2):
        l = torch.zeros(T, E, device="cuda")
        sets.append((l, torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda"),
                     swg.expert_plan_alloc(T, E, top)))
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for l, e, w, p in sets:
            swg.expert_route_into(e, w, l, plan=p)
        s.synchronize()
        for l, e, w, p in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                swg.expert_route_into(e, w, l, plan=p)
            graphs.append(g)
    for seed in range(3):
        want = []
        for k, (l, e, w, p) in enumerate(sets):
            l.copy_(logits_of(T, E, "f32", 10 * seed + k))
            want.append(plain.route(f64(l), None, top)[0])
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        torch.cuda.synchronize()
        for (l, e, w, p), x in zip(sets, want):
            assert np.array_equal(e.cpu().numpy(), x)
            check_plan(p, x, E)


@pytest.mark.parametrize("i", range(10))
def test_helpers_accept_what_fits(i):
    """Each helper with the arguments that the tests of refusals start from."""
    f, tensors, rest = helper_calls()[i]
    rest = dict(rest)
    if "plan" in rest:
        rest["plan"] = tuple(x.cuda() for x in rest["plan"])
    f(**{k: v.cuda() for k, v in tensors.items()}, **rest)
    assert swg.get_device_error() == 0
