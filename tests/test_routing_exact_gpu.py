"""Choices that FP32 cannot tell apart, by the ways in which the router decides them."""
import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from experts_plain import f64
from test_routing_gpu import INF, run_route

pytestmark = pytest.mark.gpu


def chosen(l, bias, top, **kw):
    T = l.shape[0]
    experts = torch.empty((T, top), dtype=torch.int32, device="cuda")
    swg.expert_route_into(experts, torch.empty((T, top), device="cuda"), l.cuda(), bias=bias.cuda(), **kw)
    assert swg.get_device_error() == 0
    return experts.cpu()


@pytest.mark.parametrize("E", [64, 300])
@pytest.mark.parametrize("apart", [-28, -30, -32])
def test_every_way_has_the_same_order(E, apart):
    """Experts 3 and 5, whose choices differ by less than a unit of FP64 or not at all:
    decided among the candidates, and, next to a bias of +inf, among all experts."""
    T = 400
    rng = np.random.default_rng(1)
    l = np.tile(rng.normal(size=E).astype(np.float32) - 3, (T, 1))
    l[:, 5], l[:, 3] = 0.0, -2.0 ** apart
    l[:, 7] = -5.0 - np.arange(T) * 2.0 ** -20           # what moves the sum, a little
    e = np.exp(l.astype(np.float64))
    bias = torch.zeros(E)
    bias[3] = float((e[T // 2, 5] - e[T // 2, 3]) / e[T // 2].sum())
    s = plain.scores(l[T // 2:T // 2 + 1].astype(np.float64), "softmax")[0]
    assert abs(s[5] - s[3] - float(bias[3])) < 2.0 ** -52
    l = torch.from_numpy(l)
    bias[E - 2] = -INF                                   # of the softmax, and not chosen
    few = chosen(l, bias, 5)
    bias[E - 2] = INF
    all_of_them = chosen(l, bias, 6)
    assert bool((all_of_them[:, 0] == E - 2).all())
    assert bool((few == 3).any(1).all()) and bool((few == 5).any(1).all())
    assert torch.equal(few, all_of_them[:, 1:])


SMALL = [-39.0, -86.0, -87.3, -87.4, -88.0, -88.7, -88.8, -90.0, -95.0, -100.0, -102.0, -103.0]


@pytest.mark.parametrize("E", [16, 15])                  # four tokens of a warp, and one
@pytest.mark.parametrize("normalise", [False, True])
def test_weights_of_small_sigmoids(E, normalise):
    """Sigmoids below FP32's smallest normal number, and beside others from which they are far."""
    l = torch.full((3, E), -INF)
    l[:, :12] = torch.tensor(SMALL)
    l[1, 0] = -INF
    l[2, 0] = 3.0
    scale = 2.0 ** 20
    weights = torch.empty((3, 8), device="cuda")
    for first in (0, 4):
        x = l.clone()
        x[:, 1:1 + first] = -INF
        experts = torch.empty((3, 8), dtype=torch.int32, device="cuda")
        swg.expert_route_into(experts, weights, x.cuda(), swg.SIGMOID, normalise=normalise, scale=scale)
        assert swg.get_device_error() == 0
        want, w = plain.route(f64(x), None, 8, "sigmoid", normalise=normalise, scale=scale)
        assert np.array_equal(experts.cpu().numpy(), want)
        if normalise:
            tol = plain.route_bound(f64(x), w, 8) - 1e-37 + scale * 2.0 ** -149     # (a share may be subnormal)
        else:
            # exponential and division 2 units each, half a one of 1 + e^x; the product is exact
            tol = 5 * 2.0 ** -23 * w + scale * 5 * 2.0 ** -149
        got = f64(weights)
        assert (np.abs(got - w) <= tol).all(), f"{got[np.abs(got - w) > tol]} {w[np.abs(got - w) > tol]}"


def test_gradients_of_small_sigmoids():
    x = torch.tensor([[*SMALL, *(-v for v in SMALL)]]).reshape(6, 4)
    experts = torch.arange(4, dtype=torch.int32).repeat(6, 1).cuda()
    dw = torch.linspace(-2, 3, 24).reshape(6, 4)
    d = torch.empty((6, 4), device="cuda")
    scale = 2.0 ** 20
    swg.expert_route_grad_into(d, dw.cuda(), x.cuda(), experts, swg.SIGMOID, normalise=False, scale=scale)
    assert swg.get_device_error() == 0
    e = np.exp(-np.abs(f64(x)))
    want = scale * f64(dw) * e / (1 + e) ** 2
    # both scores: exponential 2 units, two halves; three products, half a one each
    tol = 7.5 * 2.0 ** -23 * np.abs(want) + scale * np.abs(f64(dw)) * 5 * 2.0 ** -149
    assert (np.abs(f64(d) - want) <= tol).all()


@pytest.mark.parametrize("E", [256, 1024])
@pytest.mark.parametrize("groups", [1, 4])
def test_one_score_above_many_equal_ones(E, groups):
    """All logits but one are the same, so that what their exponentials are off by does not
    cancel in their sum, and biases bring the choices of six within a unit of FP32 of the one's:
    the error of the sum moves a difference of choices by more than is between them."""
    met = 0
    for low in np.linspace(-7.0, -3.0, 25).astype(np.float32):
        l = torch.full((1, E), float(low))
        l[0, E // 2] = 0.0
        s = plain.scores(f64(l), "softmax")[0]
        for j in (-2, -1, 0, 1, 2):
            bias = torch.full((E,), -1.0)
            bias[1:7] = 0.25 + torch.arange(6) * 2.0 ** -25
            bias[E // 2] = float(np.float32(0.25 + 2.0 ** -24 + s[1] - s[E // 2])) + j * 2.0 ** -26
            c = np.sort(s + f64(bias))[-7:]
            if np.diff(c).min() < 1e-14:
                continue
            met += 1
            run_route(l, 4, bias=bias, groups=groups, top_groups=max(groups // 2, 1), group_sum=2)
    assert met > 100
