"""Choices that FP32 cannot tell apart, by the ways in which the router decides them."""
import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from test_routing_gpu import INF

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
