"""A whole expert layer, trained: route, dispatch, the grouped products and
combine, and their gradients back to tokens, logits and weights, against
autograd in 64 bits."""
import pytest
import torch

import swiglu_mlp_gb300 as swg
from test_routing_gpu import gen

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("T,E,top,D,H,score,normalise", [(150, 6, 2, 200, 136, "softmax", True), (70, 9, 3, 64, 72, "sigmoid", True),
                                                        (33, 4, 2, 72, 64, "softmax", False)])
def test_layer_and_gradients(T, E, top, D, H, score, normalise):
    code = {"softmax": swg.SOFTMAX, "sigmoid": swg.SIGMOID}[score]
    bf = lambda *s, seed, std: (torch.randn(s, generator=gen(seed)) * std).bfloat16()  # noqa: E731
    x, d_out = bf(T, D, seed=1, std=1.0), bf(T, D, seed=2, std=1.0)
    wu, wd = bf(E, D, 2 * H, seed=3, std=D ** -0.5), bf(E, H, D, seed=4, std=H ** -0.5)
    l = torch.randn((T, E), generator=gen(5)) * 2
    l[T // 2] = -float("inf")                            # a padding token
    new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    X, DO, WU, WD, L = (t.cuda() for t in (x, d_out, wu, wd, l))
    experts, weights, plan = new(T, top, t=torch.int32), new(T, top, t=torch.float32), swg.expert_plan_alloc(T, E, top)
    swg.expert_route_into(experts, weights, L, code, normalise=normalise, plan=plan)
    off, _, pos = plan
    rows = swg.expert_dispatch_into(new(T * top, D), X, pos)
    y = swg.swiglu_grouped_into(new(T * top, H), rows, WU, off)
    z = swg.gemm_grouped_into(new(T * top, D), y, WD, off)
    out = swg.expert_combine_into(new(T, D), z, pos, weights)
    dz, dw = swg.expert_combine_grad_into(new(T * top, D), new(T, top, t=torch.float32), DO, z, pos, weights)
    dl = swg.expert_route_grad_into(new(T, E, t=torch.float32), dw, L, experts, code, normalise=normalise)
    dy = swg.gemm_grouped_into(new(T * top, H), dz, WD, off, transB=1)
    dh = swg.swiglu_grouped_grad_into(new(T * top, 2 * H), rows, WU, dy, off)
    drows = swg.gemm_grouped_into(new(T * top, D), dh, WU, off, transB=1)
    dx = swg.expert_combine_into(new(T, D), drows, pos)
    dwu = swg.gemm_grouped_wgrad_into(new(E, D, 2 * H), rows, dh, off)
    dwd = swg.gemm_grouped_wgrad_into(new(E, H, D), y, dz, off)
    assert swg.get_device_error() == 0

    x64, wu64, wd64, l64 = (t.double().requires_grad_() for t in (x, wu, wd, l))
    e = experts.cpu().long()
    on = e >= 0
    assert int((~on).sum()) == top and not on[T // 2].any()
    live = torch.where(torch.isinf(l64), torch.zeros_like(l64), l64)
    s = live.softmax(-1) if score == "softmax" else live.sigmoid()
    w = s.gather(1, e.clamp(min=0)) * on
    if normalise:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    want = torch.zeros(T, D, dtype=torch.float64)
    for k in range(E):
        t, j = (e == k).nonzero(as_tuple=True)
        h = x64[t] @ wu64[k]
        want = want.index_add(0, t, (torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2]) @ wd64[k] * w[t, j][:, None])
    want.backward(d_out.double())
    # roundings to bf16 on the way, at most half a unit, 2^-8, each: two forward and the
    # last, and as many back; each grows by at most 1.5 (the norms of random weights) twice
    step = 2.0 ** -8
    assert rel(out, want.detach()) < 4 * step
    for got, ref in ((dx, x64.grad), (dwu, wu64.grad), (dwd, wd64.grad), (dl, l64.grad)):
        assert rel(got, ref) < 8 * step
