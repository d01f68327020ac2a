"""The router where four tokens share a warp (up to 256 experts, eight of them a
token): what a team of lanes decides alone, what the warp decides together for one of
the four, and calls that have to go the other way."""
import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from experts_plain import f64
from test_routing_gpu import CHOICES, INF, TYPE, gen, logits_of, run_route

pytestmark = pytest.mark.gpu


def near_row(E, score, seed, spread):
    """Logits and biases that make all choices of the token equal but for `spread`."""
    rng = np.random.default_rng(seed)
    while True:
        l = rng.normal(size=E).astype(np.float32).astype(np.float64)
        s = plain.scores(l[None], score)[0]
        bias = (0.4 - s + rng.uniform(1e-3, 1, E) * spread).astype(np.float32)
        c = s + bias.astype(np.float64)
        if np.diff(np.sort(c)).min() > 1e-14:
            return torch.from_numpy(l).float(), torch.from_numpy(bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(28, 1, 1), (64, 2, 1), (128, 4, 2), (128, 2, 1), (256, 8, 4), (256, 4, 3), (256, 2, 1), (66, 1, 1)])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("spread", [1e-9, 1e-7, 1e-5])
def test_near_choices_of_some_of_the_four(score, E, groups, top_groups, group_sum, spread):
    l = logits_of(23, E, "f32", E)
    for seed in range(3):
        row, bias = near_row(E, score, seed, spread)
        for at in ([0], [1, 2], [3, 5, 6], [19, 22]):
            x = l.clone()
            x[at] = row
            run_route(x, 8, bias=bias, score=score, groups=groups, top_groups=top_groups, group_sum=group_sum)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 2), (256, 8), (256, 4)])
def test_near_groups(score, E, groups):
    """Groups whose two largest add up to nearly the same, the largest apart."""
    size = E // groups
    for seed in range(6):
        rng = np.random.default_rng(seed)
        l = rng.normal(size=(9, E)).astype(np.float32)
        s = plain.scores(l[4:5].astype(np.float64), score)[0].reshape(groups, size)
        want = np.full((groups, size), 0.1)
        order = rng.permuted(np.tile(np.arange(size), (groups, 1)), axis=1)
        apart = rng.uniform(0.0, 0.1, groups)
        for g in range(groups):
            want[g, order[g, 0]] = 0.5 + apart[g]
            want[g, order[g, 1]] = 0.5 - apart[g] + rng.uniform(1e-3, 1) * 10.0 ** rng.integers(-9, -6)
            want[g, order[g, 2:]] -= rng.uniform(0, 0.1, size - 2)
        bias = torch.from_numpy((want - s).reshape(E).astype(np.float32))
        run_route(torch.from_numpy(l), 6, bias=bias, score=score, groups=groups, top_groups=max(groups // 2, 1), group_sum=2)


@pytest.mark.parametrize("E", [4, 28, 32, 36, 64, 128, 132, 256])
@pytest.mark.parametrize("how", range(4))
def test_masks(E, how):
    l = logits_of(41, E, "f32", E)
    l[1] = -INF
    l[2, 1:] = -INF
    l[3, ::2] = -INF
    l[6, E // 2:] = -INF
    l[7, :E // 2] = -INF
    l[8, torch.arange(E) % 4 != 1] = -INF
    l[9] = torch.finfo(torch.float32).min
    l[10, 3] = float("nan")
    l[13, E - 1] = INF
    l[14] = float("nan")
    l[37:] = -INF
    top = min(E, 8)
    for bias in (None, torch.zeros(E), torch.where(torch.arange(E) % 3 == 0, -INF, 0.1), torch.full((E,), -INF)):
        run_route(l, top, bias=bias, **CHOICES[how])
        if E % 64 == 0:
            for group_sum in (1, 2):
                run_route(l, top, bias=bias, groups=E // 32, top_groups=E // 64, group_sum=group_sum, **CHOICES[how])
                run_route(l, 3, bias=bias, groups=2, top_groups=1, group_sum=group_sum, **CHOICES[how])


@pytest.mark.parametrize("bias", [INF, 3e38, float("nan")])
def test_biases_without_a_bound(bias):
    b = torch.zeros(64)
    b[[5, 40]] = bias
    run_route(logits_of(30, 64, "f32", 1), 4, bias=b, score="sigmoid")
    run_route(logits_of(30, 64, "f32", 1), 4, bias=b, groups=2, top_groups=1, group_sum=2)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 64, 65, 67, 300, 9000])
@pytest.mark.parametrize("planned", [True, False])
def test_tokens(T, planned):
    l = logits_of(T, 256, "bf16", T)
    run_route(l, 8, score="sigmoid", bias=torch.randn(256, generator=gen(T)) * 0.05, groups=8, top_groups=4, group_sum=2,
              scale=2.5, planned=planned)
    run_route(l[:, :20], 1, normalise=False, planned=planned)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pitch,first", [(80, 0), (80, 4), (80, 8), (80, 3), (78, 0), (77, 1)])
def test_any_alignment_gives_the_same(dtype, pitch, first):
    x = logits_of(50, 64, dtype, pitch)
    big = torch.full((50, pitch + 8), 9.0, dtype=TYPE[dtype], device="cuda").flatten()[: 50 * pitch + 8]
    l = big[first:].as_strided((50, 64), (pitch, 1))
    l.copy_(x)
    experts, weights = torch.empty((50, 8), dtype=torch.int32, device="cuda"), torch.empty((50, 8), device="cuda")
    swg.expert_route_into(experts, weights, l)
    want, w = plain.route(f64(x), None, 8)
    assert np.array_equal(experts.cpu().numpy(), want)
    assert (np.abs(f64(weights) - w) <= plain.route_bound(f64(x), w, 8)).all()


def test_equal_choices_beyond_a_teams_room():
    for E, groups in ((64, 2), (256, 8), (256, 1)):
        l = logits_of(11, E, "f32", E)
        l[[0, 2, 3, 9]] = 0.25
        run_route(l, 8, bias=torch.zeros(E), groups=groups, top_groups=max(groups // 2, 1), group_sum=2)
        run_route(l, 8)


@pytest.mark.parametrize("E", [64, 66, 256, 257, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_of_many_equal_choices_is_apart(E, score):
    """... by less than FP32 shows: one that is better comes first, one that is worse
    is passed over."""
    l = torch.zeros(9, E)
    l[4] = logits_of(1, E, "f32", E)
    for at, by in ((E - 2, 1e-9), (3, 1e-9), (3, -1e-9), (0, -1e-9), (7, -1e-10), (8, 1e-10)):
        bias = torch.zeros(E)
        bias[at] = by
        run_route(l, 8, bias=bias, score=score)
        if E % 64 == 0:
            run_route(l, 8, bias=bias, score=score, groups=2, top_groups=1, group_sum=2)
    bias = torch.zeros(E)
    bias[::2] = -INF
    run_route(l, 8, bias=bias, score=score)
