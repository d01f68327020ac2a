"""Tokens and slots as many as the entry points accept."""
import pytest
import torch

import swiglu_mlp_gb300 as swg

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1024


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 2 ** 30:
        pytest.skip(f"needs {gigabytes} GB of the GPU's memory")


def counts_up(t, first, last, start=0):
    """Whether t[first:last] is start, start + 1, ..."""
    step = 2 ** 27
    for i in range(first, last, step):
        n = min(step, last - i)
        if not torch.equal(t[i:i + n], torch.arange(start + i - first, start + i - first + n, dtype=torch.int32, device="cuda")):
            return False
    return True


@pytest.mark.parametrize("none", [0, 1, 400001])
def test_sort_of_the_most_slots(none):
    """Two experts' slots one after the other, the last `none` without an expert."""
    room(40)
    top, E = 32, 3
    T, half = MOST // top, MOST // 2 + 5
    experts = torch.zeros((T, top), dtype=torch.int32, device="cuda")
    flat = experts.view(-1)
    flat[half:] = 2
    flat[MOST - none:] = -1
    offsets, source, position = plan = swg.expert_plan_alloc(T, E, top)
    for t in plan:
        t.fill_(99)
    swg.expert_sort_into(plan, experts)
    assert swg.get_device_error() == 0
    rows = MOST - none
    assert offsets.tolist() == [0, half, half, rows]
    assert counts_up(source, 0, rows) and counts_up(position.view(-1), 0, rows)
    assert bool((source[rows:] == -1).all()) and bool((position.view(-1)[rows:] == -1).all())


@pytest.mark.parametrize("E", [4, 3])                    # four tokens of a warp, and one
def test_route_of_the_most_tokens(E):
    """Token t's best expert is t % E, but for the last one, which has none."""
    room(60)
    T = MOST
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        logits[e::E, e] = 1.0
    logits[T - 1] = -float("inf")
    experts = torch.full((T, 1), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((T, 1), 7.0, device="cuda")
    swg.expert_route_into(experts, weights, logits)
    assert swg.get_device_error() == 0
    for e in range(E):
        assert bool((experts[e:T - 1:E] == e).all())
    assert experts[-1].item() == -1 and weights[-1].item() == 0
    assert bool((weights[:-1] == 1).all())
