"""Plans of as many slots as the entry points accept."""
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
