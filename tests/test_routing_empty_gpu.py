"""Positions are looked at where there is nothing to move, too."""
import pytest
import torch

import swiglu_mlp_gb300 as swg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,D", [(0, 16), (0, 0), (8, 0), (8, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wrong_positions_of_no_rows_or_columns(R, D, dtype):
    z = lambda *s: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    for wrong in (R, -2, 2 ** 31 - 1, None):
        p = torch.full((40, 2), -1, dtype=torch.int32, device="cuda")
        if wrong is not None:
            p[33, 1] = wrong
        calls = [lambda: swg.expert_dispatch_into(z(R, D), z(40, D), p), lambda: swg.expert_combine_into(z(40, D), z(R, D), p),
                 lambda: swg.expert_combine_grad_into(z(R, D), None, z(40, D), None, p),
                 lambda: swg.expert_combine_grad_into(z(R, D), torch.ones(40, 2, device="cuda"), z(40, D), z(R, D), p)]
        for call in calls:
            call()
            assert swg.get_device_error() == (wrong is not None) and swg.get_device_error() == 0
