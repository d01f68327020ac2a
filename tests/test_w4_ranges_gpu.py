"""4-bit products by expert whose contraction is split over a cluster: the number of ranges
goes by the chunks that the rows are expected to fill, whichever experts have them."""
import pytest

from test_w4_gpu import run_gemm
from test_w4_gpu import test_swiglu as check_swiglu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [[16] * 4, [64, 0, 0, 0], [0, 31, 33, 2, 0, 30], [100]])
@pytest.mark.parametrize("N", [300, 2000, 6000])         # room for eight ranges, two, one
@pytest.mark.parametrize("K", [200, 600, 1200, 2100])    # one step of the contraction, three, five, nine
def test_ranges_of_groups(rows, N, K):
    run_gemm(rows, N, K, 64, True, "bf16", "f32", alpha=0.5, beta=1.0, seed=N + K)
    run_gemm(rows, N, K, 128, False, "f16", seed=N, before=5, after=3)


@pytest.mark.parametrize("rows", [[40, 0, 9, 31], [0, 0, 64]])
@pytest.mark.parametrize("K", [600, 2100])
def test_swiglu_of_ranges(rows, K):
    check_swiglu(rows, 150, K, 32, True, "f16")
