"""The expert-MLP operators beyond 2^31 elements, on several streams and from
several threads, and at the ends of the 4-bit formats' ranges."""
import threading

import numpy as np
import pytest
import torch

import experts_plain as plain
import swiglu_mlp_gb300 as swg
import synth

pytestmark = pytest.mark.gpu

FMT = {"mx": swg.MXFP4, "nv": swg.NVFP4}


def test_grouped_product_beyond_two_giga_elements():
    """A and C of 2.3e9 elements each: sampled rows, the last ones among them."""
    M, K, N, G = 1_130_000, 2048, 2056, 3
    off = torch.tensor([0, 17, 1_100_001, M], dtype=torch.int32)
    A = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for i in range(0, M, 100_000):
        part = A[i:i + 100_000]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    B = synth.normal((G, K, N), synth.generator(2), K ** -0.5).cuda()
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    swg.gemm_grouped_into(C, A, B, off.cuda())
    assert swg.get_device_error() == 0
    for r in (0, 16, 17, 18, 500_000, 1_050_000, 1_100_000, 1_100_001, M - 2, M - 1):
        e = int((off <= r).sum()) - 1
        a, w = plain.f64(A[r:r + 1]), plain.f64(B[e])
        want = a @ w
        tol = plain.fp32_sum_bound(K, np.abs(a) @ np.abs(w)) + plain.ROUND["bf16"] * np.abs(want)
        assert (np.abs(plain.f64(C[r:r + 1]) - want) <= tol).all(), r
    # and the weight gradient over all of them, in one of its columns
    D = C
    W = torch.empty((G, 64, N), dtype=torch.float32, device="cuda")
    swg.gemm_grouped_wgrad_into(W, A[:, :64], D, off.cuda())
    assert swg.get_device_error() == 0
    a, b = int(off[2]), int(off[3])
    want = A[a:b, 7].double() @ D[a:b].double()
    mags = A[a:b, 7].double().abs() @ D[a:b].double().abs()
    assert bool(((W[2, 7].double() - want).abs() <= plain.fp32_sum_bound(b - a, 1.0) * mags + 1e-6).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_conversion_beyond_two_giga_elements(fmt):
    M, K = 560_000, 4096
    X = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for i in range(0, M, 100_000):
        part = X[i:i + 100_000]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    Q, S = swg.mx4_alloc(M, K, FMT[fmt])
    swg.mx4_quantize_into(Q, S, X, FMT[fmt])
    V = torch.empty_like(X)
    swg.mx4_dequantize_into(V, Q, S, FMT[fmt])
    assert swg.get_device_error() == 0
    rows = [0, 127, 128, 524_287, 524_288, M - 1]
    assert np.array_equal(plain.f64(V[rows]), plain.quantised(plain.f64(X[rows]), fmt))


def test_ends_of_the_scales_range():
    """MXFP4: blocks of bfloat16's smallest (subnormal) and largest values;
    NVFP4: blocks below and above what its scales reach."""
    x = torch.tensor([[2.0 ** -133, 3 * 2.0 ** -133, -2.0 ** -130], [2.0 ** -126, 2.0 ** -127, 0.0],
                      [2.0 ** -125, -2.0 ** -126, 2.0 ** -128], [3.38e38, -1.7e38, 1e37]]).bfloat16()
    x = torch.nn.functional.pad(x, (0, 29))
    Q, S = swg.mx4_alloc(4, 32, swg.MXFP4)
    V = torch.empty((4, 32), dtype=torch.float32, device="cuda")
    swg.mx4_quantize_into(Q, S, x.cuda(), swg.MXFP4)
    swg.mx4_dequantize_into(V, Q, S, swg.MXFP4)
    assert np.array_equal(plain.f64(V), plain.quantised(plain.f64(x), "mx"))
    x = torch.tensor([[2.0 ** -13, 2.0 ** -10, -2.0 ** -9], [2700.0, -2688.0, 2500.0], [1e5, -448.0, 6.0]]).bfloat16()
    x = torch.nn.functional.pad(x, (0, 29))
    Q, S = swg.mx4_alloc(3, 32, swg.NVFP4)
    V = torch.empty((3, 32), dtype=torch.float32, device="cuda")
    swg.mx4_quantize_into(Q, S, x.cuda(), swg.NVFP4)
    swg.mx4_dequantize_into(V, Q, S, swg.NVFP4)
    assert np.array_equal(plain.f64(V), plain.quantised(plain.f64(x), "nv"))


def _case(seed):
    g = synth.generator(seed)
    off = torch.tensor([0, 3, 3, 40, 64], dtype=torch.int32).cuda()
    A, B = synth.normal((64, 4096), g).cuda(), synth.normal((4, 4096, 264), g, 0.02).cuda()
    W, SW = swg.mx4_alloc(4 * 264, 4096, swg.MXFP4, groups=4)
    rows = torch.arange(5, dtype=torch.int32).cuda() * 264
    swg.mx4_quantize_into(W, SW, synth.normal((4 * 264, 4096), g, 0.02).cuda(), swg.MXFP4, offsets=rows)
    torch.cuda.synchronize()
    return off, A, B, W.view(4, 264, -1), SW


def _run(case, out, stream):
    off, A, B, W, SW = case
    C, D, G, Q, S = out
    swg.gemm_grouped_into(C, A, B, off, stream=stream)
    swg.mx4_quantize_into(Q, S, A, swg.MXFP4, offsets=off, stream=stream)
    swg.gemm_mx4_into(D, Q, S, W, SW, 4096, swg.MXFP4, offsets=off, stream=stream)
    swg.gemm_grouped_wgrad_into(G, A, C, off, stream=stream)


def _buffers():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    return e(64, 264), e(64, 264), e(4, 4096, 264), *swg.mx4_alloc(64, 4096, swg.MXFP4, groups=4)


@pytest.mark.parametrize("threads", [False, True])
def test_streams_and_threads(threads):
    """Overlapping calls, each stream with its own workspace, give bit for bit
    what the same calls give alone."""
    cases = [_case(100 + i) for i in range(4)]
    want = []
    for c in cases:
        out = _buffers()
        _run(c, out, torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([t.clone() for t in out[:3]])
    streams, bufs = [torch.cuda.Stream() for _ in cases], [_buffers() for _ in cases]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(5):
            _run(cases[i], bufs[i], streams[i])

    if threads:
        ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    else:
        for _ in range(5):
            for i in range(4):
                _run(cases[i], bufs[i], streams[i])
    torch.cuda.synchronize()
    assert swg.get_device_error() == 0
    for w, b in zip(want, bufs):
        for x, y in zip(w, b[:3]):
            assert torch.equal(x, y)


# The last rows that 32 bits can number: 2^31 - 1024 of them, more than the
# tiles of a group could be counted in when rows and tiles were added up.
MOST = 2 ** 31 - 1024


def _last_rows(x, rows):
    g = synth.generator(77)
    part = synth.normal((rows, x.shape[1]), g).cuda()
    x[-rows:] = part
    return part


def test_grouped_product_of_the_most_rows():
    A = torch.zeros((MOST, 8), dtype=torch.bfloat16, device="cuda")
    last = _last_rows(A, 700)
    B = synth.normal((2, 8, 8), synth.generator(78)).cuda()
    C = torch.full((MOST, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    swg.gemm_grouped_into(C, A, B, torch.tensor([0, 5, MOST], dtype=torch.int32).cuda())
    assert swg.get_device_error() == 0
    want = plain.f64(last) @ plain.f64(B[1])
    tol = plain.fp32_sum_bound(8, np.abs(plain.f64(last)) @ np.abs(plain.f64(B[1]))) \
        + plain.ROUND["bf16"] * np.abs(want)
    assert (np.abs(plain.f64(C[-700:]) - want) <= tol).all()
    for i in range(0, MOST - 700, 2 ** 28):
        assert not C[i:min(i + 2 ** 28, MOST - 700)].any()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_conversion_of_the_most_rows(fmt):
    X = torch.zeros((MOST, 8), dtype=torch.bfloat16, device="cuda")
    last = _last_rows(X, 700)
    off = torch.tensor([0, MOST - 100, MOST], dtype=torch.int32).cuda()
    Q, S = swg.mx4_alloc(MOST, 8, FMT[fmt], groups=2)
    swg.mx4_quantize_into(Q, S, X, FMT[fmt], offsets=off)
    X.fill_(7.0)
    swg.mx4_dequantize_into(X, Q, S, FMT[fmt], offsets=off)
    assert swg.get_device_error() == 0
    assert np.array_equal(plain.f64(X[-700:]), plain.quantised(plain.f64(last), fmt))
    for i in range(0, MOST - 700, 2 ** 28):
        assert not X[i:min(i + 2 ** 28, MOST - 700)].any()
