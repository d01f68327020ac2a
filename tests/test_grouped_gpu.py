"""Products grouped by expert with ragged sizes against their 64-bit forms
(experts_plain.py, where the bounds are derived), at the sizes, groups,
strides and values where a tiled kernel can go wrong."""
import numpy as np
import pytest
import torch

import experts_plain as plain
import swiglu_mlp_gb300 as swg
import synth
from helpers import Guarded
from test_experts_host import expert_calls

pytestmark = pytest.mark.gpu

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DTYPES = [("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f32")]
# row counts of the groups: empty first, middle and last; one row; tile edges
RAGGED = [0, 5, 1, 0, 130, 257, 16, 0]


def offsets_of(rows, before=0):
    return np.concatenate([[before], before + np.cumsum(rows)]).astype(np.int32)


def padded(rows, cols, g, dtype, std=1.0, extra=0):
    """rows x cols, in storage with `extra` more 16-byte units per row that hold NaN."""
    ld = -(-cols // 8) * 8 + 8 * extra
    t = torch.full((rows, ld), float("nan"), dtype=dtype)
    t[:, :cols] = synth.normal((rows, cols), g, std, dtype)
    return t.cuda()[:, :cols]


def check(got, want, tol, what):
    got = plain.f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, e.g. {np.argwhere(bad)[:4].tolist()}, " \
        f"got {got[bad][:4]}, want {want[bad][:4]}, bound {tol[bad][:4]}"


def run_gemm(rows, N, K, types, transB=0, alpha=1.0, beta=0.0, extra=0, seed=1, before=0, after=0,
             stream=None):
    g = synth.generator(seed)
    off = offsets_of(rows, before)
    M, G = int(off[-1]) + after, len(rows)
    t_in, t_out = TYPE[types[0]], TYPE[types[1]]
    A = padded(M, K, g, t_in, extra=extra)
    shape = (N, K) if transB else (K, N)
    B = padded(G * shape[0], shape[1], g, t_in, std=0.2, extra=extra).unflatten(0, (G, shape[0]))
    C0 = synth.normal((M, N), g, dtype=torch.float32).to(t_out)
    C = Guarded(M, N, t_out, init=C0)
    swg.gemm_grouped_into(C.view, A, B, torch.from_numpy(off).cuda(), transB=transB, alpha=alpha,
                          beta=beta, stream=stream)
    assert swg.get_device_error(stream) == 0
    want, tol = plain.product(plain.f64(A), plain.f64(B), off, transB, alpha, beta, plain.f64(C0),
                              types[1])
    check(C.cpu("gemm_grouped"), want, tol, f"gemm_grouped {rows} N={N} K={K} {types}")
    return C.view


@pytest.mark.parametrize("types", DTYPES)
@pytest.mark.parametrize("transB", [0, 1])
@pytest.mark.parametrize("N,K", [(264, 136), (33, 77), (8, 520), (640, 64)])
def test_ragged_groups(types, transB, N, K):
    run_gemm(RAGGED, N, K, types, transB, extra=2, seed=N + K)


@pytest.mark.parametrize("rows", [[1], [2], [17], [0], [1, 1, 1], [64, 64], [300], [513, 0, 255],
                                  [0, 0, 0, 9], [7] * 100])
@pytest.mark.parametrize("transB", [0, 1])
def test_group_sizes(rows, transB):
    run_gemm(rows, 200, 320, ("bf16", "bf16"), transB, seed=len(rows))


@pytest.mark.parametrize("K", [1, 8, 15, 63, 64, 65, 129, 0])
def test_contraction_lengths(K):
    run_gemm([3, 40, 0, 129], 72, K, ("bf16", "f32"), 0, seed=K + 5)
    run_gemm([3, 40, 0, 129], 72, K, ("f16", "f16"), 1, seed=K + 6, beta=0.5)


@pytest.mark.parametrize("alpha,beta", [(0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (0.0, 1.0)])
@pytest.mark.parametrize("types", DTYPES)
def test_alpha_beta(types, alpha, beta):
    run_gemm(RAGGED, 104, 200, types, alpha=alpha, beta=beta, seed=11)


def test_rows_outside_the_groups_are_left_alone():
    """Rows before offsets[0] and from offsets[G] on keep their values, and
    NaN in them (and beyond each row's columns) reaches no result."""
    g = synth.generator(21)
    rows, N, K = [20, 0, 150], 96, 72
    off = offsets_of(rows, 7)
    M = int(off[-1]) + 9
    A = padded(M, K, g, torch.bfloat16, extra=1)
    A[:7] = float("nan")
    A[int(off[-1]):] = float("inf")
    B = padded(3 * K, N, g, torch.bfloat16, 0.2).unflatten(0, (3, K))
    B[1] = float("nan")                                  # an empty group's weight
    C0 = synth.normal((M, N), g)
    C = Guarded(M, N, torch.bfloat16, init=C0)
    swg.gemm_grouped_into(C.view, A, B, torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    a, b = plain.f64(A), plain.f64(B)
    a[:7] = 0
    a[int(off[-1]):] = 0
    b[1] = 0
    want, tol = plain.product(a, b, off, 0, 1.0, 0.0, plain.f64(C0), "bf16")
    check(C.cpu(), want, tol, "outside rows")


def test_beta_zero_does_not_read_c():
    rows, N, K = [5, 33], 40, 64
    g = synth.generator(3)
    off = offsets_of(rows)
    A, B = padded(38, K, g, torch.bfloat16), padded(2 * K, N, g, torch.bfloat16).unflatten(0, (2, K))
    C = Guarded(38, N, torch.bfloat16, fill=float("nan"))
    swg.gemm_grouped_into(C.view, A, B, torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    assert torch.isfinite(C.cpu()).all()


def run_wgrad(rows, N, K, types, alpha=1.0, beta=0.0, extra=0, seed=2, before=0, after=0,
              poison=False):
    g = synth.generator(seed)
    off = offsets_of(rows, before)
    M, G = int(off[-1]) + after, len(rows)
    t_in, t_out = TYPE[types[0]], TYPE[types[1]]
    A = padded(M, K, g, t_in, extra=extra)
    D = padded(M, N, g, t_in, std=0.3, extra=extra)
    if poison:                                           # rows of no group
        A[:before] = D[:before] = float("nan")
        A[M - after:] = D[M - after:] = float("inf")
    C0 = synth.normal((G * K, N), g, dtype=torch.float32).to(t_out)
    C = Guarded(G * K, N, t_out, init=C0)
    view = C.view.unflatten(0, (G, K))
    swg.gemm_grouped_wgrad_into(view, A, D, torch.from_numpy(off).cuda(), alpha=alpha, beta=beta)
    assert swg.get_device_error() == 0
    a, d = np.nan_to_num(plain.f64(A), posinf=0), np.nan_to_num(plain.f64(D), posinf=0)
    want, tol = plain.wgrad(a, d, off, alpha, beta, plain.f64(C0).reshape(G, K, N), types[1])
    check(C.cpu("wgrad").unflatten(0, (G, K)), want, tol, f"wgrad {rows} N={N} K={K} {types}")
    return C.view


@pytest.mark.parametrize("types", DTYPES)
@pytest.mark.parametrize("N,K", [(264, 136), (33, 77), (8, 520), (640, 64)])
def test_wgrad_ragged_groups(types, N, K):
    run_wgrad(RAGGED, N, K, types, extra=2, seed=N + K)


@pytest.mark.parametrize("rows", [[1], [0], [15], [16], [17], [63, 64, 65], [0, 0, 700, 0], [3] * 50])
def test_wgrad_group_sizes(rows):
    run_wgrad(rows, 136, 264, ("bf16", "bf16"), seed=len(rows))


@pytest.mark.parametrize("alpha,beta", [(0.5, 0.0), (1.0, 1.0), (-2.0, 0.25)])
@pytest.mark.parametrize("types", DTYPES)
def test_wgrad_alpha_beta(types, alpha, beta):
    run_wgrad(RAGGED, 104, 200, types, alpha, beta, seed=12)


def test_wgrad_neighbours_do_not_leak():
    """Rows that belong to no group hold NaN and infinities; groups end inside
    a block of rows, so a block read whole contains them."""
    run_wgrad([37, 0, 90, 1], 72, 200, ("bf16", "bf16"), before=5, after=70, poison=True)


def test_wgrad_infinity_stays_in_its_group():
    g = synth.generator(4)
    off = offsets_of([30, 34, 20])
    A, D = padded(84, 64, g, torch.bfloat16), padded(84, 40, g, torch.bfloat16)
    A[40] = float("inf")
    C = torch.empty((3, 64, 40), dtype=torch.bfloat16, device="cuda")
    swg.gemm_grouped_wgrad_into(C, A, D, torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    finite = torch.isfinite(C).flatten(1).all(1).tolist()
    assert finite == [True, False, True]


def weights(G, K, N, g):
    return synth.normal((G, K, 2 * N), g, K ** -0.5)


@pytest.mark.parametrize("rows", [[1], [2, 0, 1], RAGGED, [300], [64] * 8])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 136), (72, 520)])
def test_swiglu_grouped(rows, N, K):
    g = synth.generator(N + K)
    off = offsets_of(rows)
    M = int(off[-1])
    A, W = synth.normal((M, K), g), weights(len(rows), K, N, g)
    Y = Guarded(M, N, torch.bfloat16, fill=9.0, ld=N)
    swg.swiglu_grouped_into(Y.view, A.cuda(), W.cuda(), torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    want, tol = plain.swiglu(plain.f64(A), plain.f64(W), off)
    check(Y.cpu("swiglu_grouped"), want, tol, f"swiglu {rows} N={N} K={K}")


@pytest.mark.parametrize("with_y", [True, False])
@pytest.mark.parametrize("rows", [[1], [2, 0, 1], RAGGED, [300]])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 136), (72, 520)])
def test_swiglu_grouped_grad(rows, N, K, with_y):
    g = synth.generator(N + K + 1)
    off = offsets_of(rows)
    M = int(off[-1])
    A, W, dY = synth.normal((M, K), g), weights(len(rows), K, N, g), synth.normal((M, N), g)
    dH = Guarded(M, 2 * N, torch.bfloat16, fill=9.0, ld=2 * N)
    Y = Guarded(M, N, torch.bfloat16, fill=9.0, ld=N)
    swg.swiglu_grouped_grad_into(dH.view, A.cuda(), W.cuda(), dY.cuda(),
                                 torch.from_numpy(off).cuda(), Y=Y.view if with_y else None)
    assert swg.get_device_error() == 0
    want, tol = plain.swiglu_grad(plain.f64(A), plain.f64(W), plain.f64(dY), off)
    check(dH.cpu("dH"), want, tol, f"dH {rows} N={N} K={K}")
    if with_y:
        want, tol = plain.swiglu(plain.f64(A), plain.f64(W), off)
        check(Y.cpu("Y"), want, tol, "Y of the gradient")
    else:
        assert (Y.cpu("Y") == 9.0).all()


def test_swiglu_grad_saturated_gates():
    """Gates of several hundred: sigmoid is 0 or 1, nothing becomes NaN."""
    g = synth.generator(8)
    off = offsets_of([20, 44])
    A, W = synth.normal((64, 64), g), synth.normal((2, 64, 80), g, 16.0)
    dY = synth.normal((64, 40), g)
    dH = Guarded(64, 80, torch.bfloat16, ld=80)
    swg.swiglu_grouped_grad_into(dH.view, A.cuda(), W.cuda(), dY.cuda(), torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    want, tol = plain.swiglu_grad(plain.f64(A), plain.f64(W), plain.f64(dY), off)
    check(dH.cpu(), want, tol, "saturated")


def test_expert_mlp_gradients_match_autograd():
    """The whole backward pass of an expert MLP from the three products,
    against autograd in 64 bits; each stage's inputs are the rounded ones."""
    g = synth.generator(31)
    rows, K, N = [37, 0, 130, 4], 136, 72
    off = offsets_of(rows)
    M, G = int(off[-1]), len(rows)
    X, W, Wd = synth.normal((M, K), g), weights(G, K, N, g), synth.normal((G, N, K), g, N ** -0.5)
    dO = synth.normal((M, K), g)
    o = torch.from_numpy(off).cuda()
    Xc, Wc, Wdc, dOc = X.cuda(), W.cuda(), Wd.cuda(), dO.cuda()
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dY = swg.gemm_grouped_into(e(M, N), dOc, Wdc, o, transB=1)
    Y = e(M, N)
    dH = swg.swiglu_grouped_grad_into(e(M, 2 * N), Xc, Wc, dY, o, Y=Y)
    dX = swg.gemm_grouped_into(e(M, K), dH, Wc, o, transB=1)
    dW = swg.gemm_grouped_wgrad_into(e(G, K, 2 * N), Xc, dH, o)
    dWd = swg.gemm_grouped_wgrad_into(e(G, N, K), Y, dOc, o)
    assert swg.get_device_error() == 0

    x, w, wd = (t.double().requires_grad_() for t in (X, W, Wd))
    outs = []
    for i, (a, b) in enumerate(plain.groups(off)):
        h = x[a:b] @ w[i]
        outs.append((torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2]) @ wd[i])
    torch.cat(outs).backward(dO.double())
    # three bf16 roundings on the way (dY, dH or Y, the result): 3 * 2^-9 of
    # the norm, and as much again for their growth through two products
    for got, ref in ((dX, x.grad), (dW, w.grad), (dWd, wd.grad)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        assert err < 6 * 2.0 ** -9, float(err)


def test_gradient_formula_against_differences():
    """The formula of swiglu_grouped_grad against central differences of the
    forward formula, in 64 bits: the truncation error is O(h^2) ~ 1e-8."""
    r = np.random.RandomState(5)
    A, W = r.randn(6, 10), r.randn(2, 10, 8) * 0.3
    dY, off = r.randn(6, 4), np.array([0, 2, 6])
    dH, _ = plain.swiglu_grad(A, W, dY, off)
    dA = np.zeros_like(A)
    for g, (a, b) in enumerate(plain.groups(off)):
        dA[a:b] = dH[a:b] @ W[g].T
    h = 1e-4
    for i in range(6):
        for k in range(10):
            up, down = A.copy(), A.copy()
            up[i, k] += h
            down[i, k] -= h
            num = ((plain.swiglu(up, W, off)[0] - plain.swiglu(down, W, off)[0]) * dY).sum() / (2 * h)
            assert abs(num - dA[i, k]) < 1e-6


@pytest.mark.parametrize("off", [[0, 5, 3, 40], [-4, 10, 20, 40], [0, 10, 90, 40]])
def test_bad_offsets_are_reported_and_stay_in_bounds(off):
    """Offsets out of order or out of range are clamped in the kernels: the
    guard bands stay whole and the error word says so."""
    g = synth.generator(6)
    o = torch.tensor(off, dtype=torch.int32).cuda()
    A, B = padded(40, 64, g, torch.bfloat16), padded(3 * 64, 72, g, torch.bfloat16).unflatten(0, (3, 64))
    C = Guarded(40, 72, torch.bfloat16)
    swg.gemm_grouped_into(C.view, A, B, o)
    assert swg.get_device_error() == 1
    C.check("bad offsets")
    D = padded(40, 72, g, torch.bfloat16)
    W = Guarded(3 * 64, 72, torch.bfloat16)
    swg.gemm_grouped_wgrad_into(W.view.unflatten(0, (3, 64)), A, D, o)
    assert swg.get_device_error() == 1
    W.check("bad offsets")
    assert swg.get_device_error() == 0


def test_offsets_written_on_the_same_stream():
    """The offsets are read on the stream: a kernel queued before the call
    may write them."""
    s = torch.cuda.Stream()
    g = synth.generator(9)
    rows = [40, 3, 0, 85]
    off = offsets_of(rows)
    A, B = padded(128, 128, g, torch.bfloat16), padded(4 * 128, 256, g, torch.bfloat16).unflatten(0, (4, 128))
    C = Guarded(128, 256, torch.bfloat16)
    o = torch.zeros(5, dtype=torch.int32, device="cuda")
    src = torch.from_numpy(off).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        o.copy_(src)
        swg.gemm_grouped_into(C.view, A, B, o)
    assert swg.get_device_error(s) == 0
    want, tol = plain.product(plain.f64(A), plain.f64(B), off, 0, 1.0, 0.0, np.zeros((128, 256)), "bf16")
    check(C.cpu(), want, tol, "own stream")


def test_graph_capture_and_repeatability():
    """Captured and replayed with other offsets, bit for bit as called alone."""
    g = synth.generator(10)
    A, B = padded(200, 512, g, torch.bfloat16), padded(4 * 512, 264, g, torch.bfloat16).unflatten(0, (4, 512))
    D = padded(200, 264, g, torch.bfloat16)
    o = torch.from_numpy(offsets_of([50, 50, 50, 50])).cuda()
    C = torch.empty((200, 264), dtype=torch.bfloat16, device="cuda")
    W = torch.empty((4, 512, 264), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()

    def both():
        swg.gemm_grouped_into(C, A, B, o)
        swg.gemm_grouped_wgrad_into(W, A, D, o)

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    o.copy_(torch.from_numpy(offsets_of([0, 150, 1, 49])))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    c, w = C.clone(), W.clone()
    for _ in range(3):
        both()
        torch.cuda.synchronize()
        assert torch.equal(c, C) and torch.equal(w, W)
    assert swg.get_device_error() == 0


# Few tiles and a long contraction: cut into ranges whose FP32 partials a second
# kernel adds in order.  (Exact for beta, alpha, every epilogue and odd columns.)
@pytest.mark.parametrize("rows,N,K,types,beta", [([1], 264, 4096, ("bf16", "bf16"), 0.0),
                                                 ([3, 0, 20], 33, 2048, ("f16", "f32"), 0.5),
                                                 ([200], 72, 3001, ("f16", "f16"), 1.0),
                                                 ([0, 300, 1], 520, 1536, ("bf16", "bf16"), 0.0)])
@pytest.mark.parametrize("transB", [0, 1])
def test_long_contractions(rows, N, K, types, beta, transB):
    run_gemm(rows, N, K, types, transB, alpha=0.5, beta=beta, before=3, after=4)


@pytest.mark.parametrize("rows", [[1], [2, 0, 5], [100, 90]])
def test_swiglu_long_contractions(rows):
    N, K = 40, 4096
    g = synth.generator(sum(rows))
    off = offsets_of(rows)
    M = int(off[-1])
    A, W, dY = synth.normal((M, K), g), weights(len(rows), K, N, g), synth.normal((M, N), g)
    Y, Y2 = (Guarded(M, N, torch.bfloat16, fill=9.0, ld=N) for _ in range(2))
    dH = Guarded(M, 2 * N, torch.bfloat16, fill=9.0, ld=2 * N)
    o = torch.from_numpy(off).cuda()
    swg.swiglu_grouped_into(Y.view, A.cuda(), W.cuda(), o)
    swg.swiglu_grouped_grad_into(dH.view, A.cuda(), W.cuda(), dY.cuda(), o, Y=Y2.view)
    assert swg.get_device_error() == 0
    want, tol = plain.swiglu(plain.f64(A), plain.f64(W), off)
    check(Y.cpu("Y"), want, tol, "Y")
    check(Y2.cpu("Y"), want, tol, "Y of the gradient")
    want, tol = plain.swiglu_grad(plain.f64(A), plain.f64(W), plain.f64(dY), off)
    check(dH.cpu("dH"), want, tol, "dH")


@pytest.mark.parametrize("rows,N,K,types,beta", [([3000], 72, 264, ("bf16", "bf16"), 0.0),
                                                 ([2500, 0, 5000], 33, 77, ("f16", "f32"), 0.5),
                                                 ([1, 4001], 8, 16, ("f16", "f16"), 1.0)])
def test_wgrad_long_groups(rows, N, K, types, beta):
    run_wgrad(rows, N, K, types, alpha=0.5, beta=beta, before=5, after=70, poison=True)


def test_split_calls_in_a_graph_need_their_workspace_first():
    """A call that would allocate while its stream is captured is refused and
    launches nothing; after the same call outside, it is captured."""
    g = synth.generator(1)
    A, B = padded(2, 4096, g, torch.bfloat16), padded(4096, 520, g, torch.bfloat16)
    C = torch.zeros((2, 520), dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, 2], dtype=torch.int32).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        C.add_(0)
        with pytest.raises(swg.SwgError) as e:
            swg.gemm_grouped_into(C, A, B.unsqueeze(0), o)
        assert e.value.status == 3
    with torch.cuda.stream(s):
        swg.gemm_grouped_into(C, A, B.unsqueeze(0), o)
    s.synchronize()
    first = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        swg.gemm_grouped_into(C, A, B.unsqueeze(0), o)
    C.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, first) and swg.get_device_error() == 0


@pytest.mark.parametrize("M", [1, 64, 65, 144, 145])
@pytest.mark.parametrize("G", [1, 2, 31, 32, 33, 96, 127, 128, 129, 600])
def test_few_rows_over_many_groups(M, G):
    """Most groups empty, the rows anywhere among them, the outer groups too."""
    r = np.random.default_rng(G * 1000 + M)
    rows = np.bincount(r.integers(0, G, M - M // 2), minlength=G) + \
        np.bincount(r.choice([0, G // 2, G - 1], M // 2), minlength=G)
    run_gemm([int(n) for n in rows], 40, 72, ("bf16", "bf16"), G % 2, seed=G)


@pytest.mark.parametrize("M", [50, 140, 200])
@pytest.mark.parametrize("G", [5, 40, 127, 130])
def test_bad_offsets_run_the_clamped_groups(M, G):
    """What runs is the groups that the documented clamping leaves."""
    r = np.random.default_rng(G * 1000 + M)
    off = np.sort(r.integers(0, M + 1, G + 1))
    off[[0, -1]] = 0, M
    at = r.choice(G + 1, 4)
    off[at] = [off[at[0]] - 30, -7, M + 9, off[at[3]] // 2]
    off[1] = max(off[1], 1)
    off[2] = 0                                        # at least one is out of order
    clamped = np.maximum.accumulate(np.clip(off, 0, M))
    g = synth.generator(G)
    A, B = padded(M, 72, g, torch.bfloat16), padded(G * 72, 40, g, torch.bfloat16).unflatten(0, (G, 72))
    C = Guarded(M, 40, torch.bfloat16, init=torch.zeros((M, 40), dtype=torch.bfloat16))
    swg.gemm_grouped_into(C.view, A, B, torch.from_numpy(off.astype(np.int32)).cuda())
    assert swg.get_device_error() == 1
    want, tol = plain.product(plain.f64(A), plain.f64(B), clamped, 0, 1.0, 0.0, np.zeros((M, 40)), "bf16")
    check(C.cpu("clamped groups"), want, tol, f"clamped groups {M} {G}")


# Several tiles for every pair of CTAs, of all widths.
MANY_TILES = [0, 300, 256, 161, 1000, 193, 0, 33, 900, 160]


@pytest.mark.parametrize("types,beta", [(("bf16", "bf16"), 0.0), (("f16", "f32"), 0.5)])
@pytest.mark.parametrize("N,K", [(5000, 40), (4600, 328)])
def test_many_tiles(types, beta, N, K):
    run_gemm(MANY_TILES, N, K, types, 1, 1.0, beta, seed=K)


@pytest.mark.parametrize("N,K", [(2504, 40), (2312, 328)])
def test_swiglu_many_tiles(N, K):
    test_swiglu_grouped(MANY_TILES, N, K)
    test_swiglu_grouped_grad(MANY_TILES, N, K, True)


@pytest.mark.parametrize("rows", [[1], [200]])
def test_sixteen_ranges(rows):
    run_gemm(rows, 136, 16384, ("bf16", "bf16"), 1)


def test_wgrad_sixteen_ranges():
    run_wgrad([20011], 72, 136, ("f16", "f32"))


@pytest.mark.parametrize("off", [[0, 50, 30], [20, 70, 41, 3], [-5, 30, 12, 50, 49]])
def test_bad_offsets_of_long_contractions(off):
    """Cut into ranges of K or not, what runs is the groups that the clamping
    leaves: up to the largest offset, not to the last."""
    M, N, K, G = 50, 72, 4096, len(off) - 1
    off = np.array(off)
    clamped = np.maximum.accumulate(np.clip(off, 0, M))
    g = synth.generator(G)
    A, B = padded(M, K, g, torch.bfloat16), padded(G * K, N, g, torch.bfloat16, K ** -0.5).unflatten(0, (G, K))
    C0 = synth.normal((M, N), g)
    C = Guarded(M, N, torch.bfloat16, init=C0)
    o = torch.from_numpy(off.astype(np.int32)).cuda()
    before = swg.launch_count()
    swg.gemm_grouped_into(C.view, A, B, o)
    assert swg.launch_count() == before + 2              # a product and a sum
    assert swg.get_device_error() == 1
    want, tol = plain.product(plain.f64(A), plain.f64(B), clamped, 0, 1.0, 0.0, plain.f64(C0), "bf16")
    check(C.cpu("clamped groups"), want, tol, f"clamped groups {off}")
    Y = torch.full((M, N // 2 // 8 * 8), 9.0, dtype=torch.bfloat16, device="cuda")
    W = B[:, :, :2 * Y.shape[1]].contiguous()
    swg.swiglu_grouped_into(Y, A.contiguous(), W, o)
    assert swg.get_device_error() == 1
    want, tol = plain.swiglu(plain.f64(A), plain.f64(W), clamped)
    rows = slice(clamped[0], clamped[-1])
    check(Y.cpu()[rows], want[rows], tol[rows], f"clamped groups {off}")
    assert (Y[:clamped[0]] == 9.0).all() and (Y[clamped[-1]:] == 9.0).all()


@pytest.mark.parametrize("i", range(8))
def test_each_tensor_has_to_be_on_the_gpu(i):
    f, tensors, rest = expert_calls()[i]
    there = {n: t.cuda() for n, t in tensors.items()}
    f(**there, **rest)
    assert swg.get_device_error() == 0
    before = swg.launch_count()
    for n, t in tensors.items():
        with pytest.raises(swg.SwgError, match="current CUDA device"):
            f(**dict(there, **{n: t}), **rest)
    assert swg.launch_count() == before


@pytest.mark.parametrize("rows", [[1], [3, 0, 70]])
@pytest.mark.parametrize("types", DTYPES)
def test_matrices_of_one_row(rows, types):
    """Contractions of length one, and single columns of a transposed weight and
    of a gradient: torch gives a lone row any stride."""
    run_gemm(rows, 21, 1, types, 0, beta=0.5, seed=1)
    run_gemm(rows, 1, 21, types, 1, seed=2)
    run_wgrad(rows, 21, 1, types, beta=0.5, seed=3)
    g = synth.generator(4)
    A, B = synth.normal((40, 1), g).cuda().t(), synth.normal((1, 40, 24), g).cuda()
    assert A.stride() == (1, 1)
    C = torch.empty((24, 1), dtype=torch.bfloat16, device="cuda").t()
    swg.gemm_grouped_into(C, A, B, torch.tensor([0, 1], dtype=torch.int32).cuda())
    assert swg.get_device_error() == 0
    want, tol = plain.product(plain.f64(A), plain.f64(B), [0, 1], 0, 1.0, 0.0, np.zeros((1, 24)), "bf16")
    check(C.cpu(), want, tol, "one row")


@pytest.mark.parametrize("N", [1, 7, 21, 40, 257])
@pytest.mark.parametrize("K", [40, 4096])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_lone_row_ends_where_its_columns_do(N, K, out):
    """The result of one row, in storage of N elements: nothing behind them is
    written, whatever row stride it is taken with."""
    g = synth.generator(N)
    A, B = padded(1, K, g, torch.bfloat16), padded(K, N, g, torch.bfloat16, K ** -0.5)
    D = padded(1, N, g, torch.bfloat16)
    o = torch.tensor([0, 1], dtype=torch.int32).cuda()
    store = torch.full((N + 64,), 7.0, dtype=TYPE[out], device="cuda")
    C = store[:N].view(1, N)
    swg.gemm_grouped_into(C, A, B.unsqueeze(0), o)
    want, tol = plain.product(plain.f64(A), plain.f64(B)[None], [0, 1], 0, 1.0, 0.0, np.zeros((1, N)), out)
    check(C.cpu(), want, tol, "lone row")
    assert (store[N:] == 7.0).all()
    swg.gemm_grouped_wgrad_into(C, A[:, :1], D, o)
    want, tol = plain.wgrad(plain.f64(A)[:, :1], plain.f64(D), [0, 1], 1.0, 0.0, np.zeros((1, 1, N)), out)
    check(C.cpu()[None], want, tol, "lone row of a gradient")
    assert (store[N:] == 7.0).all()
    Q, S = swg.mx4_alloc(1, N, swg.NVFP4)
    swg.mx4_quantize_into(Q, S, D, swg.NVFP4)
    swg.mx4_dequantize_into(C, Q, S, swg.NVFP4)
    assert np.array_equal(plain.f64(C), plain.quantised(plain.f64(D), "nv"))
    assert (store[N:] == 7.0).all() and swg.get_device_error() == 0
