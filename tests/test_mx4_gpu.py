"""Microscaled 4-bit floating point against its 64-bit definition
(experts_plain.py): the conversions bit for bit, the products within the FP32
bound derived there."""
import numpy as np
import pytest
import torch

import experts_plain as plain
import swiglu_mlp_gb300 as swg
import synth
from helpers import Guarded
from test_grouped_gpu import RAGGED, check, offsets_of

pytestmark = pytest.mark.gpu

FMT = {"mx": swg.MXFP4, "nv": swg.NVFP4}
TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def storage(x, extra=0):
    """x in rows that are a multiple of 16 bytes, NaN in what is left over."""
    unit = 16 // x.element_size()
    t = torch.full((x.shape[0], -(-x.shape[1] // unit) * unit + extra * unit), float("nan"), dtype=x.dtype)
    t[:, :x.shape[1]] = x
    return t.cuda()[:, :x.shape[1]]


def quantise(x, fmt, off=None, scale=1.0, extra=0):
    """Q and S (both guarded against writes past their ends) of a CPU matrix."""
    M, K = x.shape
    G = 1 if off is None else len(off) - 1
    Q = torch.full((M + 2, -(-K // 32) * 16 + 16), 0xA5, dtype=torch.uint8, device="cuda")
    n = swg.mx4_scale_bytes(FMT[fmt], G, M, K)
    S = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    o = None if off is None else torch.from_numpy(off).cuda()
    q = Q[1:-1, :-(-K // 32) * 16]
    swg.mx4_quantize_into(q, S[:n], storage(x, extra), FMT[fmt], scale=scale, offsets=o)
    assert swg.get_device_error() == 0
    assert (Q[0] == 0xA5).all() and (Q[-1] == 0xA5).all() and (Q[:, -(-K // 32) * 16:] == 0xA5).all()
    assert (S[n:] == 0xA5).all()
    return q, S[:n]


def outliers(M, K, g, dtype):
    x = synth.normal((M, K), g, dtype=torch.float32)
    x[:, ::37] *= 30.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (3, 17), (5, 48), (127, 100), (128, 256),
                                 (129, 1000), (300, 4096), (1, 4105)])
def test_codes_and_scales_bit_for_bit(fmt, dtype, M, K):
    x = outliers(M, K, synth.generator(M + K), TYPE[dtype])
    q, s = quantise(x, fmt, extra=1)
    x64 = plain.f64(x)
    v = plain.quantised(x64, fmt)
    # codes carry x's sign (-0 for what rounds to zero from below)
    want_q, want_s = plain.pack(np.copysign(v, x64), fmt, plain.block_scales(x64, fmt), [M])
    assert np.array_equal(s.cpu().numpy()[:want_s.size], want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    back = Guarded(M, K, torch.bfloat16)
    swg.mx4_dequantize_into(back.view, q, s, FMT[fmt])
    assert swg.get_device_error() == 0
    assert np.array_equal(plain.f64(back.cpu("dequantize")), v)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_every_tie_and_edge(fmt):
    """Values halfway between codes, at and beyond the largest, zeros of both
    signs, for scales over the whole range of the format."""
    b = plain.BLOCK[fmt]
    rows = []
    exps = range(-100, 100, 7) if fmt == "mx" else range(-12, 9)
    for e in exps:
        block = np.zeros(b)
        block[:12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5, -0.0, .1]
        rows.append(block * 2.0 ** e)
        rows.append(np.where(np.arange(b) == 0, 7.9, block) * 2.0 ** e)
        rows.append(np.where(np.arange(b) == 0, 6.5, -block) * 2.0 ** e)
    rows.append(np.zeros(b))
    x = torch.from_numpy(np.stack(rows)).float().bfloat16()
    q, s = quantise(x, fmt)
    out = torch.empty((len(rows), b), dtype=torch.float32, device="cuda")
    swg.mx4_dequantize_into(out, q, s, FMT[fmt])
    assert np.array_equal(plain.f64(out), plain.quantised(plain.f64(x), fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_f32_input_and_scale_factor(fmt):
    """FP32 inputs, times a factor.  MXFP4's scale is a power of two, so the
    values are exact; NVFP4 divides in FP32, which may choose either
    neighbour where the exact quotient is within 1e-6 of a tie."""
    x = synth.normal((40, 500), synth.generator(4), dtype=torch.float32) * 3.0
    q, s = quantise(x, fmt, scale=0.25)
    out = torch.empty((40, 500), dtype=torch.float32, device="cuda")
    swg.mx4_dequantize_into(out, q, s, FMT[fmt], scale=4.0)
    x64 = plain.f64(x) * 0.25
    got = plain.f64(out)
    lo, hi = (4.0 * plain.quantised(x64, fmt) if fmt == "mx" else
              4.0 * plain.e2m1_round(x64 * f / np.repeat(plain.block_scales(x64, fmt), 16, 1)[:, :500])
              * np.repeat(plain.block_scales(x64, fmt), 16, 1)[:, :500] for f in (1 - 1e-6, 1 + 1e-6))
    assert ((got == lo) | (got == hi)).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_and_infinity_blocks(fmt):
    x = synth.normal((4, 128), synth.generator(1))
    x[1, 40] = float("nan")
    x[2, 100] = float("-inf")
    q, s = quantise(x, fmt)
    out = torch.empty((4, 128), dtype=torch.bfloat16, device="cuda")
    swg.mx4_dequantize_into(out, q, s, FMT[fmt])
    want = plain.quantised(plain.f64(x), fmt)
    assert np.array_equal(plain.f64(out), want, equal_nan=True)
    assert np.isnan(want).sum() == 2 * plain.BLOCK[fmt]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows", [RAGGED, [1, 127, 128, 129], [0, 0, 3]])
def test_grouped_scale_tiles(fmt, rows):
    """Each group's scales begin a new row of tiles; rows of no group are
    left alone."""
    g = synth.generator(sum(rows))
    off = offsets_of(rows, 6)
    M, K = int(off[-1]) + 5, 328
    x = outliers(M, K, g, torch.bfloat16)
    q, s = quantise(x, fmt, off)
    x64 = plain.f64(x)[6:off[-1]]
    v = plain.quantised(x64, fmt)
    want_q, want_s = plain.pack(np.copysign(v, x64), fmt, plain.block_scales(x64, fmt), rows)
    q = q.cpu().numpy()
    assert np.array_equal(q[6:off[-1]], want_q)
    assert (q[:6] == 0xA5).all() and (q[off[-1]:] == 0xA5).all()
    assert np.array_equal(s.cpu().numpy()[:want_s.size], want_s)
    out = torch.full((M, K), 9.0, dtype=torch.bfloat16, device="cuda")
    swg.mx4_dequantize_into(out, torch.from_numpy(q).cuda(), s, FMT[fmt], offsets=torch.from_numpy(off).cuda())
    assert np.array_equal(plain.f64(out)[6:off[-1]], v)
    assert (out[:6] == 9.0).all() and (out[off[-1]:] == 9.0).all()


def weight(G, N, K, fmt, g, std=0.3):
    """[G, N, K] values on the grid, their codes and scale tiles (made on the CPU)."""
    x = plain.f64(synth.normal((G * N, K), g, std))
    v = plain.quantised(x, fmt)
    q, s = plain.pack(v, fmt, plain.block_scales(x, fmt), [N] * G)
    return v.reshape(G, N, K), torch.from_numpy(q).cuda().unflatten(0, (G, N)), torch.from_numpy(s).cuda()


def run_product(rows, N, K, fmt, out="bf16", alpha=1.0, beta=0.0, seed=1, dense=False):
    g = synth.generator(seed)
    off = None if dense else offsets_of(rows)
    M = sum(rows)
    x = outliers(M, K, g, torch.bfloat16)
    W, Wq, Ws = weight(len(rows), N, K, fmt, g)
    q, s = quantise(x, fmt, off)
    C0 = synth.normal((M, N), g, dtype=torch.float32).to(TYPE[out])
    C = Guarded(M, N, TYPE[out], init=C0)
    o = None if dense else torch.from_numpy(off).cuda()
    swg.gemm_mx4_into(C.view, q.contiguous(), s, Wq[0] if dense else Wq, Ws, K, FMT[fmt], alpha=alpha,
                      beta=beta, offsets=o)
    assert swg.get_device_error() == 0
    a = plain.quantised(plain.f64(x), fmt)
    want, tol = plain.product(a, W, offsets_of(rows), 1, alpha, beta, plain.f64(C0), out)
    check(C.cpu("gemm_mx4"), want, tol, f"gemm_mx4 {fmt} {rows} N={N} K={K} {out}")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (1, 300, 4096), (16, 64, 64), (33, 257, 1000), (128, 128, 32),
                                   (200, 520, 136), (257, 96, 520), (5, 7, 1), (400, 300, 17),
                                   (2, 264, 8192), (130, 40, 6001)])
def test_dense_product(fmt, M, N, K):
    run_product([M], N, K, fmt, dense=True, seed=M + N + K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows", [RAGGED, [1, 0, 1], [200, 64, 65], [130] * 3])
@pytest.mark.parametrize("N,K", [(264, 320), (40, 1032)])
def test_grouped_product(fmt, rows, N, K):
    run_product(rows, N, K, fmt, seed=N)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("alpha,beta", [(0.5, 0.0), (1.0, 1.0), (-0.25, 2.0)])
def test_product_alpha_beta(fmt, out, alpha, beta):
    run_product([40, 3, 90], 104, 200, fmt, out, alpha, beta)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows,dense", [([1], True), ([200], True), (RAGGED, False), ([1, 0, 1, 64], False)])
@pytest.mark.parametrize("N,K", [(8, 32), (136, 328), (264, 1000)])
def test_swiglu(fmt, rows, dense, N, K):
    g = synth.generator(N + K)
    off = offsets_of(rows)
    M, alpha = sum(rows), 0.25
    x = outliers(M, K, g, torch.bfloat16)
    W, Wq, Ws = weight(len(rows), 2 * N, K, fmt, g)
    q, s = quantise(x, fmt, None if dense else off)
    Y = Guarded(M, N, torch.bfloat16, fill=9.0, ld=N)
    swg.swiglu_mx4_into(Y.view, q.contiguous(), s, Wq[0] if dense else Wq, Ws, K, FMT[fmt], alpha=alpha,
                        offsets=None if dense else torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    a = plain.quantised(plain.f64(x), fmt)
    want, tol = plain.swiglu(a, W.transpose(0, 2, 1), off, alpha)
    check(Y.cpu("swiglu_mx4"), want, tol, f"swiglu_mx4 {fmt} {rows}")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_nan_rows_stay_in_their_rows(fmt):
    """A NaN activation gives a NaN row of the product and no other."""
    g = synth.generator(2)
    x = synth.normal((70, 256), g)
    x[33, 200] = float("nan")
    _, Wq, Ws = weight(1, 136, 256, fmt, g)
    q, s = quantise(x, fmt)
    C = torch.zeros((70, 136), dtype=torch.bfloat16, device="cuda")
    swg.gemm_mx4_into(C, q.contiguous(), s, Wq[0], Ws, 256, FMT[fmt])
    assert swg.get_device_error() == 0
    bad = torch.isnan(C).cpu()
    assert bad[33].all() and bad.sum() == 136


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_products_repeat_bit_for_bit_and_in_graphs(fmt):
    g = synth.generator(3)
    x = synth.normal((40, 2048), g)
    _, Wq, Ws = weight(1, 520, 2048, fmt, g)
    X = x.cuda()
    Q, S = swg.mx4_alloc(40, 2048, FMT[fmt])
    C = torch.empty((40, 520), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()

    def call():
        swg.mx4_quantize_into(Q, S, X, FMT[fmt])
        swg.gemm_mx4_into(C, Q, S, Wq[0], Ws, 2048, FMT[fmt])

    with torch.cuda.stream(s):
        call()
    s.synchronize()
    first = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for _ in range(3):
        C.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, first)
    assert swg.get_device_error() == 0


# Several tiles for every pair of CTAs, of all widths and in both accumulators.
MANY_TILES = [0, 300, 256, 161, 1000, 193, 0, 33, 900, 160]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("out,beta", [("bf16", 0.0), ("f32", 0.5)])
@pytest.mark.parametrize("N,K", [(5000, 40), (4600, 584)])
def test_many_tiles(fmt, out, beta, N, K):
    run_product(MANY_TILES, N, K, fmt, out, 1.0, beta, seed=K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("N,K", [(2504, 40), (2312, 584)])
def test_swiglu_many_tiles(fmt, N, K):
    test_swiglu(fmt, MANY_TILES, False, N, K)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", [(2500, 2600, 72), (1500, 4104, 520), (770, 7700, 264)])
def test_dense_many_tiles(fmt, M, N, K):
    run_product([M], N, K, fmt, dense=True, seed=M)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("G", [36, 37, 38, 39, 40, 128, 505, 512, 1024])
@pytest.mark.parametrize("M", [40, 700])
def test_many_groups(fmt, G, M):
    """What the table of groups takes of shared memory the ring does without."""
    r = np.random.default_rng(G + M)
    rows = np.bincount(r.integers(0, G, M), minlength=G)
    rows[G // 3] += M
    run_product([int(n) for n in rows], 40, 600, fmt, seed=G)


# many groups of few rows, and among them some of several tiles
SKEWED = {
    "few": [0, 1, 5, 2, 0, 4, 31, 32, 33, 3, 0, 64, 1, 8, 0, 0, 7, 12],
    "one large": [0] * 40 + [300] + [1, 0, 2] * 20 + [129],
    "300 groups": [int(n) for n in np.random.default_rng(5).integers(0, 4, 300)],
    "1024 groups": [int(n) for n in np.random.default_rng(6).integers(0, 3, 1023)] + [260],
}


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows", SKEWED)
def test_scale_tiles_of_few_rows(fmt, rows):
    test_grouped_scale_tiles(fmt, SKEWED[rows])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("G,M", [(5, 700), (60, 200), (300, 500)])
def test_bad_offsets_of_a_conversion(fmt, G, M):
    """The rows of the clamped groups are converted and no others, and the
    error word says so."""
    r = np.random.default_rng(G)
    off = np.sort(r.integers(0, M + 1, G + 1))
    off[[0, -1]] = 0, M
    off[G // 2], off[1], off[2] = M + 5, max(int(off[1]), 1), -3
    x = outliers(M, 200, synth.generator(M), torch.bfloat16)
    clamped = np.maximum.accumulate(np.clip(off, 0, M))
    rows = [int(n) for n in np.diff(clamped)]
    q, s = swg.mx4_alloc(M, 200, FMT[fmt], groups=G)
    swg.mx4_quantize_into(q, s, x.cuda(), FMT[fmt], offsets=torch.from_numpy(off.astype(np.int32)).cuda())
    assert swg.get_device_error() == 1
    x64 = plain.f64(x)
    v = plain.quantised(x64, fmt)
    want_q, want_s = plain.pack(np.copysign(v, x64), fmt, plain.block_scales(x64, fmt), rows)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy()[:want_s.size], want_s)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,G,K", [(20, 64, 200), (3, 300, 8192)])
def test_bad_offsets_behind_the_rows(fmt, M, G, K):
    """An offset out of order among the empty groups behind all rows is reported too."""
    off = np.minimum(np.arange(G + 1), M)
    off[G * 2 // 3] = 1
    x = outliers(M, K, synth.generator(M), torch.bfloat16).cuda()
    o = torch.from_numpy(off.astype(np.int32)).cuda()
    q, s = swg.mx4_alloc(M, K, FMT[fmt], groups=G)
    swg.mx4_quantize_into(q, s, x, FMT[fmt], offsets=o)
    assert swg.get_device_error() == 1
    swg.mx4_dequantize_into(x, q, s, FMT[fmt], offsets=o)
    assert swg.get_device_error() == 1


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("rows", [[1], [5, 0, 3]])
def test_products_over_no_columns(fmt, rows):
    M, G, N = sum(rows), len(rows), 16
    off = torch.from_numpy(offsets_of(rows)).cuda()
    q, s = swg.mx4_alloc(M, 0, FMT[fmt], groups=G)
    w, sw = swg.mx4_alloc(G * 2 * N, 0, FMT[fmt], groups=G)
    swg.mx4_quantize_into(q, s, torch.empty((M, 0), dtype=torch.bfloat16, device="cuda"), FMT[fmt], offsets=off)
    Y = torch.full((M, N), 9.0, dtype=torch.bfloat16, device="cuda")
    swg.swiglu_mx4_into(Y, q, s, w.view(G, 2 * N, 0), sw, 0, FMT[fmt], offsets=off)
    assert not Y.any()
    C = torch.full((M, 2 * N), 9.0, dtype=torch.bfloat16, device="cuda")
    swg.gemm_mx4_into(C, q, s, w.view(G, 2 * N, 0), sw, 0, FMT[fmt], beta=0.5, offsets=off)
    assert (C == 4.5).all() and swg.get_device_error() == 0


def e4m3_scales():
    """Every scale of NVFP4: 2^-9 to 448."""
    return np.array([m * 2.0 ** -9 for m in range(1, 8)] +
                    [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


@pytest.mark.parametrize("factor", [1.0, 0.3, 1.7e-3])
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_f32_ties_and_their_neighbours(fmt, factor):
    """FP32 values at, just below and just above what lies halfway between two
    codes or two scales, for every scale, are rounded as the definition says:
    the FP32 product with the factor, divided exactly, ties to even."""
    b = plain.BLOCK[fmt]
    scales = e4m3_scales() if fmt == "nv" else 2.0 ** np.arange(-90, 91, 6)
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
    f = np.float32(factor)
    blocks = []

    def around(v):
        """FP32 numbers whose product with the factor is v, or the nearest, and their neighbours."""
        x = np.float32(v / np.float64(f))
        return [x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(0))]

    for i, s in enumerate(scales):
        near = np.array([n for t in ties for n in around(t * s)], dtype=np.float32)
        near[1::2] *= -1
        for part in (near[:b - 1], near[b - 1:]):
            block = np.zeros(b, np.float32)
            block[0] = around(6 * s)[0]
            block[1:1 + len(part)] = part
            blocks.append(block)
        if i + 1 < len(scales):             # halfway between two scales
            for x in around(6 * (s + scales[i + 1]) / 2):
                blocks.append(np.r_[x, (near / 1.1)[:b - 1], np.zeros(b)][:b].astype(np.float32))
    x = np.stack(blocks)
    q, s = quantise(torch.from_numpy(x), fmt, scale=factor)
    out = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    swg.mx4_dequantize_into(out, q, s, FMT[fmt])
    assert swg.get_device_error() == 0
    assert np.array_equal(plain.f64(out), plain.quantised((x * f).astype(np.float64), fmt))
