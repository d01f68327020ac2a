"""4-bit weights with group scales against their 64-bit forms (routing_plain.py,
where the bounds are derived): the conversion bit for bit, the products at the sizes,
groups, strides and values where they can go wrong."""
import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from experts_plain import FAST_EXP, ROUND, TINY, f64, fp32_sum_bound, groups, sigmoid
from helpers import Guarded
from test_grouped_gpu import offsets_of
from test_routing_gpu import close, gen, padded

pytestmark = pytest.mark.gpu

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = {"f16": 65504.0, "bf16": float(torch.finfo(torch.bfloat16).max)}


def rounder(stype):
    return lambda s: torch.from_numpy(s).to(TYPE[stype]).float().numpy()


def weight(G, N, K, group, zero, stype, seed=0, std=0.05):
    """Codes, scales and zero points drawn at random, with junk in the padding, and the
    values [G, N, K] they stand for."""
    rng = np.random.default_rng(seed)
    Q, S, Z = swg.w4_alloc(N, K, group, TYPE[stype], zeros=zero, experts=G, device="cpu")
    Q.copy_(torch.from_numpy(rng.integers(0, 256, Q.shape).astype(np.uint8)))
    S.copy_(torch.from_numpy(rng.uniform(0.2, 1.0, S.shape) * std))
    S[:, :, N:] = float("nan")
    if zero:
        Z.copy_(torch.from_numpy(rng.integers(0, 256, Z.shape).astype(np.uint8)))      # the upper bits do not count
    w = np.stack([plain.values(Q[g].numpy(), f64(S[g]), None if Z is None else Z[g].numpy(), N, K, group) for g in range(G)])
    return (Q.cuda(), S.cuda(), None if Z is None else Z.cuda()), w


# -------------------------------------------------------------- conversion

def check_conversion(x, group, zero, stype, what=""):
    N, K = x.shape
    Q, S, Z = swg.w4_alloc(N, K, group, TYPE[stype], zeros=zero)
    for t in (Q, S, Z) if zero else (Q, S):
        t.fill_(99)
    swg.w4_quantize_into(Q, S, Z, x, group)
    assert swg.get_device_error() == 0
    q, s, z = plain.quantised(f64(x).astype(np.float32), group, zero, rounder(stype), LARGEST[stype])
    full = np.zeros((N, Q.shape[1] * 2), np.int64)
    full[:, :K] = q
    got = plain.unpack(Q.cpu().numpy(), full.shape[1])
    assert np.array_equal(got, full), f"{what}: codes differ at {np.argwhere(got != full)[:4].tolist()}"
    assert np.array_equal(f64(S)[:, :N], s, equal_nan=True), f"{what}: scales"
    assert bool((S[:, N:].float() == 99).all())          # columns that no row has are left alone
    if zero:
        assert np.array_equal(Z.cpu().numpy()[:, :N], z), f"{what}: zero points"
    return Q, S, Z


@pytest.mark.parametrize("N,K", [(1, 1), (1, 32), (3, 31), (5, 33), (32, 256), (33, 257), (40, 300), (100, 1000), (257, 96)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("xtype,stype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "f16")])
def test_quantise_and_back(N, K, group, zero, xtype, stype):
    x = padded(N, K, xtype, N + K, std=0.02)
    Q, S, Z = check_conversion(x, group, zero, stype)
    w = plain.values(Q.cpu().numpy(), f64(S), None if Z is None else Z.cpu().numpy(), N, K, group)
    for out in ("bf16", "f16", "f32"):
        y = Guarded(N, K, TYPE[out], fill=1.0)
        swg.w4_dequantize_into(y.view, Q, S, Z, group)
        assert swg.get_device_error() == 0
        want = torch.from_numpy(w).float().to(TYPE[out])
        assert torch.equal(y.cpu("dequantise"), want)
    # no value is further than half a step, and a scale's rounding of the range, from x
    step = np.repeat(f64(S)[:, :N], group, 0)[:K].T
    assert (np.abs(w - f64(x)) <= step * (0.5 + 15 * ROUND[stype] + (0.5 if zero else 0)) + TINY[stype] * 15).all()


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("stype", ["bf16", "f16"])
def test_values_where_rounding_decides(zero, stype):
    """Halves of steps of many scales, and the floats next to them."""
    rng = np.random.default_rng(3)
    rows = []
    for i in range(300):
        s = np.float32(rounder(stype)(np.array([rng.uniform(1, 2) * 2.0 ** rng.integers(-9, 4)], np.float32))[0])
        half = (rng.integers(-7, 7, 128) + 0.5).astype(np.float32) * s
        x = np.where(rng.random(128) < 0.5, half, np.nextafter(half, rng.choice([-np.inf, np.inf], 128).astype(np.float32)))
        x[:2] = s * 7, -s * 7
        if zero:
            x[0] = s * 8
        rows.append(x)
    x = torch.from_numpy(np.array(rows, np.float32)).cuda()
    check_conversion(x, 128, zero, stype)
    check_conversion(x.to(TYPE[stype]), 64, zero, stype)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("stype", ["bf16", "f16"])
def test_extreme_values(zero, stype):
    x = torch.randn((20, 128), generator=gen(9))
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 70] = float("inf")
    x[3, 3] = -float("inf")
    x[4] *= 1e-42
    x[5] *= 1e-38
    x[6] *= 1e-30
    x[7] *= 1e38
    x[8] = 3.4e38
    x[9] = x[9].abs()
    x[10] = -x[10].abs()
    x[11, 1:] = 0
    x[12] *= 2.0 ** -18
    x[13] = 1e-8
    x[14] = -0.0
    x[15, :64] = 3.4e38
    x[15, 64:] = -3.4e38
    for group in (32, 64, 128):
        check_conversion(x.cuda(), group, zero, stype, f"group {group}")


def test_experts_of_a_weight():
    """[G, N, K] at once is each matrix by itself."""
    G, N, K, group = 3, 50, 100, 32
    x = torch.randn((G, N, 104), generator=gen(2)).bfloat16().cuda()[:, :, :K]
    Q, S, Z = swg.w4_alloc(N, K, group, torch.bfloat16, zeros=True, experts=G)
    swg.w4_quantize_into(Q, S, Z, x, group)
    back = swg.w4_dequantize_into(torch.empty((G, N, 104), dtype=torch.bfloat16, device="cuda")[:, :, :K], Q, S, Z, group)
    for g in range(G):
        q, s, z = swg.w4_quantize_into(*swg.w4_alloc(N, K, group, torch.bfloat16, zeros=True), x[g], group)
        assert torch.equal(q, Q[g]) and torch.equal(s[:, :N], S[g, :, :N]) and torch.equal(z[:, :N], Z[g, :, :N])
        assert torch.equal(swg.w4_dequantize_into(torch.empty((N, K + 4), dtype=torch.bfloat16, device="cuda")[:, :K], q, s, z, group), back[g])


# ---------------------------------------------------------------- products

def product(a, w, off, alpha, beta, old, out):
    want, tol = old.copy(), np.zeros_like(old)
    for g, (i, j) in enumerate(groups(off)):
        p = alpha * (a[i:j] @ w[g].T) + (beta * old[i:j] if beta else 0)
        want[i:j] = p
        tol[i:j] = plain.w4_bound(a[i:j], w[g], p, alpha, out, np.abs(beta * old[i:j]) if beta else 0.0)
    return want, tol


def run_gemm(rows, N, K, group=128, zero=False, stype="bf16", out=None, alpha=1.0, beta=0.0, before=0, after=0, seed=1,
             dense=False, stream=None):
    out = out or stype
    off = offsets_of(rows, before)
    M, G = int(off[-1]) + after, len(rows)
    W, w = weight(G, N, K, group, zero, stype, seed)
    A = padded(M, K, stype, seed)
    A[:before] = float("nan")
    A[M - after:] = float("nan")
    old = torch.randn((M, N), generator=gen(seed)).to(TYPE[out])
    C = Guarded(M, N, TYPE[out], init=old)
    swg.gemm_w4_into(C.view, A, *W, group, alpha=alpha, beta=beta, offsets=None if dense else torch.from_numpy(off).cuda(),
                     stream=stream)
    assert swg.get_device_error(stream) == 0
    a = np.nan_to_num(f64(A))
    want, tol = product(a, w, off, alpha, beta, f64(old), out)
    close(C.cpu("gemm_w4"), want, tol, f"{rows} N={N} K={K} group={group}")
    return C.view


@pytest.mark.parametrize("K", [1, 7, 8, 31, 32, 33, 64, 127, 128, 129, 500, 1024, 1025, 3200])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_contraction_lengths(K, group, zero):
    run_gemm([3], 40, K, group, zero, "bf16", "f32", seed=K, dense=True)
    run_gemm([1], 33, K, group, zero, "f16", seed=K + 1, dense=True)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 100, 5000])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 17, 40])
def test_rows_and_columns(M, N):
    run_gemm([M], N, 200, 32, True, "f16", seed=M, dense=True)
    run_gemm([M], N, 200, 128, False, "bf16", seed=N, dense=True)


@pytest.mark.parametrize("rows", [[1], [0], [0, 5, 1, 0, 13, 8, 0], [1] * 40, [0, 0, 0, 9], [33, 0, 40], [0] * 31 + [2] + [0] * 40 + [17]])
@pytest.mark.parametrize("stype", ["bf16", "f16"])
def test_ragged_groups(rows, stype):
    run_gemm(rows, 72, 300, 64, True, stype, seed=len(rows))
    run_gemm(rows, 72, 160, 32, False, stype, "f32", seed=len(rows) + 1, before=3, after=2)


@pytest.mark.parametrize("K", [2049, 2300, 4096, 9000])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("M", [1, 8, 16, 40])
def test_long_rows(K, group, zero, M):
    run_gemm([M], 200, K, group, zero, "bf16" if zero else "f16", "f32", seed=K, dense=True)


@pytest.mark.parametrize("N", [1, 2, 31, 63, 64, 65, 96, 127, 128, 129, 1000])
@pytest.mark.parametrize("M", [9, 15, 17, 31, 32, 33, 70])
def test_many_rows_and_columns(M, N):
    run_gemm([M], N, 2100, 64, True, "f16", seed=M, dense=True, alpha=0.5, beta=1.0)


@pytest.mark.parametrize("M,N,K,group", [(9, 2100, 9000, 32), (16, 2303, 8200, 128), (31, 1100, 8200, 64), (32, 1057, 9001, 32),
                                         (40, 1000, 9000, 128), (70, 520, 8500, 64)])
@pytest.mark.parametrize("zero,stype", [(False, "bf16"), (True, "f16")])
def test_many_rows_of_large_weights(M, N, K, group, zero, stype):
    run_gemm([M], N, K, group, zero, stype, "f32", seed=N, dense=True)


@pytest.mark.parametrize("rows", [[16], [60, 0, 7, 1, 0, 33], [0, 0, 0, 70], [32, 64, 31], [17] * 20])
@pytest.mark.parametrize("N,K,group,zero", [(72, 100, 32, True), (130, 700, 64, False), (8, 2100, 128, True)])
@pytest.mark.parametrize("stype", ["bf16", "f16"])
def test_ragged_groups_of_many_rows(rows, N, K, group, zero, stype):
    run_gemm(rows, N, K, group, zero, stype, seed=N, before=3, after=2)


@pytest.mark.parametrize("rows,N,K", [([40], 100, 2100), ([12], 64, 4000), ([30, 0, 40], 70, 600), ([2], 20, 4500)])
def test_swiglu_of_many_rows(rows, N, K):
    test_swiglu(rows, N, K, 64, True, "bf16")


@pytest.mark.parametrize("alpha,beta", [(0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (0.0, 1.0)])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
def test_alpha_beta(alpha, beta, out):
    for stype in ("bf16", "f16"):
        run_gemm([4, 0, 7], 51, 96, 32, True, stype, out, alpha, beta, seed=5)


def test_no_columns():
    """K = 0: C = beta * C."""
    C = torch.ones((3, 8), device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    swg.gemm_w4_into(C, e(3, 0), e(8, 0, t=torch.uint8), e(0, 16), None, 32, beta=0.5)
    assert float(C.sum()) == 12 and swg.get_device_error() == 0


def test_infinities_and_nans_stay_in_their_rows():
    W, w = weight(1, 40, 64, 32, True, "bf16", 1)
    A = torch.randn((5, 64), generator=gen(1)).bfloat16()
    A[1, 3], A[3, 9] = float("nan"), float("inf")
    C = torch.empty((5, 40), device="cuda")
    swg.gemm_w4_into(C, A.cuda(), *W, 32)
    assert bool(torch.isnan(C[1]).all()) and not bool(torch.isfinite(C[3]).any())
    keep = [0, 2, 4]
    a = f64(A)[keep]
    close(C[keep], a @ w[0].T, plain.w4_bound(a, w[0], a @ w[0].T, 1.0, "f32"))


def test_a_group_that_reads_back_as_nan():
    x = torch.randn((20, 64), generator=gen(1)).bfloat16()
    x[4, 40] = float("inf")
    W = swg.w4_quantize_into(*swg.w4_alloc(20, 64, 32, torch.bfloat16), x.cuda(), 32)
    C = torch.empty((2, 32), device="cuda")[:, :20]
    swg.gemm_w4_into(C, torch.ones((2, 64), dtype=torch.bfloat16, device="cuda"), *W, 32)
    assert torch.isnan(C).cpu().sum(0).tolist() == [2 if n == 4 else 0 for n in range(20)]


def swiglu(a, w, off, alpha):
    M, N = a.shape[0], w.shape[1] // 2
    y, tol = np.zeros((M, N)), np.zeros((M, N))
    for g, (i, j) in enumerate(groups(off)):
        h = alpha * (a[i:j] @ w[g].T)
        e = fp32_sum_bound(a.shape[1], abs(alpha) * (np.abs(a[i:j]) @ np.abs(w[g]).T))
        gt, up, eg, eu = h[:, 0::2], h[:, 1::2], e[:, 0::2], e[:, 1::2]
        s = gt * sigmoid(gt)
        y[i:j] = s * up
        tol[i:j] = 1.1 * np.abs(up) * eg + np.abs(s) * eu + 1.1 * eg * eu
    return y, tol


@pytest.mark.parametrize("rows", [[1], [3], [0, 5, 1, 0, 13], [1] * 20, [24]])
@pytest.mark.parametrize("N,K,group,zero", [(8, 128, 128, False), (33, 200, 32, True), (600, 96, 64, True), (1, 32, 32, False)])
@pytest.mark.parametrize("stype", ["bf16", "f16"])
def test_swiglu(rows, N, K, group, zero, stype):
    off = offsets_of(rows)
    M = int(off[-1])
    W, w = weight(len(rows), 2 * N, K, group, zero, stype, N + K)
    A = padded(M, K, stype, K)
    Y = Guarded(M, N, TYPE[stype], fill=3.0)
    swg.swiglu_w4_into(Y.view, A, *W, group, alpha=0.5, offsets=torch.from_numpy(off).cuda())
    assert swg.get_device_error() == 0
    want, tol = swiglu(f64(A), w, off, 0.5)
    close(Y.cpu("swiglu_w4"), want, tol + (ROUND[stype] + FAST_EXP) * np.abs(want) + TINY[stype], "swiglu_w4")


def test_wrong_offsets_are_clamped_and_reported():
    W, w = weight(3, 40, 64, 32, False, "bf16", 1)
    A = torch.randn((6, 64), generator=gen(1)).bfloat16()
    for off, clamped in (([0, 4, 2, 6], [0, 4, 4, 6]), ([-3, 2, 3, 9], [0, 2, 3, 6]), ([0, 7, 1, 2], [0, 6, 6, 6])):
        C = torch.full((6, 40), 3.0, device="cuda")
        swg.gemm_w4_into(C, A.cuda(), *W, 32, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert swg.get_device_error() == 1 and swg.get_device_error() == 0
        want, tol = product(f64(A), w, np.array(clamped), 1.0, 0.0, np.full((6, 40), 3.0), "f32")
        close(C, want, tol, str(off))
    A = torch.randn((60, 64), generator=gen(1)).bfloat16()       # chunks of 32 rows
    for off, clamped in (([0, 40, 2, 60], [0, 40, 40, 60]), ([-3, 20, 33, 90], [0, 20, 33, 60]), ([0, 70, 1, 2], [0, 60, 60, 60])):
        C = torch.full((60, 40), 3.0, device="cuda")
        swg.gemm_w4_into(C, A.cuda(), *W, 32, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert swg.get_device_error() == 1 and swg.get_device_error() == 0
        want, tol = product(f64(A), w, np.array(clamped), 1.0, 0.0, np.full((60, 40), 3.0), "f32")
        close(C, want, tol, str(off))


def test_same_bits_again_and_on_another_stream():
    for rows, K in (([5, 9], 1000), ([5], 9000), ([40], 2100)):
        a = run_gemm(rows, 300, K, 64, True, "bf16", seed=8)
        b = run_gemm(rows, 300, K, 64, True, "bf16", seed=8, stream=torch.cuda.Stream())
        assert torch.equal(a, b)


def test_beyond_32_bits():
    """Codes of an expert that begin beyond 2^31 bytes."""
    G, N, K, group = 3, 40000, 65536, 128
    Q = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda")
    S = torch.zeros((G, K // group, N), dtype=torch.bfloat16, device="cuda")
    Q[2, N - 3:] = 0x99                                  # 9 - 8
    S[2, :, N - 3:] = 0.5
    A = torch.ones((2, K), dtype=torch.bfloat16, device="cuda")
    C = torch.empty((2, N), device="cuda")
    off = torch.tensor([0, 0, 0, 2], dtype=torch.int32, device="cuda")
    swg.gemm_w4_into(C, A, Q, S, None, group, offsets=off)
    assert swg.get_device_error() == 0
    assert C[:, N - 3:].tolist() == [[K / 2] * 3] * 2 and float(C[:, :N - 3].abs().sum()) == 0
    X = swg.w4_dequantize_into(torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda"), Q, S, None, group)
    assert float(X[2, N - 3:].float().sum()) == 3 * K / 2 and float(X[1, :16].abs().sum()) == 0


# -------------------------------------------------------------- as one layer

def test_decoded_layer_in_a_graph():
    """route, dispatch, swiglu_w4, gemm_w4 and combine, captured once and replayed with other tokens."""
    T, E, top, D, H, group = 9, 8, 2, 200, 136, 64
    up, wu = weight(E, 2 * H, D, group, True, "bf16", 1)
    down, wd = weight(E, D, H, group, False, "bf16", 2)
    t = dict(dtype=torch.bfloat16, device="cuda")
    x, l = torch.empty((T, D), **t), torch.empty((T, E), device="cuda")
    experts, weights = torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda")
    plan = swg.expert_plan_alloc(T, E, top)
    rows, y, z, out = (torch.empty((n, d), **t) for n, d in ((T * top, D), (T * top, H), (T * top, D), (T, D)))

    def layer():
        swg.expert_route_into(experts, weights, l, swg.SIGMOID, plan=plan)
        swg.expert_dispatch_into(rows, x, plan[2])
        swg.swiglu_w4_into(y, rows, *up, group, offsets=plan[0])
        swg.gemm_w4_into(z, y, *down, group, offsets=plan[0])
        swg.expert_combine_into(out, z, plan[2], weights)

    g = torch.cuda.CUDAGraph()
    x.zero_()
    l.zero_()
    layer()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer()
    for seed in range(3):
        x.copy_(torch.randn((T, D), generator=gen(seed)))
        l.copy_(torch.randn((T, E), generator=gen(seed + 50)))
        if seed == 2:
            l[5:] = -float("inf")                        # a batch that is not full
        g.replay()
        torch.cuda.synchronize()
        assert swg.get_device_error() == 0
        e, w = plain.route(f64(l), None, top, "sigmoid")
        want, tol = np.zeros((T, D)), np.zeros((T, D))
        for i in range(T):
            for j in range(top):
                k = e[i, j]
                if k < 0:
                    continue
                a = f64(x)[i:i + 1]
                h, eh = swiglu(a, wu[[k]], [0, 1], 1.0)
                eh = eh + (ROUND["bf16"] + FAST_EXP) * np.abs(h)
                o = h @ wd[k].T
                eo = eh @ np.abs(wd[k]).T + plain.w4_bound(np.abs(h) + eh, wd[k], o, 1.0, "bf16")
                want[i] += w[i, j] * o[0]
                tol[i] += w[i, j] * (eo[0] + 2.0 ** -18 * np.abs(o[0]))
        close(out, want, tol * 1.01 + ROUND["bf16"] * np.abs(want) + 1e-30, f"layer {seed}")
