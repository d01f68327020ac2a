"""Plain 64-bit forms of the expert-MLP operators for the tests: products
grouped by expert and microscaled 4-bit numbers, with the error bounds that
the comparisons use.  numpy only; nothing of the library is used here.

Bounds.  A sum of K products in FP32, in any order, with each addition off by
at most one unit in the last place, is within K * 2^-23 * sum |a b| of the
exact one (the products of 16-bit or 4-bit values are exact in FP32 but for
the block scales, one more rounding); 8 more roundings cover alpha, beta and
the epilogue.  Rounding to the output type adds half a unit: 2^-8 (bf16, 8
significant bits) or 2^-11 (f16) of the result, 2^-24 for f32, and half the smallest f16 subnormal.
"""
import numpy as np

ROUND = {"bf16": 2.0 ** -7.99, "f16": 2.0 ** -10.99, "f32": 2.0 ** -23}
TINY = {"bf16": 1e-38, "f16": 2.0 ** -25, "f32": 1e-38}
FAST_EXP = 1e-5          # sigmoid through the fast exponential and division, relative


def f64(t):
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def fp32_sum_bound(K, mags):
    return (K + 8) * 2.0 ** -23 * mags


def groups(offsets):
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def product(A, B, offsets, transB, alpha, beta, C, out):
    """(expected rows, bound) of C <- alpha A op(B_g) + beta C; rows outside
    the groups come back as C with bound 0."""
    want, tol = C.copy(), np.zeros_like(C)
    K = A.shape[1]
    for g, (a, b) in enumerate(groups(offsets)):
        W = B[g].T if transB else B[g]
        p = alpha * (A[a:b] @ W)
        mags = abs(alpha) * (np.abs(A[a:b]) @ np.abs(W))
        if beta:
            p = p + beta * C[a:b]
            mags = mags + np.abs(beta * C[a:b])
        want[a:b] = p
        tol[a:b] = fp32_sum_bound(K, mags) + ROUND[out] * np.abs(p) + TINY[out]
    return want, tol


def wgrad(A, D, offsets, alpha, beta, C, out):
    want, tol = np.empty_like(C), np.empty_like(C)
    for g, (a, b) in enumerate(groups(offsets)):
        p = alpha * (A[a:b].T @ D[a:b])
        mags = abs(alpha) * (np.abs(A[a:b]).T @ np.abs(D[a:b]))
        if beta:
            p = p + beta * C[g]
            mags = mags + np.abs(beta * C[g])
        want[g] = p
        tol[g] = fp32_sum_bound(b - a, mags) + ROUND[out] * np.abs(p) + TINY[out]
    return want, tol


def gate_up(A, W, offsets, alpha=1.0):
    """Gate, Up and their FP32 bounds; W [G, K, 2N] interleaved."""
    M, N = A.shape[0], W.shape[2] // 2
    h, e = np.zeros((M, 2 * N)), np.zeros((M, 2 * N))
    for g, (a, b) in enumerate(groups(offsets)):
        h[a:b] = alpha * (A[a:b] @ W[g])
        e[a:b] = fp32_sum_bound(A.shape[1], abs(alpha) * (np.abs(A[a:b]) @ np.abs(W[g])))
    return h[:, 0::2], h[:, 1::2], e[:, 0::2], e[:, 1::2]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(A, W, offsets, alpha=1.0):
    """Y and its bound.  |d SiLU| <= 1.1 |dg|, |SiLU(g)| <= |g|."""
    g, u, eg, eu = gate_up(A, W, offsets, alpha)
    y = g * sigmoid(g) * u
    tol = 1.1 * np.abs(u) * eg + np.abs(g * sigmoid(g)) * eu + 1.1 * eg * eu
    return y, tol + (ROUND["bf16"] + FAST_EXP) * np.abs(y) + TINY["bf16"]


def swiglu_grad(A, W, dY, offsets):
    """dH (interleaved) and its bound: SiLU' is at most 1.1 and changes by at
    most 0.5 per unit of g; its fast form is off by FAST_EXP of its terms."""
    g, u, eg, eu = gate_up(A, W, offsets)
    s = sigmoid(g)
    d1 = s * (1 + g * (1 - s))
    dg, du = dY * u * d1, dY * g * s
    tg = np.abs(dY) * (0.5 * (np.abs(u) + eu) * eg + 1.1 * eu
                       + FAST_EXP * np.abs(u) * s * (1 + np.abs(g)))
    tu = np.abs(dY) * 1.1 * eg
    M, N = dY.shape
    dH, tol = np.empty((M, 2 * N)), np.empty((M, 2 * N))
    dH[:, 0::2], dH[:, 1::2] = dg, du
    tol[:, 0::2], tol[:, 1::2] = tg, tu
    return dH, tol + (ROUND["bf16"] + FAST_EXP) * np.abs(dH) + TINY["bf16"]


# --------------------------------------------------------------- 4 bits

BLOCK = {"mx": 32, "nv": 16}


def _ceil(a, b):
    return -(-a // b)


def block_scales(x, fmt):
    """Scale of each block of x [rows, K], from the definition; NaN where the
    block holds a NaN or an infinity."""
    b = BLOCK[fmt]
    rows, K = x.shape
    p = np.zeros((rows, _ceil(K, b) * b))
    p[:, :K] = x
    top = np.abs(p.reshape(rows, -1, b)).max(-1)
    bad = ~np.isfinite(top)
    top = np.where(bad, 1.0, top)
    if fmt == "mx":
        e = np.frexp(top)[1] - 1 - 2
        s = np.ldexp(1.0, np.where(top > 0, np.maximum(e, -127), -127))
    else:
        t = top / 6.0
        step = np.ldexp(1.0, np.frexp(np.maximum(t, 2.0 ** -6))[1] - 1 - 3)
        s = np.clip(np.round(t / step) * step, 2.0 ** -9, 448.0)
    return np.where(bad, np.nan, s)


def e2m1_round(v):
    a = np.abs(v)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.sign(v) * np.minimum(np.round(a / step) * step, 6.0)


def quantised(x, fmt):
    """The values that x [rows, K] becomes."""
    s = block_scales(x, fmt)
    s = np.repeat(s, BLOCK[fmt], -1)[:, :x.shape[1]]
    with np.errstate(invalid="ignore"):
        return np.where(np.isnan(s), np.nan, e2m1_round(np.where(np.isnan(s), 0, x) / np.where(np.isnan(s), 1, s)) * s)


GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def pack(v, fmt, scales, group_rows):
    """Codes [rows, bytes] and scale tiles of values v [rows, K] that lie on
    the grid of `scales`, the groups' row counts given; written from the
    documented layout, element by element."""
    rows, K = v.shape
    b = BLOCK[fmt]
    s = np.repeat(scales, b, -1)[:, :K]
    code = np.argmin(np.abs(np.abs(v / s)[..., None] - GRID), -1).astype(np.uint8)
    code |= (np.signbit(v).astype(np.uint8) << 3)
    full = np.zeros((rows, _ceil(K, 32) * 32), np.uint8)
    full[:, :K] = code
    q = full[:, 0::2] | (full[:, 1::2] << 4)
    if fmt == "mx":
        byte = (np.frexp(scales)[1] - 1 + 127).astype(np.uint8)
    else:
        e = np.frexp(scales)[1] - 1
        byte = np.where(scales < 2.0 ** -6, scales * 512,
                        (np.clip(e, -6, 8) + 7) * 8 + scales / np.ldexp(1.0, e) * 8 - 8).astype(np.uint8)
    return q, tiles(byte, group_rows)


def tiles(byte, group_rows):
    """Scale bytes [rows, blocks] in the tiles of their groups."""
    blocks = byte.shape[1]
    across = _ceil(blocks, 4)
    out = []
    row = 0
    for n in group_rows:
        t = np.zeros((_ceil(n, 128), across, 32, 4, 4), np.uint8)
        for r in range(n):
            for j in range(blocks):
                t[r // 128, j // 4, r % 32, r % 128 // 32, j % 4] = byte[row + r, j]
        row += n
        out.append(t.reshape(-1))
    return np.concatenate(out) if out else np.zeros(0, np.uint8)
