"""Plain 64-bit forms of the routing operators and of 4-bit weights with group
scales for the tests, with the error bounds that the comparisons use.  numpy only;
nothing of the library is used here.

Bounds.  U = 2^-24 is half a unit of FP32.  An exponential is off by 2 units (4 U)
and by the rounding of its argument, a difference of logits at most `spread`:
spread * U.  A quotient of two such, a sum of n of them and a few products: R =
(2 * spread + 2 * n + 24) * U of the result covers it.
"""
import numpy as np

from experts_plain import ROUND, TINY, fp32_sum_bound

U = 2.0 ** -24


def scores(l, score):
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
        z = e.sum(1, keepdims=True)
        return e / np.where(z == 0, 1.0, z)


def route(l, bias, top, score="softmax", groups=1, top_groups=None, group_sum=1, normalise=True, scale=1.0):
    """(experts, weights) token by token, from the definition."""
    T, E = l.shape
    s = scores(l, score)
    top_groups = top_groups or groups
    experts, weights = np.full((T, top), -1, np.int64), np.zeros((T, top))
    for t in range(T):
        c = l[t] if bias is None and group_sum == 1 else s[t] if bias is None else s[t] + bias
        left = ~np.isneginf(l[t]) & ~np.isneginf(c)
        if np.isnan(c[left]).any() or np.isnan(s[t]).any():
            experts[t], weights[t] = np.arange(top), np.nan
            continue
        if top_groups < groups:
            size = E // groups
            value = []
            for g in range(groups):
                own = np.sort(c[g * size:(g + 1) * size][left[g * size:(g + 1) * size]])[::-1]
                value.append(own[:group_sum].sum() if len(own) else -np.inf)
            best = sorted((g for g in range(groups) if value[g] > -np.inf), key=lambda g: (-value[g], g))[:top_groups]
            left &= np.isin(np.arange(E) // size, best)
        by = l[t] if bias is None else c                 # (groups are chosen by their scores all the same)
        order = sorted(np.flatnonzero(left), key=lambda e: (-by[e], e))[:top]
        experts[t, :len(order)] = order
        w = s[t, order]
        if normalise and len(order):
            # through logarithms: all scores may be too small for 64 bits
            log = l[t, order] if score == "softmax" else -np.logaddexp(0.0, -l[t, order])
            w = np.exp(log - log.max())
            w = w / w.sum()
        weights[t, :len(order)] = scale * w
    return experts, weights


def spread(l):
    on = np.isfinite(l)
    d = np.where(on, l, -np.inf).max(1, initial=-np.inf) - np.where(on, l, np.inf).min(1, initial=np.inf)
    return np.maximum(d, 0.0)[:, None]                   # (0 where no logit is finite)


def route_bound(l, weights, top):
    """Of the weights: sums of `top` or of a row's scores."""
    return (2 * spread(l) + 2 * max(top, l.shape[1] // 32 + 8) + 24) * U * np.abs(weights) + 1e-37


def route_grad(l, experts, dw, score, normalise, scale):
    """(d_logits, magnitudes that its FP32 errors are relative to)."""
    T, E = l.shape
    s = scores(l, score)
    out, mags = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = np.flatnonzero(experts[t] >= 0)
        e = experts[t, on]
        d = scale * dw[t, on]
        p = s[t, e]
        if normalise:
            p = p / p.sum() if len(on) else p
            x, m = p * (d - (p * d).sum()), p * (np.abs(d) + (p * np.abs(d)).sum())
            if score == "sigmoid":
                x, m = x * (1 - s[t, e]), m * (1 - s[t, e])
            np.add.at(out[t], e, x)
            np.add.at(mags[t], e, m)
        elif score == "sigmoid":
            np.add.at(out[t], e, d * p * (1 - p))
            np.add.at(mags[t], e, np.abs(d) * p * (1 - p))
        else:
            g, a = np.zeros(E), np.zeros(E)
            np.add.at(g, e, d)
            np.add.at(a, e, np.abs(d))
            out[t] = s[t] * (g - (d * p).sum())
            mags[t] = s[t] * (a + (np.abs(d) * p).sum())
    return out, mags


def grad_bound(l, want, mags, top, out):
    r = (2 * spread(l) + 2 * max(top, l.shape[1] // 32 + 8) + 24) * U
    return 3 * r * mags + ROUND[out] * np.abs(want) + TINY[out]


def plan(experts, E):
    flat = experts.reshape(-1)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    source, position = np.full(len(flat), -1), np.full(len(flat), -1)
    r = 0
    for e in range(E):
        for i in np.flatnonzero(flat == e):
            source[r], position[i] = i, r
            r += 1
    return offsets, source, position.reshape(experts.shape)


def combine(rows, position, weights, beta, old, out):
    T, top = position.shape
    want, mags = beta * old, np.abs(beta * old)
    for t in range(T):
        for j in range(top):
            if position[t, j] >= 0:
                x = weights[t, j] * rows[position[t, j]]
                want[t] += x
                mags[t] += np.abs(x)
    return want, (top + 3) * U * mags + ROUND[out] * np.abs(want) + TINY[out]


# ------------------------------------------------------------ 4-bit weights

def unpack(Q, K):
    """Codes [rows, K] of bytes, from the documented layout, one by one."""
    rows = Q.shape[0]
    words = Q.reshape(rows, -1, 4).astype(np.int64) @ (1 << np.array([0, 8, 16, 24]))
    q = np.empty((rows, K), np.int64)
    for k in range(K):
        q[:, k] = words[:, k // 8] >> (16 * (k % 2) + 4 * (k % 8 // 2)) & 15
    return q


def values(Q, S, Z, rows, K, group):
    """w [rows, K] of one matrix: bytes, scales and zero points [blocks, lds] (None: 8)."""
    q = unpack(Q, K).astype(np.float64)
    block = np.arange(K) // group
    s = S[block, :rows].T
    z = 8.0 if Z is None else (Z[block, :rows].T & 15).astype(np.float64)
    return s * (q - z)


def quantised(x, group, zero, round_scale, largest):
    """(codes, scales, zero points) of x [rows, K] float32, as the definition rounds: quotients in FP32."""
    rows, K = x.shape
    f = np.float32
    q = np.zeros((rows, K), np.int64)
    blocks = -(-K // group)
    S, Z = np.zeros((blocks, rows), np.float64), np.zeros((blocks, rows), np.int64)
    with np.errstate(all="ignore"):
        for b in range(blocks):
            p = x[:, b * group:(b + 1) * group].astype(f)
            bad = ~np.isfinite(p).all(1)
            p = np.where(bad[:, None], f(0), p)
            lo, hi = np.minimum(p.min(1), f(0)), np.maximum(p.max(1), f(0))
            s = (hi - lo) / f(15) if zero else np.maximum(hi, -lo) / f(7)
            s = np.minimum(round_scale(s.astype(f)), f(largest)).astype(f)
            div = lambda a: np.where(s > 0, a / np.where(s > 0, s, f(1)), f(0)).astype(f)  # noqa: E731
            z = np.clip(np.rint(div(-lo)), 0, 15) if zero else np.full(rows, 8.0)
            c = np.clip(np.rint(np.where(s[:, None] > 0, p / np.where(s > 0, s, f(1))[:, None], f(0)))
                        + z[:, None], 0, 15)
            q[:, b * group:(b + 1) * group] = np.where(bad[:, None], 0, c)
            S[b], Z[b] = np.where(bad, np.nan, s), np.where(bad, 0, z)
    return q, S, Z


def w4_bound(A, W, want, alpha, out, extra=0.0):
    mags = np.abs(alpha) * (np.abs(A) @ np.abs(W).T) + extra
    return fp32_sum_bound(A.shape[1], mags) + ROUND[out] * np.abs(want) + TINY[out]
