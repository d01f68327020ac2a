"""Cases of the expert-MLP operators: matrix products grouped by expert with
ragged sizes, and microscaled 4-bit floating point (quantisation and product).

A case's ``op``:

* ``gemm``    C = A op(B_g) for the rows of each group (``trans`` 0: forward,
              1: the gradient of the input).
* ``wgrad``   C_g = A_g^T D_g, the gradient of each group's weight.
* ``swiglu``  Y = SiLU(A W1_g) * (A W2_g), weights interleaved column by column.
* ``dswiglu`` the gradient of that in the pre-activations, and Y again.
* ``round``   x to 4 bits with block scales, and the values those stand for.
* ``linear``  x to 4 bits, then the product with 4-bit weights.
* ``mlp4``    x to 4 bits, then SwiGLU with 4-bit weights (of each expert).

Rows are sorted by group; ``offsets`` (groups + 1 numbers on the GPU) says
where each group begins.  4-bit formats: ``mx`` (e2m1 in blocks of 32 with a
power-of-two scale) and ``nv`` (e2m1 in blocks of 16 with an e4m3 scale).
Two e2m1 codes are kept in a byte, the lower index in the lower half.  Scales
are kept in tiles of 128 rows x 4 blocks (512 bytes): row r, block b of a tile
at byte 16 * (r % 32) + 4 * (r // 32) + b; a row of tiles covers all of K, and
each group of rows begins a new row of tiles.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"mx": 32, "nv": 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    """Real work over the range of sizes, types and directions."""
    return [
        # one token through two of eight experts of the small model: the latency of decoding
        dict(name="swiglu_decode", op="swiglu", M=2, G=8, K=896, N=4864, route=5, skew=0.0),
        # 32 decoded tokens, two experts each, of 64 fine-grained experts; some stay empty
        dict(name="gemm_decode_f16", op="gemm", trans=0, type="f16", out="f16", M=64, G=64, K=1216, N=896, pad=0, route=2, skew=0.7),
        # prefill of 8192 tokens, two of 16 experts each
        dict(name="swiglu_prefill", op="swiglu", M=16384, G=16, K=4096, N=1792, route=3, skew=0.5),
        # input gradient in fp16 at odd sizes, rows in padded storage, uneven experts
        dict(name="gemm_dx_odd", op="gemm", trans=1, type="f16", out="f16", M=5003, G=12, K=2051, N=1003, pad=16, route=4, skew=1.0),
        # weight gradient of a training step
        dict(name="wgrad_train", op="wgrad", type="bf16", out="bf16", M=16384, G=16, K=1792, N=4096, pad=0, route=5, skew=0.5),
        # weight gradient of a small step, most experts with few rows or none
        dict(name="wgrad_small", op="wgrad", type="f16", out="f16", M=203, G=48, K=896, N=521, pad=8, route=6, skew=1.2),
        # activation gradient of a training step, Gate and Up computed again
        dict(name="dswiglu_train", op="dswiglu", M=8192, G=8, K=4096, N=1792, route=7, skew=0.5),
        # a weight of the 8B-class model to 4 bits and back
        dict(name="round_mx_weight", op="round", fmt="mx", type="bf16", M=14336, K=4096),
        # a few activations at an odd width
        dict(name="round_nv_odd", op="round", fmt="nv", type="f16", M=333, K=4105),
        # one decoded token through a 4-bit layer of the 8B-class model
        dict(name="linear_mx_decode", op="linear", fmt="mx", out="bf16", M=1, K=4096, N=14336),
        # prefill through the same layer
        dict(name="linear_nv_prefill", op="linear", fmt="nv", out="bf16", M=8192, K=4096, N=14336),
        # ragged experts in 4 bits
        dict(name="mlp4_mx_experts", op="mlp4", fmt="mx", M=4099, G=32, K=2048, N=1216, route=8, skew=0.8),
    ]


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest of them."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gemm", "gemm", "wgrad", "swiglu", "dswiglu", "round", "linear", "mlp4"])
    while True:
        if op in ("gemm", "wgrad"):
            c = dict(op=op, type=rng.choice(["bf16", "f16"]), M=log(1, 16384), G=log(1, 128), K=log(64, 4096),
                     N=log(64, 4096), pad=rng.choice([0, 8, 40]), route=rng.randrange(10 ** 6), skew=rng.choice([0.0, 0.5, 1.0]))
            c["out"] = c["type"]
            if op == "gemm":
                c["trans"] = rng.randrange(2)
        elif op in ("swiglu", "dswiglu"):
            c = dict(op=op, M=log(1, 16384), G=log(1, 128), K=8 * log(8, 512), N=8 * log(8, 608),
                     route=rng.randrange(10 ** 6), skew=rng.choice([0.0, 0.5, 1.0]))
        elif op == "round":
            c = dict(op=op, fmt=rng.choice(["mx", "nv"]), type=rng.choice(["bf16", "f16"]), M=log(1, 14336), K=log(32, 8192))
        elif op == "linear":
            c = dict(op=op, fmt=rng.choice(["mx", "nv"]), out=rng.choice(["bf16", "f16"]), M=log(1, 8192), K=log(64, 8192), N=log(64, 14336))
        else:
            c = dict(op=op, fmt=rng.choice(["mx", "nv"]), M=log(1, 8192), G=log(1, 64), K=log(64, 4096),
                     N=8 * log(8, 256), route=rng.randrange(10 ** 6), skew=rng.choice([0.0, 0.5, 1.0]))
        w = work(c)
        if w["flops"] <= 4.8e11 and w["bytes"] <= 1.2e9 and c.get("G", 1) * c["K"] * c.get("N", 1) <= 2 ** 29:
            return c


# ------------------------------------------------------------------ inputs

def rows_of(case):
    """Rows of each group: a draw of the router's kind, some groups more
    wanted than others (``skew``), from the case alone."""
    r = np.random.RandomState(case["route"])
    p = (1.0 + np.arange(case["G"])) ** -case["skew"]
    return r.multinomial(case["M"], r.permutation(p / p.sum()))


def pad_to(x, m):
    return -(-x // m) * m


def normal(shape, g, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rows_in(rows, cols, g, std, dtype, pad):
    """A rows x cols matrix in storage whose row length is a multiple of 16
    bytes, ``pad`` more elements of it unused."""
    return normal((rows, pad_to(cols, 8) + pad), g, std, dtype)[:, :cols]


def activations(M, K, g, dtype):
    """Normal, with one channel in 64 eight times as large, as outlier
    channels of a transformer's residual stream are."""
    x = torch.randn((M, pad_to(K, 8)), generator=g, device="cuda")
    x[:, ::64] *= 8.0
    return x.to(dtype)[:, :K]


def random_4bit(rows, K, fmt, g, groups=1):
    """A weight in 4 bits, in hand: codes [groups * rows, bytes] and scale
    tiles, quantised from N(0, 0.02) (x 64 for the e4m3 scales' range)."""
    b = BLOCK[fmt]
    x = torch.randn((groups * rows, K), generator=g, device="cuda") * (0.02 if fmt == "mx" else 1.28)
    codes, scale = quantise(x, fmt)
    q = codes.new_zeros((groups * rows, pad_to(K, 32)))
    q[:, :K] = codes
    q = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    tiles = -(-K // (4 * b))
    s = scale.new_zeros((groups, pad_to(rows, 128), tiles * 4), dtype=torch.uint8)
    s[:, :rows, :scale.shape[1]] = scale_code(scale, fmt).view(groups, rows, -1)
    s = s.view(groups, -1, 4, 32, tiles, 4).permute(0, 1, 4, 3, 2, 5).contiguous()
    return q, s.view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N", 0)
    if "G" in case:
        G = case["G"]
        n = rows_of(case)
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        s["offsets"] = torch.from_numpy(off).cuda()
        s["most"] = int(n.max())
    if op in ("gemm", "wgrad"):
        t, pad = TYPES[case["type"]], case["pad"]
        s["A"] = rows_in(M, K, g, 1.0, t, pad)
        if op == "gemm":
            shape = (K, N) if case["trans"] == 0 else (N, K)
            s["B"] = rows_in(G * shape[0], shape[1], g, K ** -0.5, t, pad).unflatten(0, (G, shape[0]))
            s["C"] = torch.empty((M, pad_to(N, 8) + pad), dtype=TYPES[case["out"]], device="cuda")[:, :N]
        else:
            s["D"] = rows_in(M, N, g, 0.1, t, pad)
            s["C"] = torch.empty((G, K, pad_to(N, 8) + pad), dtype=TYPES[case["out"]], device="cuda")[:, :, :N]
    elif op in ("swiglu", "dswiglu"):
        s["A"] = normal((M, K), g)
        s["W"] = normal((G, K, 2 * N), g, K ** -0.5)
        s["Y"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        if op == "dswiglu":
            s["dY"] = normal((M, N), g, 0.1)
            s["dH"] = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
    elif op == "round":
        s["X"] = activations(M, K, g, TYPES[case["type"]])
        s["V"] = torch.empty((M, pad_to(K, 8)), dtype=torch.bfloat16, device="cuda")[:, :K]
    else:
        G = case.get("G", 1)
        s["X"] = activations(M, K, g, torch.bfloat16)
        if op == "linear":
            s["W"], s["SW"] = random_4bit(N, K, case["fmt"], g)
            s["C"] = torch.empty((M, pad_to(N, 8)), dtype=TYPES[case["out"]], device="cuda")[:, :N]
        else:
            s["W"], s["SW"] = random_4bit(2 * N, K, case["fmt"], g, G)
            s["W"] = s["W"].unflatten(0, (G, 2 * N))
            s["Y"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    if "fmt" in case:  # where the call keeps the 4-bit rows: codes and scale tiles
        tiles = (pad_to(M, 128) // 128 + case.get("G", 1)) * -(-K // (4 * BLOCK[case["fmt"]]))
        s["Q"] = torch.empty((M, pad_to(K, 32) // 2), dtype=torch.uint8, device="cuda")
        s["S"] = torch.empty(tiles * 512, dtype=torch.uint8, device="cuda")
        s["alpha"] = weight_alpha(case["fmt"], K)
    return s


def weight_alpha(fmt, K):
    """What the layer multiplies its sums by: brings the products of unit
    activations and the weight above to about one."""
    std = 0.02 if fmt == "mx" else 1.28
    return 2.0 ** round(math.log2(1.0 / (std * math.sqrt(K))))


# -------------------------------------------------------------- plain form

def power(e):
    """2^e for whole numbers e from -126 to 127 (0 below), from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def quantise(x, fmt):
    """e2m1 codes (sign in bit 3) and the block scales, in 32 bits."""
    b = BLOCK[fmt]
    rows, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, pad_to(K, b) - K)).view(rows, -1, b)
    top = x.abs().amax(-1)
    if fmt == "mx":
        e = torch.frexp(top).exponent - 3
        scale = power(torch.where(top > 0, e, -126).clamp(-126, 127))
    else:
        scale = (top / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    v = (x / scale[..., None]).abs()
    # halfway values go to the code whose last bit is 0
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75)
            + (v > 2.5) + (v >= 3.5) + (v > 5.0)).to(torch.uint8)
    code = code | (torch.signbit(x).to(torch.uint8) << 3)
    return code.view(rows, -1)[:, :K], scale


def values(code, scale, fmt):
    """What codes [rows, K] with block scales [rows, blocks] stand for, in 32 bits."""
    K = code.shape[-1]
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=code.device)
    return grid[code.long()] * scale.repeat_interleave(BLOCK[fmt], -1)[..., :K]


def scale_code(scale, fmt):
    """The byte that a block scale is kept in."""
    if fmt == "mx":
        return (torch.frexp(scale).exponent + 126).to(torch.uint8)
    return scale.to(torch.float8_e4m3fn).view(torch.uint8)


def unpack(q, s, rows, K, fmt):
    """The values of weights kept in 4 bits: q [.., rows, bytes], s scale tiles."""
    q = q.reshape(-1, rows, q.shape[-1])
    code = torch.stack((q & 15, q >> 4), -1).flatten(2)[..., :K]
    tiles = -(-K // (4 * BLOCK[fmt]))
    byte = s.view(q.shape[0], -1, tiles, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(q.shape[0], -1, tiles * 4)[:, :rows]
    scale = power(byte.int() - 127) if fmt == "mx" else byte.contiguous().view(torch.float8_e4m3fn).float()
    return values(code, scale, fmt)


def spread(x, s):
    """Rows of x in 32 bits, group by group and padded with zeros: [G, most, columns]."""
    begin = s["offsets"].long()
    at = begin[:-1, None] + torch.arange(s["most"], device="cuda")
    inside = at < begin[1:, None]
    return x.float()[at.clamp(max=x.shape[0] - 1)] * inside[..., None]


def gather(x, s, M):
    """The rows of a [G, most, columns] product, back in their order."""
    begin = s["offsets"].long()
    i = torch.arange(M, device="cuda")
    group = torch.searchsorted(begin, i, right=True) - 1
    return x[group, i - begin[group]]


def swiglu(h):
    g, u = h[..., 0::2], h[..., 1::2]
    return g * torch.sigmoid(g) * u


def run(state):
    if own:
        return run_own(state)
    s, c = state, state["case"]
    op, M, K = c["op"], c["M"], c["K"]
    if op == "gemm":
        b = s["B"].float()
        return gather(torch.bmm(spread(s["A"], s), b if c["trans"] == 0 else b.transpose(1, 2)), s, M).to(TYPES[c["out"]])
    if op == "wgrad":
        return torch.bmm(spread(s["A"], s).transpose(1, 2), spread(s["D"], s)).to(TYPES[c["out"]])
    if op == "swiglu":
        return gather(swiglu(torch.bmm(spread(s["A"], s), s["W"].float())), s, M).to(torch.bfloat16)
    if op == "dswiglu":
        h = gather(torch.bmm(spread(s["A"], s), s["W"].float()), s, M)
        g, u, d = h[:, 0::2], h[:, 1::2], s["dY"].float()
        sg = torch.sigmoid(g)
        dh = torch.stack((d * u * sg * (1 + g * (1 - sg)), d * g * sg), -1).flatten(1)
        return {"dH": dh.to(torch.bfloat16), "Y": (g * sg * u).to(torch.bfloat16)}
    x = values(*quantise(s["X"], c["fmt"]), c["fmt"])
    if op == "round":
        return x.to(torch.bfloat16)
    if op == "linear":
        w = unpack(s["W"], s["SW"], c["N"], K, c["fmt"])[0]
        return (s["alpha"] * (x @ w.t())).to(TYPES[c["out"]])
    w = unpack(s["W"], s["SW"], 2 * c["N"], K, c["fmt"])
    return gather(swiglu(s["alpha"] * torch.bmm(spread(x, s), w.transpose(1, 2))), s, M).to(torch.bfloat16)


# ------------------------------------------------------- framework's calls

def run_own(s):
    import swiglu_mlp_gb300 as swg
    c = s["case"]
    op = c["op"]
    if op == "gemm":
        return swg.gemm_grouped_into(s["C"], s["A"], s["B"], s["offsets"], transB=c["trans"])
    if op == "wgrad":
        return swg.gemm_grouped_wgrad_into(s["C"], s["A"], s["D"], s["offsets"])
    if op == "swiglu":
        return swg.swiglu_grouped_into(s["Y"], s["A"], s["W"], s["offsets"])
    if op == "dswiglu":
        swg.swiglu_grouped_grad_into(s["dH"], s["A"], s["W"], s["dY"], s["offsets"], Y=s["Y"])
        return {"dH": s["dH"], "Y": s["Y"]}
    fmt = swg.MXFP4 if c["fmt"] == "mx" else swg.NVFP4
    off = s.get("offsets")
    swg.mx4_quantize_into(s["Q"], s["S"], s["X"], fmt, offsets=off)
    if op == "round":
        return swg.mx4_dequantize_into(s["V"], s["Q"], s["S"], fmt)
    if op == "linear":
        return swg.gemm_mx4_into(s["C"], s["Q"], s["S"], s["W"], s["SW"], c["K"], fmt, alpha=s["alpha"])
    return swg.swiglu_mx4_into(s["Y"], s["Q"], s["S"], s["W"], s["SW"], c["K"], fmt, alpha=s["alpha"], offsets=off)


# ------------------------------------------------------------- work, exact

def work(case):
    """What one pass cannot do without: each input read once (of the weights
    those of groups that have rows), each output written once."""
    op, M, K, N, G = case["op"], case["M"], case["K"], case.get("N", 0), case.get("G", 1)
    used = int((rows_of(case) > 0).sum()) if "G" in case else 1
    bits = 0.5 + 1.0 / BLOCK[case["fmt"]] if "fmt" in case else 0
    if op == "gemm":
        return {"bytes": 2 * M * K + 2 * used * K * N + 2 * M * N, "flops": 2 * M * N * K}
    if op == "wgrad":
        return {"bytes": 2 * M * (K + N) + 2 * G * K * N, "flops": 2 * M * N * K}
    if op == "swiglu":
        return {"bytes": 2 * M * K + 4 * used * K * N + 2 * M * N, "flops": 4 * M * N * K}
    if op == "dswiglu":
        return {"bytes": 2 * M * K + 4 * used * K * N + 8 * M * N, "flops": 4 * M * N * K}
    if op == "round":  # x in, 4 bits and scales out, values out
        return {"bytes": M * K * (4 + bits), "flops": 4 * M * K}
    if op == "linear":
        return {"bytes": 2 * M * K + bits * N * K + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": 2 * M * K + 2 * bits * used * N * K + 2 * M * N, "flops": 4 * M * N * K}


def exact(case, seed):
    """From the definitions, in 64 bits, group after group."""
    s = prepare(case, seed)
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N", 0)
    if op in ("round", "linear", "mlp4"):
        x = rounded_64(s["X"], case["fmt"])
        if op == "round":
            return x
    else:
        x = s["A"].double()
    end = np.concatenate([[0], np.cumsum(rows_of(case))]) if "G" in case else np.array([0, M])

    def weight(g):
        if op == "gemm":
            b = s["B"][g].double()
            return b if case["trans"] == 0 else b.t()
        if op in ("swiglu", "dswiglu"):
            return s["W"][g].double()
        rows = N if op == "linear" else 2 * N
        w = s["W"] if op == "linear" else s["W"][g]
        return weight_64(w, s["SW"], g, rows, K, case["fmt"]).t()

    parts = []
    for g in range(len(end) - 1):
        xg = x[end[g]:end[g + 1]]
        if op == "wgrad":
            parts.append(xg.t() @ s["D"][end[g]:end[g + 1]].double())
        elif len(xg):
            parts.append(xg @ weight(g) * (s["alpha"] if "alpha" in s else 1.0))
    if op == "wgrad":
        return torch.stack(parts)
    h = torch.cat(parts)
    if op in ("gemm", "linear"):
        return h
    gate, up = h.unflatten(1, (N, 2)).unbind(-1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if op != "dswiglu":
        return gate * sig * up
    d = s["dY"].double()
    dg = d * up * (sig + gate * sig * (1.0 - sig))
    return {"dH": torch.stack((dg, d * gate * sig), 2).flatten(1), "Y": gate * sig * up}


def power_64(e):
    """2^e for whole numbers e from -1022 to 1023, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def rounded_64(x, fmt):
    """x on the grid of its blocks: steps of 1/2 up to 2, 1 up to 4, 2 up to 6,
    ties to even, in units of the block scale."""
    b = BLOCK[fmt]
    rows, K = x.shape
    x = torch.cat((x.double(), x.new_zeros((rows, -K % b)).double()), 1).view(rows, -1, b)
    top = x.abs().max(-1).values
    if fmt == "mx":
        scale = power_64(torch.where(top > 0, torch.frexp(top).exponent - 3, 0))
    else:  # e4m3: three fraction bits, steps of 2^-9 below 2^-6, at most 448
        t = top / 6.0
        step = power_64(torch.frexp(t.clamp(min=2.0 ** -6)).exponent - 4)
        scale = (torch.round(t / step) * step).clamp(2.0 ** -9, 448.0)
    v = x / scale[..., None]
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(v) * a * scale[..., None]).view(rows, -1)[:, :K]


def weight_64(q, tiles, g, rows, K, fmt):
    """Group g's weight in 64 bits, read element by element of the layout above."""
    b = BLOCK[fmt]
    r = torch.arange(rows, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    code = (q[r, k // 2].long() >> (4 * (k % 2))) & 15
    across = -(-K // (4 * b))
    tile = (g * -(-rows // 128) + r // 128) * across + k // (4 * b)
    byte = tiles[tile * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + k // b % 4].double()
    if fmt == "mx":
        scale = power_64(byte - 127)
    else:
        e, m = torch.floor(byte / 8), byte % 8
        scale = torch.where(e > 0, (8 + m) * power_64(e - 10), m * 2.0 ** -9)
    e, m = (code >> 1) & 3, (code & 1).double()
    size = torch.where(e > 0, (2 + m) * power_64(e - 2), m / 2)
    return torch.where(code >= 8, -size, size) * scale
