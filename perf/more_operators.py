"""Cases of the operators around the expert products: the router and its plan
of rows, moving rows to the experts and back, and products with weights of 4
bits and group scales.

A case's ``op``:

* ``route``    scores of T tokens over E experts, the ``top`` best of each, their
               weights, and the plan: rows sorted by expert.  ``grad``: and the
               gradient of the logits from that of the weights.
* ``dispatch`` each token's row to the places that the plan gives it.
* ``combine``  a token's rows, weighted, summed.  ``grad``: and the gradients of
               rows and weights.
* ``linear``   C = A W^T for few rows, W in 4 bits (``G``: rows by expert).
* ``swiglu``   Y = SiLU(A W1^T) * (A W2^T), rows of W1 and W2 alternating.
* ``round``    a weight to 4 bits, and the values those stand for.
* ``layer``    route, dispatch, swiglu, linear and combine: a decoded expert layer.

Plan: ``offsets`` [E + 1], where each expert's rows begin; ``source`` [T * top],
the flat index t * top + j that row r comes from, rows of an expert in that
order, -1 behind the last; ``position`` [T, top], the other way, -1 where a slot
has no expert.  An expert whose logit is -inf is not chosen.

4-bit weights: w[n, k] = s[k // g, n] * (q[n, k] - z[k // g, n]), z = 8 where it is not
stored.  Eight codes of a row are a 32-bit word: columns 0, 2, 4, 6 in bits 0, 4, 8,
12 and columns 1, 3, 5, 7 in bits 16, 20, 24, 28.  Rows are a multiple of 32 codes,
s and z rows a multiple of 16 values.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    """Real work over the range of sizes, types and directions."""
    return [
        # four decoded tokens: the latency of a router
        dict(name="route_decode", op="route", T=4, E=64, top=6, score="softmax", bias=0, groups=1, top_groups=1, sum=1, norm=1, scale=1.0, type="bf16", pad=0, grad=0),
        # prefill: sigmoid scores with a balancing bias, four of eight groups of experts, the batch's last rows padding
        dict(name="route_prefill", op="route", T=16384, E=256, top=8, score="sigmoid", bias=1, groups=8, top_groups=4, sum=2, norm=1, scale=2.5, type="f32", pad=300, grad=0),
        # a training step's router, forward and backward
        dict(name="route_train", op="route", T=8192, E=16, top=2, score="softmax", bias=0, groups=1, top_groups=1, sum=1, norm=1, scale=1.0, type="bf16", pad=0, grad=1),
        # rows of 8192 tokens to two of 16 experts each
        dict(name="dispatch_prefill", op="dispatch", T=8192, D=4096, E=16, top=2, type="bf16", route=3, skew=0.5, pad=0),
        # 32 decoded tokens' results of eight experts each
        dict(name="combine_decode", op="combine", T=32, D=4096, E=64, top=8, type="bf16", route=4, skew=0.5, pad=0, grad=0),
        # a training step's, at an odd width in fp16, with padding tokens
        dict(name="combine_train_odd", op="combine", T=5003, D=2051, E=48, top=4, type="f16", route=5, skew=0.8, pad=70, grad=1),
        # one decoded token through a layer of the 8B-class model
        dict(name="linear_decode", op="linear", M=1, K=4096, N=14336, G=0, g=128, zero=0, type="bf16", out="bf16"),
        # a small batch through its down projection, zero points, fp16
        dict(name="linear_batch", op="linear", M=32, K=14336, N=4096, G=0, g=64, zero=1, type="f16", out="f32"),
        # 64 rows over 64 fine-grained experts, some of them empty
        dict(name="swiglu_experts", op="swiglu", M=64, K=896, N=1216, G=64, g=32, zero=0, type="bf16", route=6, skew=0.7),
        # a weight of the 8B-class model to 4 bits and back
        dict(name="round_weight", op="round", N=14336, K=4096, g=128, zero=0, type="bf16"),
        # an odd one, with zero points
        dict(name="round_odd", op="round", N=1003, K=2051, g=64, zero=1, type="f16"),
        # eight decoded tokens through an expert layer, two of 16 experts each
        dict(name="layer_decode", op="layer", T=8, E=16, top=2, D=4096, H=1792, g=128, zero=0, type="bf16"),
    ]


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest of them."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "route", "dispatch", "combine", "linear", "linear", "swiglu", "round", "layer"])
    half = rng.choice(["bf16", "f16"])
    while True:
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            c = dict(op=op, T=log(1, 16384), E=groups * log(2, 512 // groups), score=rng.choice(["softmax", "sigmoid"]), bias=rng.randrange(2),
                     groups=groups, top_groups=rng.randint(1, groups), sum=rng.choice([1, 2]), norm=rng.randrange(2), scale=rng.choice([1.0, 2.5]),
                     type=rng.choice(["bf16", "f16", "f32"]), grad=rng.randrange(2))
            c["top"] = rng.randint(1, min(8, c["E"] // groups * c["top_groups"]))
            c["pad"] = rng.choice([0, c["T"] // 8])
        elif op in ("dispatch", "combine"):
            c = dict(op=op, T=log(1, 16384), D=log(64, 8192), E=log(8, 256), top=rng.randint(1, 8), type=rng.choice([half, half, "f32"]),
                     route=rng.randrange(10 ** 6), skew=rng.choice([0.0, 0.5, 1.0]))
            c["pad"] = rng.choice([0, c["T"] // 8])
            if op == "combine":
                c["grad"] = rng.randrange(2)
        elif op in ("linear", "swiglu"):
            c = dict(op=op, M=log(1, 64), K=log(64, 16384), N=8 * log(8, 2048), G=rng.choice([0, log(2, 128)]) if op == "linear" else log(1, 128),
                     g=rng.choice([32, 64, 128]), zero=rng.randrange(2), type=half)
            if op == "linear":
                c["out"] = rng.choice([half, "f32"])
            if c["G"]:
                c.update(route=rng.randrange(10 ** 6), skew=rng.choice([0.0, 0.5, 1.0]))
        elif op == "round":
            c = dict(op=op, N=log(1, 14336), K=log(32, 8192), g=rng.choice([32, 64, 128]), zero=rng.randrange(2), type=half)
        else:
            c = dict(op=op, T=log(1, 32), E=log(8, 64), top=rng.randint(1, 4), D=8 * log(16, 512), H=8 * log(16, 256), g=rng.choice([32, 64, 128]),
                     zero=rng.randrange(2), type=half)
        most = max(c.get("G", 1), 1) * c.get("N", 1) * c.get("K", 1) * (2 if op == "swiglu" else 1)
        most = max(most, c["E"] * c["D"] * c["H"] * 3 if op == "layer" else 0)
        if work(c)["bytes"] <= 2.0e8 and most <= 2 ** 28:
            return c


# ------------------------------------------------------------------ inputs

def pad_to(x, m):
    return -(-x // m) * m


def normal(shape, g, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def rows_in(rows, cols, g, std, dtype):
    """A rows x cols matrix in storage whose row length is a multiple of 16 bytes."""
    return normal((rows, pad_to(cols, 8)), g, std, dtype)[:, :cols]


def room(rows, cols, dtype):
    return torch.zeros((rows, pad_to(cols, 8)), dtype=dtype, device="cuda")[:, :cols]


def rows_of(case):
    """Rows of each expert: a draw of the router's kind, some more wanted than
    others (``skew``), from the case alone."""
    r = np.random.RandomState(case["route"])
    p = (1.0 + np.arange(case["G"])) ** -case["skew"]
    return r.multinomial(case["M"], r.permutation(p / p.sum()))


def logits_of(T, E, g, dtype, pad):
    """A router's logits: tokens agree in part on what they want."""
    x = torch.randn((T, E), generator=g, device="cuda") * 1.5 + torch.randn((1, E), generator=g, device="cuda") * 0.5
    x = x.to(dtype)
    if pad:
        x[-pad:] = float("-inf")
    return x


def chosen(case, g):
    """The experts [T, top] that a router chose, all different, -1 for padding tokens."""
    T, E, top = case["T"], case["E"], min(case["top"], case["E"])
    r = np.random.RandomState(case["route"])
    p = (1.0 + np.arange(E)) ** -case["skew"]
    want = torch.from_numpy(r.permutation(p / p.sum())).float().cuda().log()
    u = torch.rand((T, E), generator=g, device="cuda")
    e = (want - (-u.clamp(min=1e-7).log()).log()).topk(top, -1).indices.int()
    if case["top"] > E:
        e = torch.cat((e, torch.full((T, case["top"] - E), -1, dtype=torch.int32, device="cuda")), 1)
    if case["pad"]:
        e[-case["pad"]:] = -1
    return e.contiguous()


def weight_4bit(groups, rows, K, g, case):
    """A weight in hand: codes, scales and zero points, quantised from N(0, 0.02)
    with a mean of its own in each row."""
    x = torch.randn((groups * rows, K), generator=g, device="cuda") * 0.02
    x = x + torch.randn((groups * rows, 1), generator=g, device="cuda") * 0.004
    q, s, z = quantise(x, case["g"], case["zero"], TYPES[case["type"]])
    blocks = s.shape[1]
    S = torch.zeros((groups, blocks, pad_to(rows, 16)), dtype=s.dtype, device="cuda")
    S[:, :, :rows] = s.view(groups, rows, blocks).transpose(1, 2)
    Z = None
    if case["zero"]:
        Z = torch.zeros(S.shape, dtype=torch.uint8, device="cuda")
        Z[:, :, :rows] = z.view(groups, rows, blocks).transpose(1, 2)
    return pack(q).view(groups, rows, -1), S, Z


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=case)
    op = case["op"]
    t = TYPES[case["type"]]
    if op == "route":
        T, E, top = case["T"], case["E"], case["top"]
        s["logits"] = logits_of(T, E, g, t, case["pad"])
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
        s["experts"] = torch.empty((T, top), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((T, top), dtype=torch.float32, device="cuda")
        s["plan"] = room_for_plan(T, E, top)
        if case["grad"]:
            s["d_weights"] = torch.randn((T, top), generator=g, device="cuda")
            s["d_logits"] = torch.empty_like(s["logits"])
    elif op in ("dispatch", "combine"):
        T, D, top = case["T"], case["D"], case["top"]
        s["position"] = plan_of(chosen(case, g), case["E"])[2]
        if op == "dispatch":
            s["X"] = rows_in(T, D, g, 1.0, t)
            s["rows"] = room(T * top, D, t)
        else:
            s["rows"] = rows_in(T * top, D, g, 1.0, t)
            s["weights"] = torch.rand((T, top), generator=g, device="cuda") * 0.9 + 0.1
            s["out"] = room(T, D, t)
            if case["grad"]:
                s["d_out"] = rows_in(T, D, g, 1.0, t)
                s["d_rows"] = room(T * top, D, t)
                s["d_weights"] = torch.empty((T, top), dtype=torch.float32, device="cuda")
    elif op in ("linear", "swiglu"):
        M, K, N, G = case["M"], case["K"], case["N"], case["G"]
        if G:
            n = rows_of(case)
            s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
            s["most"] = int(n.max())
        s["A"] = rows_in(M, K, g, 1.0, t)
        s["W"] = weight_4bit(max(G, 1), N if op == "linear" else 2 * N, K, g, case)
        s["C"] = room(M, N, TYPES[case["out"]] if op == "linear" else t)
    elif op == "round":
        N, K = case["N"], case["K"]
        s["X"] = rows_in(N, K, g, 0.02, t)
        s["V"] = room(N, K, t)
        s["W"] = room_for_weight(N, K, case)
    else:
        T, E, top, D, H = case["T"], case["E"], case["top"], case["D"], case["H"]
        s["X"] = normal((T, D), g, 1.0, t)
        s["logits"] = logits_of(T, E, g, torch.float32, 0)
        s["up"] = weight_4bit(E, 2 * H, D, g, case)
        s["down"] = weight_4bit(E, D, H, g, case)
        s["experts"] = torch.empty((T, top), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((T, top), dtype=torch.float32, device="cuda")
        s["plan"] = room_for_plan(T, E, top)
        s["rows"], s["Y"], s["Z"] = (torch.zeros((T * top, d), dtype=t, device="cuda") for d in (D, H, D))
        s["out"] = torch.zeros((T, D), dtype=t, device="cuda")
    return s


def room_for_plan(T, E, top):
    """Where a call writes the plan: offsets, source, position."""
    return tuple(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * top, (T, top)))


def room_for_weight(N, K, case):
    blocks = -(-K // case["g"])
    S = torch.zeros((1, blocks, pad_to(N, 16)), dtype=TYPES[case["type"]], device="cuda")
    Z = torch.zeros(S.shape, dtype=torch.uint8, device="cuda") if case["zero"] else None
    return torch.zeros((1, N, pad_to(K, 32) // 2), dtype=torch.uint8, device="cuda"), S, Z


# -------------------------------------------------------------- plain form

def route(logits, bias, c):
    """(experts, weights, scores of all, in 64 bits: choices may be next to one another)."""
    x = logits.double()
    masked = torch.isneginf(x)
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
        score = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = x if bias is None and c["sum"] == 1 else score if bias is None else score + bias.double()
    low = float("-inf")
    choice = choice.masked_fill(masked, low)
    if c["groups"] > 1:
        of = choice.unflatten(-1, (c["groups"], -1))
        best = of.sort(dim=-1, descending=True).values[..., :c["sum"]]
        best = torch.where(best.isneginf(), 0.0, best).sum(-1).masked_fill(best[..., 0].isneginf(), low)
        rank = best.sort(dim=-1, descending=True, stable=True).indices.argsort(-1)
        choice = of.masked_fill((rank >= c["top_groups"])[..., None], low).flatten(-2)
    value, expert = choice.sort(dim=-1, descending=True, stable=True)
    value, expert = value[:, :c["top"]], expert[:, :c["top"]]
    none = value.isneginf()
    w = score.gather(-1, expert).masked_fill(none, 0.0)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return expert.int().masked_fill(none, -1), (w * c["scale"]).float(), score


def route_grad(score, expert, d_weights, c):
    """The gradient of the logits, in 64 bits like the scores."""
    none = expert < 0
    at = expert.long().clamp(min=0)
    s = score.gather(-1, at).masked_fill(none, 0.0)
    d = d_weights.double().masked_fill(none, 0.0) * c["scale"]
    if c["norm"]:
        total = s.sum(-1, keepdim=True).clamp(min=1e-300)
        d = (d - (d * s).sum(-1, keepdim=True) / total) / total
    g = torch.zeros_like(score).scatter_add_(-1, at, d.masked_fill(none, 0.0))
    if c["score"] == "softmax":
        return score * (g - (g * score).sum(-1, keepdim=True))
    return g * score * (1.0 - score)


def plan_of(experts, E):
    """offsets, source, position of rows sorted by expert."""
    flat = torch.where(experts < 0, E, experts).flatten().long()
    order = flat.argsort(stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((count.new_zeros(1), count[:E].cumsum(0)))
    row = torch.arange(len(flat), device="cuda")
    position = torch.empty_like(flat).scatter_(0, order, row)
    return (offsets.int(), torch.where(row < offsets[E], order, -1).int(),
            torch.where(flat < E, position, -1).int().view(experts.shape))


def dispatch(rows, X, position):
    """rows, those that the plan fills replaced."""
    at = position.flatten().long()
    spare = torch.cat((rows, rows[:1]))
    x = X.unsqueeze(1).expand(-1, position.shape[1], -1).flatten(0, 1)
    return spare.index_copy_(0, torch.where(at < 0, len(rows), at), x)[:-1]


def taken(rows, position):
    """Each slot's row in 32 bits, zeros where it has none: [T, top, D]."""
    return rows.float()[position.long().clamp(min=0)].masked_fill((position < 0)[..., None], 0.0)


def quantise(x, g, zero, dtype):
    """Codes [rows, K], scales and zero points [rows, blocks], in 32 bits."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, pad_to(K, g) - K)).view(rows, -1, g)
    if zero:
        lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / torch.full_like(hi, 15.0)).to(dtype).float()  # (divided by a number, torch multiplies by its inverse)
        z = torch.where(s > 0, torch.round(-lo / s), 0.0).clamp(0, 15)
    else:
        top = x.abs().amax(-1)
        s = (top / torch.full_like(top, 7.0)).to(dtype).float()
        z = torch.full_like(s, 8.0)
    q = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), 0.0) + z[..., None]
    return q.clamp(0, 15).view(rows, -1)[:, :K].to(torch.uint8), s.to(dtype), z.to(torch.uint8)


def pack(q):
    """Codes [rows, K] to bytes, even columns of eight in the lower half of their word."""
    rows, K = q.shape
    q = torch.nn.functional.pad(q, (0, pad_to(K, 32) - K)).view(rows, -1, 2, 2, 2)
    return (q[..., 0, :] | (q[..., 1, :] << 4)).transpose(2, 3).reshape(rows, -1)


def unpack(W, rows, K, g):
    """The values of weights kept in 4 bits, [groups, rows, K] in 32 bits."""
    Q, S, Z = W
    b = Q.view(Q.shape[0], rows, -1, 2, 2)
    q = torch.stack((b & 15, b >> 4), -1).flatten(-2).transpose(-1, -2).flatten(2)[..., :K].float()
    s = S[:, :, :rows].transpose(1, 2).float().repeat_interleave(g, -1)[..., :K]
    z = 8.0 if Z is None else Z[:, :, :rows].transpose(1, 2).float().repeat_interleave(g, -1)[..., :K]
    return s * (q - z)


def spread(x, begin, most):
    """Rows of x in 32 bits, expert by expert and padded with zeros: [G, most, columns]."""
    at = begin[:-1, None].long() + torch.arange(most, device="cuda")
    return x.float()[at.clamp(max=x.shape[0] - 1)] * (at < begin[1:, None])[..., None]


def gather(x, begin, M):
    """The rows of a [G, most, columns] product, back in their order."""
    i = torch.arange(M, device="cuda")
    group = (torch.searchsorted(begin.long(), i, right=True) - 1).clamp(max=len(begin) - 2)
    return x[group, (i - begin[group]).clamp(max=x.shape[1] - 1)]


def swiglu(h):
    g, u = h[..., 0::2], h[..., 1::2]
    return g * torch.sigmoid(g) * u


def run(state):
    if own:
        return run_own(state)
    s, c = state, state["case"]
    op = c["op"]
    t = TYPES[c["type"]]
    if op == "route":
        experts, weights, score = route(s["logits"], s["bias"], c)
        out = (experts, weights) + plan_of(experts, c["E"])
        return out + (route_grad(score, experts, s["d_weights"], c).to(t),) if c["grad"] else out
    if op == "dispatch":
        return dispatch(s["rows"], s["X"], s["position"])
    if op == "combine":
        rows = taken(s["rows"], s["position"])
        out = (rows * s["weights"][..., None]).sum(1).to(t)
        if not c["grad"]:
            return out
        d = s["d_out"].float()[:, None]
        d_rows = dispatch_each(s["d_rows"], (d * s["weights"][..., None]).to(t), s["position"])
        return out, d_rows, (rows * d).sum(-1)
    if op == "round":
        Q, S, Z = s["W"]
        q, scale, z = quantise(s["X"], c["g"], c["zero"], t)
        step = scale.float().repeat_interleave(c["g"], -1)[:, :c["K"]]
        return (step * (q.float() - z.float().repeat_interleave(c["g"], -1)[:, :c["K"]])).to(t)
    if op in ("linear", "swiglu"):
        M, K, rows = c["M"], c["K"], c["N"] * (1 if op == "linear" else 2)
        w = unpack(s["W"], rows, K, c["g"])
        if c["G"]:
            h = gather(torch.bmm(spread(s["A"], s["offsets"], s["most"]), w.transpose(1, 2)), s["offsets"], M)
        else:
            h = s["A"].float() @ w[0].t()
        return (h if op == "linear" else swiglu(h)).to(s["C"].dtype)
    experts, weights, _ = route(s["logits"], None, layer_router(c))
    begin, source, position = plan_of(experts, c["E"])
    x = s["X"][source.long().clamp(min=0) // c["top"]]
    h = swiglu(torch.bmm(spread(x, begin, c["T"]), unpack(s["up"], 2 * c["H"], c["D"], c["g"]).transpose(1, 2)))
    rows = gather(torch.bmm(h, unpack(s["down"], c["D"], c["H"], c["g"]).transpose(1, 2)), begin, len(x))
    return experts, weights, (taken(rows, position) * weights[..., None]).sum(1).to(t)


def dispatch_each(rows, x, position):
    """rows, those of the slots replaced by x [T, top, D]."""
    at = position.flatten().long()
    return torch.cat((rows, rows[:1])).index_copy_(0, torch.where(at < 0, len(rows), at), x.flatten(0, 1))[:-1]


def layer_router(c):
    return dict(score="softmax", sum=1, groups=1, top_groups=1, top=c["top"], norm=1, scale=1.0)


# ------------------------------------------------------- framework's calls

def run_own(s):
    import swiglu_mlp_gb300 as swg
    c = s["case"]
    op = c["op"]
    if op == "route":
        score = swg.SOFTMAX if c["score"] == "softmax" else swg.SIGMOID
        swg.expert_route_into(s["experts"], s["weights"], s["logits"], score, bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                              group_sum=c["sum"], normalise=bool(c["norm"]), scale=c["scale"], plan=s["plan"])
        out = (s["experts"], s["weights"]) + s["plan"]
        if not c["grad"]:
            return out
        return out + (swg.expert_route_grad_into(s["d_logits"], s["d_weights"], s["logits"], s["experts"], score,
                                                 normalise=bool(c["norm"]), scale=c["scale"]),)
    if op == "dispatch":
        return swg.expert_dispatch_into(s["rows"], s["X"], s["position"])
    if op == "combine":
        out = swg.expert_combine_into(s["out"], s["rows"], s["position"], s["weights"])
        if not c["grad"]:
            return out
        swg.expert_combine_grad_into(s["d_rows"], s["d_weights"], s["d_out"], s["rows"], s["position"], s["weights"])
        return out, s["d_rows"], s["d_weights"]
    if op == "round":
        swg.w4_quantize_into(*s["W"], s["X"], c["g"])
        return swg.w4_dequantize_into(s["V"], *s["W"], c["g"])
    if op == "linear":
        return swg.gemm_w4_into(s["C"], s["A"], *s["W"], c["g"], offsets=s.get("offsets"))
    if op == "swiglu":
        return swg.swiglu_w4_into(s["C"], s["A"], *s["W"], c["g"], offsets=s.get("offsets"))
    swg.expert_route_into(s["experts"], s["weights"], s["logits"], swg.SOFTMAX, plan=s["plan"])
    offsets, _, position = s["plan"]
    swg.expert_dispatch_into(s["rows"], s["X"], position)
    swg.swiglu_w4_into(s["Y"], s["rows"], *s["up"], c["g"], offsets=offsets)
    swg.gemm_w4_into(s["Z"], s["Y"], *s["down"], c["g"], offsets=offsets)
    return s["experts"], s["weights"], swg.expert_combine_into(s["out"], s["Z"], position, s["weights"])


# ------------------------------------------------------------- work, exact

def work(case):
    """What one pass cannot do without: each input read once (of the experts'
    weights those of experts that have rows), each output written once."""
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    if op == "route":
        T, E, top = case["T"], case["E"], case["top"]
        grad = size * T * E + 4 * T * top if case["grad"] else 0
        return {"bytes": size * T * E + 16 * T * top + 4 * (E + 1) + grad, "flops": 8 * T * E}
    if op in ("dispatch", "combine"):
        T, D, top = case["T"] - case["pad"], case["D"], min(case["top"], case["E"])
        rows = size * T * top * D
        moved = size * T * D + rows + 4 * T * top
        if case.get("grad"):  # d_out in and d_rows out; the rows are read once
            return {"bytes": moved + size * T * D + rows + 8 * T * top, "flops": 5 * T * top * D}
        return {"bytes": moved + (4 * T * top if op == "combine" else 0), "flops": 2 * T * top * D}
    bits = 0.5 + (2.0 + case["zero"]) / case["g"]
    if op == "round":  # x in, codes out and in again, values out
        return {"bytes": case["N"] * case["K"] * (4 + 2 * bits), "flops": 6 * case["N"] * case["K"]}
    if op == "layer":
        T, E, top, D, H = case["T"], case["E"], case["top"], case["D"], case["H"]
        used = E * (1.0 - (1.0 - min(top, E) / E) ** T)
        return {"bytes": 3 * used * D * H * bits + 4 * T * D + 4 * T * E + 8 * T * top, "flops": 6 * T * top * D * H}
    M, K, N, G = case["M"], case["K"], case["N"] * (1 if op == "linear" else 2), case["G"]
    used = int((rows_of(case) > 0).sum()) if G else 1
    out = {"bf16": 2, "f16": 2, "f32": 4}[case.get("out", case["type"])] * case["N"]
    return {"bytes": used * N * K * bits + M * (2 * K + out), "flops": 2 * M * N * K}


def weight_64(W, expert, rows, K, g):
    """An expert's weight in 64 bits, read element by element of the layout above."""
    Q, S, Z = W
    n = torch.arange(rows, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    bit = 16 * (k % 2) + 4 * (k % 8 // 2)
    q = (Q[expert][n, k // 8 * 4 + bit // 8].long() >> (bit % 8)) & 15
    z = 8 if Z is None else Z[expert][k // g, n].long()
    return S[expert][k // g, n].double() * (q - z).double()


def exact(case, seed):
    """From the definitions, in 64 bits; whole numbers have no other value."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        want = s["rows"].double()
        slots = (s["position"] >= 0).nonzero()
        want[s["position"][slots[:, 0], slots[:, 1]].long()] = s["X"].double()[slots[:, 0]]
        return want
    if op == "route":
        experts = chosen_64(s["logits"], s["bias"], case)
        out = (None, weights_64(s["logits"], experts, case), None, None, None)
        return out + (grad_64(s["logits"], experts, s["d_weights"], case),) if case["grad"] else out
    if op == "combine":
        T, top = s["position"].shape
        out = torch.zeros((T, case["D"]), dtype=torch.float64, device="cuda")
        d_rows, d_w = (s["d_rows"].double(), torch.zeros((T, top), dtype=torch.float64, device="cuda")) if case["grad"] else (None, None)
        for j in range(top):
            on = (s["position"][:, j] >= 0).nonzero()[:, 0]
            at = s["position"][on, j].long()
            w = s["weights"][on, j].double()[:, None]
            out[on] += w * s["rows"][at].double()
            if case["grad"]:
                d_rows[at] = w * s["d_out"][on].double()
                d_w[on, j] = (s["rows"][at].double() * s["d_out"][on].double()).sum(1)
        return (out, d_rows, d_w) if case["grad"] else out
    if op == "round":
        return rounded_64(s["X"], case)
    if op == "layer":
        experts = chosen_64(s["logits"], None, layer_router(case))
        w = weights_64(s["logits"], experts, layer_router(case))
        out = torch.zeros(s["X"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            token, slot = (experts == e).nonzero(as_tuple=True)
            if len(token):
                h = s["X"][token].double() @ weight_64(s["up"], e, 2 * case["H"], case["D"], case["g"]).t()
                y = h[:, 0::2] / (1.0 + torch.exp(-h[:, 0::2])) * h[:, 1::2]
                y = y @ weight_64(s["down"], e, case["D"], case["H"], case["g"]).t()
                out.index_add_(0, token, y * w[token, slot][:, None])
        return None, w, out
    rows = case["N"] * (1 if op == "linear" else 2)
    end = np.concatenate([[0], np.cumsum(rows_of(case))]) if case["G"] else np.array([0, case["M"]])
    parts = [s["A"][end[e]:end[e + 1]].double() @ weight_64(s["W"], e, rows, case["K"], case["g"]).t()
             for e in range(len(end) - 1) if end[e + 1] > end[e]]
    h = torch.cat(parts)
    return h if op == "linear" else h[:, 0::2] / (1.0 + torch.exp(-h[:, 0::2])) * h[:, 1::2]


def best_64(value, count, still):
    """The places of the `count` largest of each row, one after the other, the first of equals;
    -1 where none is left of those `still` in it."""
    place = torch.arange(value.shape[-1], device="cuda").expand_as(value)
    found = []
    for _ in range(count):
        top = torch.where(still, value, float("-inf")).amax(-1, keepdim=True)
        at = torch.where(still & (value == top), place, value.shape[-1]).amin(-1, keepdim=True)
        found.append(torch.where(at < value.shape[-1], at, -1))
        still = still & (place != at)
    return torch.cat(found, -1)


def chosen_64(logits, bias, c):
    """The experts by choice in 64 bits."""
    x = logits.double()
    value = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    if bias is not None:
        value = value + bias.double()
    elif c["sum"] == 1:
        value = x
    still = x > float("-inf")
    if c["groups"] > 1:
        shape = (x.shape[0], c["groups"], -1)
        of, on = value.reshape(shape), still.reshape(shape)
        at = best_64(of, min(c["sum"], of.shape[-1]), on)
        total = torch.where(at >= 0, of.gather(-1, at.clamp(min=0)), 0.0).sum(-1)
        groups = best_64(total, c["top_groups"], on.any(-1))
        kept = (groups[:, None, :] == torch.arange(c["groups"], device="cuda")[:, None]).any(-1)
        still = (on & kept[..., None]).reshape(x.shape)
    return best_64(value, c["top"], still).int()


def weights_64(logits, experts, c):
    """The chosen experts' weights, through logarithms of the scores."""
    x = logits.double()
    log = x - torch.logsumexp(x, -1, keepdim=True) if c["score"] == "softmax" else -torch.logaddexp(torch.zeros_like(x), -x)
    log = log.gather(1, experts.long().clamp(min=0)).masked_fill(experts < 0, float("-inf"))
    if c["norm"]:
        log = log - torch.logsumexp(log, -1, keepdim=True)
    return torch.where(experts < 0, 0.0, torch.exp(log)) * c["scale"]


def grad_64(logits, experts, d_weights, c):
    """The gradient of the logits by the Jacobian of the logarithms of the weights."""
    x = logits.double()
    none = experts < 0
    u = (weights_64(logits, experts, c) * d_weights.double()).masked_fill(none, 0.0)
    if c["norm"]:
        share = weights_64(logits, experts, dict(c, scale=1.0))
        u = u - share * u.sum(-1, keepdim=True)
    at = experts.long().clamp(min=0)
    if c["score"] == "softmax":
        g = torch.zeros_like(x).scatter_add_(1, at, u)
        if c["norm"]:
            return g
        p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)).nan_to_num(0.0)
        return g - p * u.sum(-1, keepdim=True)
    return torch.zeros_like(x).scatter_add_(1, at, u * (1.0 / (1.0 + torch.exp(x.gather(1, at)))).masked_fill(none, 0.0))


def rounded_64(X, case):
    """X on the grid of its groups: scales of the type's precision, codes by nearest, ties to even."""
    N, K = X.shape
    out = torch.empty((N, K), dtype=torch.float64, device="cuda")
    for k in range(0, K, case["g"]):
        x = X[:, k:k + case["g"]].double()
        if case["zero"]:
            lo, hi = x.amin(1, keepdim=True).clamp(max=0), x.amax(1, keepdim=True).clamp(min=0)
            s = ((hi - lo).float().double() / 15.0).float().to(X.dtype).double()
            z = torch.round(-lo / s).clamp(0, 15)
        else:
            s = (x.abs().amax(1, keepdim=True) / 7.0).float().to(X.dtype).double()
            z = torch.full_like(s, 8.0)
        out[:, k:k + case["g"]] = s * ((torch.round(x / s) + z).clamp(0, 15) - z)
    return out
