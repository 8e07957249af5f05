"""Operators of the experts' training step, as a user calls them, beside their plain forms.

Four operators:

* ``dgrad``: the gradient of the products grouped by expert with respect to their rows, dA = dC B per expert, with
  ragged row counts; with a gated activation the product is the gradient of the activation's output and the
  gradients of the gate and up projections (and the recomputed activation) come out of it.
* ``wgrad``: the gradient of the same products with respect to the experts' weights, dB[e] = dC_e^T A_e, the ragged
  row count being the summed axis; written in bf16 or fp32, or added to an fp32 buffer.
* ``combine``: the gradient of the weighted combine with respect to the experts' outputs and the routing weights.
* ``orth``: the orthogonalised update of a stack of weight matrices by Newton-Schulz products.

``own`` selects the framework's kernels; otherwise the operators run in elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

#: Coefficients (a, b, c) of the quintic Newton-Schulz step X <- a X + (b A + c A^2) X, A = X X^T.
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7

ACT = {"none": 0, "swiglu": 1, "geglu": 2, "reglu": 3}


def listed():
    return [
        # the tiny layer's down projection: a test-sized step, where a launch's latency is the cost
        {"name": "dgrad_tiny_gated", "op": "dgrad", "rows": 128, "E": 8, "N": 128, "K": 256, "act": "swiglu", "empty": 1},
        # Mixtral-shaped gate/up projections, 16 tokens to two experts each: the weights' bytes count
        {"name": "dgrad_mixtral_16_tokens", "op": "dgrad", "rows": 32, "E": 8, "N": 28672, "K": 4096, "act": "none", "empty": 0},
        # Mixtral-shaped down projection, 4096 tokens: the activation's gradient in the epilogue
        {"name": "dgrad_mixtral_gated", "op": "dgrad", "rows": 8192, "E": 8, "N": 4096, "K": 14336, "act": "swiglu", "empty": 0},
        # fine-grained gate/up projections, one rank's 64 experts, skewed row counts and experts with no rows
        {"name": "dgrad_fine_grained", "op": "dgrad", "rows": 16384, "E": 64, "N": 4096, "K": 7168, "act": "none", "empty": 13},
        # the tiny layer's gate/up projections
        {"name": "wgrad_tiny", "op": "wgrad", "rows": 128, "E": 8, "N": 512, "K": 128, "out": "f32", "empty": 1},
        # Mixtral-shaped down projection, the second of several micro-batches added to the fp32 gradient
        {"name": "wgrad_mixtral_add", "op": "wgrad", "rows": 8192, "E": 8, "N": 4096, "K": 14336, "out": "f32_add", "empty": 0},
        # fine-grained gate/up projections, skewed row counts: most of the time goes to writing 64 experts' gradients
        {"name": "wgrad_fine_grained", "op": "wgrad", "rows": 16384, "E": 64, "N": 4096, "K": 7168, "out": "bf16", "empty": 13},
        # 16 tokens of a Mixtral-shaped layer
        {"name": "combine_16_tokens", "op": "combine", "T": 16, "H": 4096, "k": 2},
        # a batch of the fine-grained layer
        {"name": "combine_fine_grained", "op": "combine", "T": 8192, "H": 7168, "k": 8},
        # the tiny layer's gate/up weights
        {"name": "orth_tiny", "op": "orth", "nb": 8, "rows": 512, "cols": 128, "in": "f32", "steps": 5},
        # one router's weight, [H, E] of the fine-grained layer: a single narrow matrix
        {"name": "orth_router", "op": "orth", "nb": 1, "rows": 7168, "cols": 256, "in": "bf16", "steps": 5},
        # 32 experts' down projections of the fine-grained layer
        {"name": "orth_fine_grained", "op": "orth", "nb": 32, "rows": 7168, "cols": 2048, "in": "f32", "steps": 5},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("dgrad", "wgrad", "combine", "orth"))
    if op == "combine":
        return {"op": op, "T": _log(rng, 1, 8192), "H": 128 * _log(rng, 1, 56), "k": rng.randint(1, 8)}
    if op == "orth":
        rows, cols = _log(rng, 1, 7168), _log(rng, 1, 4096)
        most = max(1, min(64, int(4e8 // (rows * cols)), int(6.5e11 // (rows * cols * min(rows, cols)))))
        return {"op": op, "nb": _log(rng, 1, most), "rows": rows, "cols": cols, "in": rng.choice(("f32", "bf16")), "steps": rng.randint(1, 6)}
    kind = rng.choice(("none", "swiglu", "geglu", "reglu") if op == "dgrad" else ("f32", "bf16", "f32_add"))
    # no more weights (dgrad), gradient bytes (wgrad) or products than the largest listed case has
    most = {"f32": 9e8, "f32_add": 4.5e8}.get(kind, 1.8e9 if op == "wgrad" else 1.4e9)
    E = _log(rng, 1, 64)
    N = 128 * _log(rng, 1, 56)
    K = 128 * _log(rng, 1, max(1, min(56, int(most / (128.0 * E * N)))))
    rows = _log(rng, E, max(E, min(16384, int(4.8e11 / (1.0 * N * K)))))
    case = {"op": op, "rows": rows, "E": E, "N": N, "K": K, "empty": rng.randint(0, E // 4)}
    case["act" if op == "dgrad" else "out"] = kind
    return case


def _counts(case, seed):
    """Rows of each expert: `empty` experts have none, the others at least one and a skewed share of the rest."""
    rs = np.random.RandomState(seed % (1 << 31))
    E, R, busy = case["E"], case["rows"], case["E"] - case["empty"]
    share = 1.0 / (4.0 + np.arange(busy)) ** 1.1
    c = np.ones(busy, dtype=np.int64) + rs.multinomial(R - busy, share / share.sum())
    counts = np.zeros(E, dtype=np.int64)
    counts[rs.permutation(E)[:busy]] = c
    return counts


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    """Normal values, drawn a slice at a time where there are many."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    for part in flat.split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda").mul_(std))
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        E, R, N, K = case["E"], case["rows"], case["N"], case["K"]
        counts = _counts(case, seed)
        s["cap"] = int(counts.max())
        s["counts"] = torch.from_numpy(counts).cuda()
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        # a gradient that arrives at the product's output
        s["dC"] = _normal(gen, R, N, std=0.01)
        s["ws"] = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
        if op == "dgrad":
            s["B"] = _normal(gen, E, N, K, std=0.02)
            s["gu"] = _normal(gen, R, 2 * K) if case["act"] != "none" else None
        else:
            s["A"] = _normal(gen, R, K)
            if case["out"] == "f32_add":
                s["dB"] = _normal(gen, E, N, K, std=0.02, dtype=torch.float32)
    elif op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        s["dout"] = _normal(gen, T, H, std=0.01)
        s["y"] = _normal(gen, T * k, H)
        s["w"] = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), 1)
        s["inv"] = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    else:
        nb, m, n = case["nb"], case["rows"], case["cols"]
        dt = torch.float32 if case["in"] == "f32" else torch.bfloat16
        # a momentum of gradients: few strong directions over many weak ones
        r = max(1, min(m, n) // 16)
        strong = torch.bmm(_normal(gen, nb, m, r, dtype=torch.float32), _normal(gen, nb, r, n, dtype=torch.float32))
        s["G"] = strong.mul_(1e-3 / math.sqrt(r)).add_(_normal(gen, nb, m, n, std=3e-4, dtype=torch.float32)).to(dt)
        # a workspace for the whole stack, by the bound that the framework documents
        p = min(m, n)
        s["ws"] = torch.zeros(65536 + nb * (12 * (m + 127) * (n + 127) + 8 * (p + 127) ** 2), dtype=torch.uint8, device="cuda")
    return s


def _scale(m, n):
    return math.sqrt(max(1.0, m / n))


def _run_own(s):
    import mixture_experts_layer_tcgen05_b200 as moe
    c = s["case"]
    op = c["op"]
    if op == "dgrad":
        E, R, N, K, act = c["E"], c["rows"], c["N"], c["K"], ACT[c["act"]]
        dA = torch.empty(R, 2 * K if act else K, dtype=torch.bfloat16, device="cuda")
        h = torch.empty(R, K, dtype=torch.bfloat16, device="cuda") if act else None
        moe.moe_grouped_gemm_dgrad(s["dC"], s["B"], s["offsets"], R, E, N, K, act, dA, gu=s["gu"], h=h, ws=s["ws"])
        return {"dA": dA, "h": h} if act else {"dA": dA}
    if op == "wgrad":
        E, R, N, K = c["E"], c["rows"], c["N"], c["K"]
        add = c["out"] == "f32_add"
        dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        dB = s["dB"] if add else torch.empty(E, N, K, dtype=dt, device="cuda")
        kind = moe.MOE_GRAD_BF16 if c["out"] == "bf16" else moe.MOE_GRAD_F32
        moe.moe_grouped_gemm_wgrad(s["dC"], s["A"], s["offsets"], R, E, N, K, kind, add, dB, ws=s["ws"])
        return {"dB": dB}
    if op == "combine":
        T, H, k = c["T"], c["H"], c["k"]
        dy = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float32, device="cuda")
        moe.moe_combine_backward(s["dout"], s["y"], s["w"], s["inv"], (T, H, 128, k, k), dy, dw, ws=s["ws"])
        return {"dy": dy, "dw": dw}
    nb, m, n = c["nb"], c["rows"], c["cols"]
    out = torch.empty(nb, m, n, dtype=torch.bfloat16, device="cuda")
    kind = moe.MOE_GRAD_F32 if c["in"] == "f32" else moe.MOE_GRAD_BF16
    moe.moe_orthogonalize(s["G"], nb, m, n, kind, c["steps"], COEFFS, EPS, _scale(m, n), out, ws=s["ws"])
    return {"O": out}


def _by_expert(s, x):
    """The rows of each expert, padded with zero rows to the longest: [E, cap, columns] in fp32."""
    at = torch.arange(s["cap"], device="cuda")
    start = s["offsets"][:-1].long()
    row = (start[:, None] + at).clamp(max=x.shape[0] - 1)
    return torch.where((at < s["counts"][:, None])[..., None], x[row].float(), 0.0)


def _rows_of(s, y):
    """The rows of [E, cap, columns] in the routed order."""
    E = y.shape[0]
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), s["counts"], output_size=s["case"]["rows"])
    r = torch.arange(s["case"]["rows"], device="cuda") - s["offsets"][:-1].long()[e]
    return y[e, r]


def _act(kind, g):
    """The activation of the gate and its derivative."""
    if kind == "swiglu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    if kind == "geglu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    return torch.clamp(g, min=0), (g > 0).to(g.dtype)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op = c["op"]
    if op == "dgrad":
        d = _rows_of(s, torch.bmm(_by_expert(s, s["dC"]), s["B"].float()))
        if c["act"] == "none":
            return {"dA": d.bfloat16()}
        g, u = s["gu"].float().chunk(2, 1)
        a, da = _act(c["act"], g)
        return {"dA": torch.cat([d * u * da, d * a], 1).bfloat16(), "h": (a * u).bfloat16()}
    if op == "wgrad":
        d = torch.bmm(_by_expert(s, s["dC"]).transpose(1, 2), _by_expert(s, s["A"]))
        if c["out"] == "f32_add":
            return {"dB": s["dB"].add_(d)}
        return {"dB": d if c["out"] == "f32" else d.bfloat16()}
    if op == "combine":
        i = s["inv"].long()
        d = s["dout"].float()[:, None, :]
        dy = torch.empty(s["y"].shape, device="cuda")
        dy[i.view(-1)] = (s["w"][..., None] * d).view(dy.shape)
        return {"dy": dy.bfloat16(), "dw": (d * s["y"].float()[i]).sum(-1)}
    return {"O": _newton_schulz(s["G"].float(), c["steps"], _scale(c["rows"], c["cols"])).bfloat16()}


def _newton_schulz(x, steps, scale):
    a, b, c = COEFFS
    wide = x.shape[1] <= x.shape[2]
    x = x if wide else x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(steps):
        g = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
    x = x * scale
    return x if wide else x.transpose(1, 2)


def work(case):
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        R, N, K, E = case["rows"], case["N"], case["K"], case["E"]
        flops = 2.0 * R * N * K
        if op == "dgrad":
            out = K if case["act"] == "none" else 5 * K  # dA; or gate and up in, their gradients and the activation out
            return {"bytes": 2.0 * (R * (N + out) + (E - case["empty"]) * N * K), "flops": flops}
        each = {"bf16": 2, "f32": 4, "f32_add": 8}[case["out"]]
        return {"bytes": 2.0 * R * (N + K) + float(each) * E * N * K, "flops": flops}
    if op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        return {"bytes": 2.0 * T * H * (1 + 2 * k) + 12.0 * T * k, "flops": 3.0 * T * k * H}
    nb, p, q = case["nb"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # the two products of p x p results are symmetric: half of each is enough
    step = 1.0 * p * p * q + 1.0 * p * p * p + 2.0 * p * p * q
    return {"bytes": float(nb) * p * q * ((4 if case["in"] == "f32" else 2) + 2), "flops": nb * case["steps"] * step}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        edges = s["offsets"].tolist()
        E, R, N, K = case["E"], case["rows"], case["N"], case["K"]
        if op == "wgrad":
            out = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
            for e in range(E):
                lo, hi = edges[e], edges[e + 1]
                if hi > lo:
                    out[e] = torch.einsum("rn,rk->nk", s["dC"][lo:hi].double(), s["A"][lo:hi].double())
            if case["out"] == "f32_add":
                out += s["dB"]
            return {"dB": out}
        out = torch.zeros(R, K, dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = edges[e], edges[e + 1]
            if hi > lo:
                out[lo:hi] = s["dC"][lo:hi].double() @ s["B"][e].double()
        if case["act"] == "none":
            return {"dA": out}
        g, u = s["gu"][:, :K].double(), s["gu"][:, K:].double()
        if case["act"] == "swiglu":
            sig = 1 / (1 + torch.exp(-g))
            value, slope = g * sig, sig + g * sig * (1 - sig)
        elif case["act"] == "geglu":
            phi = torch.special.ndtr(g)
            value, slope = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        else:
            value, slope = torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, 0.0).double()
        dA = torch.empty(R, 2 * K, dtype=torch.float64, device="cuda")
        dA[:, :K] = out * u * slope
        dA[:, K:] = out * value
        return {"dA": dA, "h": value * u}
    if op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        dy = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        d = s["dout"].double()
        for j in range(k):
            at = s["inv"][:, j].long()
            dy[at] = d * s["w"][:, j, None].double()
            dw[:, j] = torch.einsum("th,th->t", d, s["y"][at].double())
        return {"dy": dy, "dw": dw}
    a, b, c = COEFFS
    m, n = case["rows"], case["cols"]
    out = torch.empty(case["nb"], m, n, dtype=torch.float64, device="cuda")
    for i in range(case["nb"]):
        x = s["G"][i].double()
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(case["steps"]):
            if m <= n:
                g = x @ x.mT
                x = a * x + (b * g + c * (g @ g)) @ x
            else:
                g = x.mT @ x
                x = a * x + x @ (b * g + c * (g @ g))
        out[i] = x * _scale(m, n)
    return {"O": out}
