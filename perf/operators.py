"""The cases by which the 8-bit integer and gated feed-forward operators are measured.

quantize_i8    rows of bf16 or fp32 to signed 8-bit codes with one scale per row
i8_matmul      the product of such codes, with scales per token and per output channel
glu            SiLU(x Wg^T) * (x Wu^T) on bf16 weights, gate and up rows fused in one matrix
glu_backward   the gradients of glu with respect to x and the fused weights
i8_ffn         the gated feed-forward layer in 8 bits: codes, gate/up, SwiGLU, codes, down projection

Sizes are those of one expert of the routed layer that they stand beside (gate/up [4096, 7168], down [7168, 2048],
prefill of 4096 tokens, decode of 1 to 16), and ragged ones.
"""

import math

import torch

own = False


def listed():
    return [
        # the activations of a decode batch on their way into an 8-bit product
        {"name": "codes_16", "op": "quantize_i8", "rows": 16, "k": 7168, "src": "bf16"},
        # one layer's weights, coded when a model is converted
        {"name": "codes_weights", "op": "quantize_i8", "rows": 4096, "k": 7168, "src": "fp32"},
        # one token through one projection: reads every weight once
        {"name": "matmul_1", "op": "i8_matmul", "t": 1, "n": 4096, "k": 7168, "out": "fp32"},
        # a batch of decode requests that is no multiple of anything, and an odd number of outputs
        {"name": "matmul_ragged", "op": "i8_matmul", "t": 77, "n": 2053, "k": 2048, "out": "bf16"},
        # a prefill chunk
        {"name": "matmul_4096", "op": "i8_matmul", "t": 4096, "n": 4096, "k": 7168, "out": "fp32"},
        # one token through the unquantised block, as when its quantised form is checked against it
        {"name": "glu_1", "op": "glu", "t": 1, "n": 4096, "k": 7168, "save": False},
        # a calibration batch, with the gate and up rows kept for the backward pass
        {"name": "glu_4096", "op": "glu", "t": 4096, "n": 4096, "k": 7168, "save": True},
        # a short, ragged training batch on a small layer
        {"name": "grad_200", "op": "glu_backward", "t": 200, "n": 1040, "k": 1032},
        # a training batch
        {"name": "grad_4096", "op": "glu_backward", "t": 4096, "n": 4096, "k": 7168},
        # the 8-bit expert that every token passes: one token, a decode batch, a prefill chunk
        {"name": "ffn_1", "op": "i8_ffn", "t": 1, "n": 4096, "h": 7168},
        {"name": "ffn_16", "op": "i8_ffn", "t": 16, "n": 4096, "h": 7168},
        {"name": "ffn_4096", "op": "i8_ffn", "t": 4096, "n": 4096, "h": 7168},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(max(round(v / step), -(-low // step)), high // step)) * step


def draw(rng):
    op = rng.choice(["quantize_i8", "i8_matmul", "glu", "glu_backward", "i8_ffn"])
    t = _spread(rng, 1, 4096)
    if op == "quantize_i8":
        return {"op": op, "rows": t, "k": _spread(rng, 16, 7168, 16), "src": rng.choice(["bf16", "fp32"])}
    if op == "i8_matmul":
        return {"op": op, "t": t, "n": _spread(rng, 33, 4096), "k": _spread(rng, 128, 7168, 16),
                "out": rng.choice(["bf16", "fp32"])}
    if op == "i8_ffn":
        return {"op": op, "t": t, "n": _spread(rng, 128, 4096, 32), "h": _spread(rng, 128, 7168, 16)}
    n, k = _spread(rng, 128, 4096, 16), _spread(rng, 128, 7168, 8)
    if op == "glu":
        return {"op": op, "t": t, "n": n, "k": k, "save": rng.random() < 0.5}
    return {"op": op, "t": t, "n": n, "k": k}


def work(case):
    op = case["op"]
    if op == "quantize_i8":
        r, k = case["rows"], case["k"]
        return {"bytes": r * k * (2 if case["src"] == "bf16" else 4) + r * k + 4 * r, "flops": 2 * r * k}
    t, n = case["t"], case["n"]
    if op == "i8_ffn":
        h = case["h"]
        return {"bytes": 2 * t * h + n * h + 4 * n + h * (n // 2) + 4 * h + 4 * t * h,
                "flops": 2 * t * n * h + 2 * t * h * (n // 2)}
    k = case["k"]
    if op == "i8_matmul":
        return {"bytes": t * k + 4 * t + n * k + 4 * n + t * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * t * n * k}
    if op == "glu":
        return {"bytes": 2 * (t * k + n * k + t * (n // 2) + (t * n if case["save"] else 0)), "flops": 2 * t * n * k}
    return {"bytes": 2 * (t * (n // 2) + t * n + 2 * t * k + 2 * n * k), "flops": 4 * t * n * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _activations(gen, t, k):
    """bf16 hidden states: one channel in a hundred is eight times as large as the others."""
    x = torch.randn((t, k), generator=gen, device="cuda")
    big = torch.rand((k,), generator=gen, device="cuda") < 0.01
    return (x * torch.where(big, 8.0, 1.0)).to(torch.bfloat16)


def _weights(gen, n, k):
    """fp32 weights whose outputs have about unit size, rows of different sizes."""
    w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
    return w * (0.5 + torch.rand((n, 1), generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "quantize_i8":
        if case["src"] == "bf16":
            s["src"] = _activations(gen, case["rows"], case["k"])
        else:
            s["src"] = _weights(gen, case["rows"], case["k"])
    elif op == "i8_matmul":
        s["xq"], s["sx"] = _codes(_activations(gen, case["t"], case["k"]))
        s["wq"], s["sw"] = _codes(_weights(gen, case["n"], case["k"]))
    elif op == "i8_ffn":
        n, h = case["n"], case["h"]
        s["x"] = _activations(gen, case["t"], h)
        s["gu"], s["sgu"] = _codes(_weights(gen, n, h))
        s["dn"], s["sdn"] = _codes(_weights(gen, h, n // 2))
    else:
        t, n, k = case["t"], case["n"], case["k"]
        s["x"] = _activations(gen, t, k)
        s["w"] = _weights(gen, n, k).to(torch.bfloat16)
        if op == "glu_backward":
            # what the forward pass kept, and the gradient that comes back through the down projection
            s["y"] = (s["x"].float() @ s["w"].float().T).to(torch.bfloat16)
            s["dact"] = (0.1 * torch.randn((t, n // 2), generator=gen, device="cuda")).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------


def _codes(src):
    """Codes and scales of the rows: scale = amax / 127, code = src * (127 / amax) to the nearest, ties to even."""
    v = src.float()
    amax = v.abs().amax(dim=1, keepdim=True)
    some = amax >= 2.0 ** -119
    # both quotients between tensors: a division by a number may be done as a product with its reciprocal
    full = torch.full_like(amax, 127.0)
    inv = torch.where(some, full / amax, torch.zeros_like(amax))
    q = torch.round(v * inv).to(torch.int8)
    return q, torch.where(some, amax / full, torch.zeros_like(amax))[:, 0].contiguous()


def _product(xq, sx, wq, sw):
    """fp32 products of codes; the integer sums pass 2^24, so they are formed in 64 bits, where they are exact."""
    acc = (xq.double() @ wq.double().T).float()
    return (acc * sx[:, None]) * sw[None, :]


def _bf16_once(v):
    """fp64 to bf16 in one rounding (a conversion by way of fp32 rounds twice): eight significant bits, ties to even."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 256.0) / 256.0, e).to(torch.bfloat16)


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import sub_bit_sparse_b200 as stq1
        if op == "quantize_i8":
            return stq1.quantize_i8(state["src"])
        if op == "i8_matmul":
            return stq1.i8_matmul(state["xq"], state["sx"], state["wq"], state["sw"],
                                  dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        if op == "glu":
            return stq1.glu(state["x"], state["w"], save=case["save"])
        if op == "glu_backward":
            return stq1.glu_backward(state["dact"], state["y"], state["x"], state["w"])
        return stq1.i8_ffn(state["x"], state["gu"], state["sgu"], state["dn"], state["sdn"])

    if op == "quantize_i8":
        return _codes(state["src"])
    if op == "i8_matmul":
        y = _product(state["xq"], state["sx"], state["wq"], state["sw"])
        return y.to(torch.bfloat16) if case["out"] == "bf16" else y
    if op == "i8_ffn":
        half = case["n"] // 2
        xq, sx = _codes(state["x"])
        y = _product(xq, sx, state["gu"], state["sgu"]).double()
        g, u = y[:, :half], y[:, half:]
        # the next codes round this once more: in 64 bits, so that no value falls on the other side of a border
        act = _bf16_once(g / (1.0 + torch.exp(-g)) * u)
        aq, sa = _codes(act)
        return _product(aq, sa, state["dn"], state["sdn"])
    half = case["n"] // 2
    if op == "glu":
        y = state["x"].float() @ state["w"].float().T
        g, u = y[:, :half], y[:, half:]
        act = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
        return (act, y.to(torch.bfloat16)) if case["save"] else act
    g, u, d = state["y"][:, :half].float(), state["y"][:, half:].float(), state["dact"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    dy = torch.cat([d * u * sg * (1.0 + g * (1.0 - sg)), d * g * sg], dim=1)
    dx = dy @ state["w"].float()
    dw = dy.T @ state["x"].float()
    return dx.to(torch.bfloat16), dw.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_codes(src):
    """The codes' own roundings are part of their definition: the quotients and the scaled values are fp32."""
    v = src.to(torch.float64)
    top = torch.maximum(v.max(dim=1).values, -v.min(dim=1).values)
    up = torch.zeros_like(top)
    live = top >= 2.0 ** -119
    up[live] = torch.div(torch.full_like(top[live], 127.0), top[live]).to(torch.float32).to(torch.float64)
    scaled = torch.mul(v, up.unsqueeze(1)).to(torch.float32).to(torch.float64)
    low = torch.floor(scaled)
    rest = scaled - low
    odd = torch.remainder(low, 2.0) == 1.0
    q = low + ((rest > 0.5) | ((rest == 0.5) & odd)).to(torch.float64)
    s = torch.zeros_like(top)
    s[live] = torch.div(top[live], torch.full_like(top[live], 127.0))
    return q, s


def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    if op == "quantize_i8":
        q, sc = _exact_codes(s["src"])
        return q.to(torch.int8), sc
    if op == "i8_matmul":
        acc = torch.einsum("tk,nk->tn", s["xq"].to(torch.float64), s["wq"].to(torch.float64))
        return acc * torch.outer(s["sx"].to(torch.float64), s["sw"].to(torch.float64))
    if op == "i8_ffn":
        # the rows between the two products are fp32, then bf16, then codes: those roundings belong to the definition
        half = case["n"] // 2
        q, sc = _exact_codes(s["x"])
        acc = torch.einsum("tk,nk->tn", q, s["gu"].to(torch.float64)).to(torch.float32)
        y = acc.mul(sc.to(torch.float32).unsqueeze(1)).mul(s["sgu"].unsqueeze(0)).to(torch.float64)
        g, u = torch.split(y, half, dim=1)
        bits = (torch.sigmoid(g) * g * u).view(torch.int64)
        even = (bits >> 45) & 1
        act = ((bits + (1 << 44) - 1 + even) >> 45 << 45).view(torch.float64)
        q, sc = _exact_codes(act)
        acc = torch.einsum("tk,nk->tn", q, s["dn"].to(torch.float64))
        return acc * torch.outer(sc, s["sdn"].to(torch.float64))
    half = case["n"] // 2
    x, w = s["x"].to(torch.float64), s["w"].to(torch.float64)
    if op == "glu":
        g, u = torch.einsum("tk,nk->tn", x, w[:half]), torch.einsum("tk,nk->tn", x, w[half:])
        act = torch.sigmoid(g) * g * u
        return (act, torch.cat((g, u), 1)) if case["save"] else act
    g, u = torch.split(s["y"].to(torch.float64), half, dim=1)
    d, sg = s["dact"].to(torch.float64), torch.sigmoid(g)
    dg = d * u * (sg + g * sg * (1.0 - sg))
    du = d * sg * g
    dx = torch.einsum("tn,nk->tk", dg, w[:half]) + torch.einsum("tn,nk->tk", du, w[half:])
    dw = torch.cat((torch.einsum("tn,tk->nk", dg, x), torch.einsum("tn,tk->nk", du, x)), 0)
    return dx, dw
