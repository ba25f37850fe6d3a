"""The operators of a feed-forward block trained in 16 bits and served in 8-bit integers, as measured cases.

  quantize_rows   int8 codes with one fp32 scale per row (a token's activations, an output channel's weights)
  product         D = (A sa) (B sb)^T + C with those codes and scales
  gated           h = act(x Wg^T) (x Wu^T), on 16-bit values or on int8 codes; for training with both projections kept
  gated_backward  the gradients of x, Wg and Wu from h's

Where `own` is false, run() computes them in elementary torch operations in 32 bits (64 where a code lies next to a
border); where it is true, through the package's entry points.
"""

import math

import torch

own = False

TOP = 127.0
TINY = 2.0 ** -100     # the least magnitude that a row's scale is made from
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's activations, ahead of a product while serving
        {"name": "quantize_rows_token", "op": "quantize_rows", "type": "bf16", "rows": 1, "cols": 4096},
        # a prompt's activations
        {"name": "quantize_rows_prompt", "op": "quantize_rows", "type": "bf16", "rows": 8192, "cols": 4096},
        # one token through the layer that leads out of the block: the weight is read once
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 8192, "out": "bf16", "c": False},
        # sizes that end inside a tile, with a residual added
        {"name": "product_ragged", "op": "product", "m": 4000, "n": 3000, "k": 2064, "out": "f16", "c": True},
        # a long prompt through a large layer
        {"name": "product_prompt", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16", "c": False},
        # one token through a block kept in 16 bits
        {"name": "gated_token", "op": "gated", "type": "bf16", "act": "silu", "batch": 0, "m": 1, "f": 8192, "k": 4096, "keep": False},
        # a batch of requests, one token each, through the block in 8-bit integers
        {"name": "gated_requests_int8", "op": "gated", "type": "i8", "act": "silu", "batch": 0, "m": 48, "f": 8192, "k": 4096, "keep": False},
        # an odd block whose rows do not start on 16-byte boundaries
        {"name": "gated_ragged", "op": "gated", "type": "f16", "act": "gelu_tanh", "batch": 0, "m": 1000, "f": 2500, "k": 1001, "keep": False},
        # a training step's forward pass: both projections are kept for the backward pass
        {"name": "gated_training", "op": "gated", "type": "bf16", "act": "silu", "batch": 0, "m": 4096, "f": 8192, "k": 4096, "keep": True},
        # a small block's backward pass
        {"name": "gated_backward_small", "op": "gated_backward", "type": "bf16", "act": "silu", "batch": 0, "m": 512, "f": 1024, "k": 512},
        # eight experts of odd sizes
        {"name": "gated_backward_experts", "op": "gated_backward", "type": "f16", "act": "gelu", "batch": 8, "m": 300, "f": 1000, "k": 520},
        # a training step's backward pass
        {"name": "gated_backward_training", "op": "gated_backward", "type": "bf16", "act": "silu", "batch": 0, "m": 4096, "f": 8192, "k": 4096},
    ]


def spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize_rows", "product", "product", "gated", "gated", "gated", "gated_backward", "gated_backward"])
    if op == "quantize_rows":
        return {"op": op, "type": rng.choice(["f16", "bf16", "f32"]), "rows": spread(rng, 1, 8192), "cols": spread(rng, 16, 16384)}
    if op == "product":
        return {"op": op, "m": spread(rng, 1, 8192), "n": spread(rng, 16, 8192), "k": 16 * spread(rng, 1, 512),
                "out": rng.choice(["f16", "bf16", "f32"]), "c": rng.random() < 0.4}
    m, f, k = spread(rng, 1, 4096), spread(rng, 16, 8192), spread(rng, 16, 4096)
    batch = rng.choice([0, 0, 0, spread(rng, 1, max(1, min(16, 4096 * 8192 * 4096 // (m * f * k))))])
    case = {"op": op, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), "batch": batch, "m": m, "f": f, "k": k}
    if op == "gated":
        case["type"] = rng.choice(["f16", "bf16", "bf16", "i8"])
        case["keep"] = case["type"] != "i8" and rng.random() < 0.5
        if case["type"] == "i8":
            case["k"] = -(-k // 16) * 16
        return case
    case["type"] = rng.choice(["f16", "bf16"])
    return case


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def to_codes(x):
    """int8 codes, padded with zeros to whole 16-byte rows, and one scale per row (a column of them)."""
    cols = x.shape[-1]
    top = x.abs().amax(dim=-1, keepdim=True).float().clamp_min(TINY)
    codes = torch.round(x.double() * TOP / top.double())
    return torch.nn.functional.pad(codes, (0, -cols % 16)).to(torch.int8), top / TOP


def stacked(case, *shape):
    return (case["batch"],) + shape if case["batch"] else shape


def activations(gen, shape):
    """Values whose features differ in size, a few of them large."""
    x = normal(gen, *shape) * torch.exp(0.5 * normal(gen, shape[-1]))
    x[..., :: 97] *= 4.0
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "quantize_rows":
        return {"case": case, "x": activations(gen, (case["rows"], case["cols"])).to(TYPES[case["type"]])}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = to_codes(activations(gen, (m, k)))
        b, sb = to_codes(normal(gen, n, k) * k ** -0.5)
        c = normal(gen, m, n).to(TYPES[case["out"]]) if case["c"] else None
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb, "c": c}
    m, f, k = case["m"], case["f"], case["k"]
    x = activations(gen, stacked(case, m, k))
    wg, wu = normal(gen, *stacked(case, f, k)) * k ** -0.5, normal(gen, *stacked(case, f, k)) * k ** -0.5
    if case["type"] == "i8":
        (x, sx), (wg, sg), (wu, su) = to_codes(x), to_codes(wg), to_codes(wu)
        return {"case": case, "x": x, "sx": sx, "wg": wg, "sg": sg, "wu": wu, "su": su}
    t = TYPES[case["type"]]
    state = {"case": case, "x": x.to(t), "wg": wg.to(t), "wu": wu.to(t)}
    if op == "gated_backward":
        state["g"], state["u"] = (torch.matmul(state["x"].float(), state[w].float().mT.contiguous()).to(t) for w in ("wg", "wu"))
        state["dh"] = (normal(gen, *stacked(case, m, f)) * 0.1).to(t)
    return state


def activation(kind, v):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if kind == "gelu_tanh":  # 0.5 (1 + tanh(t)) = 1 / (1 + exp(-2 t))
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return torch.where(v > 0, v, torch.zeros_like(v))


def slope(kind, v):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if kind == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-a * (v + 0.044715 * v * v * v)))
        return s + v * s * (1 - s) * a * (1 + 3 * 0.044715 * v * v)
    return (v > 0).to(v.dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from stride_layouts_lds_amd import api
        if op == "quantize_rows":
            return api.quantize_rows(state["x"])
        if op == "product":
            return api.gemm(state["a"], state["b"], state["c"], sfa=state["sa"], sfb=state["sb"], dtype=TYPES[case["out"]])
        if op == "gated":
            if case["type"] == "i8":
                return api.gated(state["x"], state["wg"], state["wu"], case["act"], sx=state["sx"], s_gate=state["sg"],
                                 s_up=state["su"], dtype=torch.bfloat16)
            return api.gated(state["x"], state["wg"], state["wu"], case["act"], keep=case["keep"])
        return api.gated_backward(state["dh"], state["x"], state["wg"], state["wu"], state["g"], state["u"], case["act"])
    if op == "quantize_rows":
        return to_codes(state["x"])
    if op == "product":
        d = torch.mm(state["a"].float(), state["b"].float().t()) * state["sa"] * state["sb"].t()
        return (d if state["c"] is None else d + state["c"].float()).to(TYPES[case["out"]])
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    if op == "gated":
        if case["type"] == "i8":
            x, wg, wu = x * state["sx"], wg * state["sg"], wu * state["su"]
        g, u = torch.matmul(x, wg.mT.contiguous()), torch.matmul(x, wu.mT.contiguous())
        h = activation(case["act"], g) * u
        t = torch.bfloat16 if case["type"] == "i8" else TYPES[case["type"]]
        return (h.to(t), g.to(t), u.to(t)) if case["keep"] else h.to(t)
    t = TYPES[case["type"]]
    g, u, dh = state["g"].float(), state["u"].float(), state["dh"].float()
    dg, du = dh * u * slope(case["act"], g), dh * activation(case["act"], g)
    dx = torch.matmul(dg, wg) + torch.matmul(du, wu)
    return dx.to(t), torch.matmul(dg.mT.contiguous(), x).to(t), torch.matmul(du.mT.contiguous(), x).to(t)


def work(case):
    op = case["op"]
    size = {"i8": 1, "f16": 2, "bf16": 2, "f32": 4}
    if op == "quantize_rows":
        n = case["rows"] * case["cols"]
        return {"bytes": size[case["type"]] * n + n + 4 * case["rows"], "flops": 2 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        moved = m * k + n * k + 4 * (m + n) + (2 if case["c"] else 1) * size[case["out"]] * m * n
        return {"bytes": moved, "flops": 2 * m * n * k}
    batch, m, f, k, e = max(1, case["batch"]), case["m"], case["f"], case["k"], size[case["type"]]
    if op == "gated":
        moved = e * (m * k + 2 * f * k) + 2 * m * f * (3 if case["keep"] else 1) + (4 * (m + 2 * f) if e == 1 else 0)
        return {"bytes": batch * moved, "flops": batch * 4 * m * f * k}
    return {"bytes": batch * e * (2 * m * k + 4 * f * k + 3 * m * f), "flops": batch * 8 * m * f * k}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize_rows":
        x = state["x"].double()
        top = torch.maximum(x.abs().max(dim=1, keepdim=True).values, torch.full_like(x[:, :1], TINY))
        v = x.abs() * TOP / top
        whole = torch.floor(v)
        up = (v - whole > 0.5) | ((v - whole == 0.5) & (whole % 2 == 1))
        q = torch.zeros(x.shape[0], -(-x.shape[1] // 16) * 16, dtype=torch.int8, device=x.device)
        q[:, : x.shape[1]] = (torch.sign(x) * (whole + up)).to(torch.int8)
        return q, top / TOP
    if op == "product":
        d = (state["a"].double() * state["sa"].double()) @ (state["b"].double() * state["sb"].double()).t()
        return d if state["c"] is None else d + state["c"].double()
    x, wg, wu = state["x"].double(), state["wg"].double(), state["wu"].double()
    if case["type"] == "i8":
        x, wg, wu = x * state["sx"].double(), wg * state["sg"].double(), wu * state["su"].double()
    kind = case["act"]

    def smooth(v):
        """The activation over v (a value between 0 and 1) and its derivative."""
        if kind == "silu":
            s = torch.sigmoid(v)
            return s, s * (1 - s)
        if kind == "gelu":
            return torch.special.ndtr(v), torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
        if kind == "gelu_tanh":
            c = math.sqrt(2 / math.pi)
            s = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
            return s, 2 * s * (1 - s) * c * (1 + 3 * 0.044715 * v.square())
        return (v > 0).double(), torch.zeros_like(v)

    if op == "gated":
        g = torch.stack([a @ b.t() for a, b in zip(x, wg)]) if case["batch"] else x @ wg.t()
        u = torch.stack([a @ b.t() for a, b in zip(x, wu)]) if case["batch"] else x @ wu.t()
        h = g * smooth(g)[0] * u
        return (h, g, u) if case["keep"] else h
    g, u, dh = state["g"].double(), state["u"].double(), state["dh"].double()
    part, rate = smooth(g)
    dg, du = dh * u * (part + g * rate), dh * g * part
    if not case["batch"]:
        return dg @ wg + du @ wu, dg.t() @ x, du.t() @ x
    each = [(a @ c + b @ d, a.t() @ y, b.t() @ y) for a, b, c, d, y in zip(dg, du, wg, wu, x)]
    return tuple(torch.stack(part) for part in zip(*each))
