"""The operators of a linear layer trained and served in 8-bit floating point, as measured cases.

  quantize       E4M3 codes with one fp32 scale per 1 x 128 (or 128 x 128) block, and, asked for, the codes of the
                 transpose, blocked along the other axis
  product        D = (A SA) (B SB)^T + C with those codes and scales
  orthogonalize  an update's Newton-Schulz orthogonalisation (five steps of x <- a x + (b G + c G^2) x, G = x x^T)

Where `own` is false, run() computes them in elementary torch operations in 32 bits; where it is true, through the
package's entry points.
"""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0            # the largest E4M3 value
TINY = 2.0 ** -100     # the least magnitude that a block's scale is made from
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def blocks(n):
    return -(-n // BLOCK)


def listed():
    return [
        # one token's activations, ahead of a product while serving
        {"name": "quantize_token", "op": "quantize", "type": "bf16", "rows": 1, "cols": 4096, "block_rows": 1, "both": False},
        # a training step's activations: along the features for the forward product, along the tokens for the weight's gradient
        {"name": "quantize_tokens_both", "op": "quantize", "type": "bf16", "rows": 8192, "cols": 4096, "block_rows": 1, "both": True},
        # an odd weight kept in 32 bits, in square blocks, with its transpose for the gradient of the activations
        {"name": "quantize_weight_ragged", "op": "quantize", "type": "f32", "rows": 4000, "cols": 3000, "block_rows": 128, "both": True},
        # one token through a layer: the weight is read once
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "out": "bf16", "b_rows": 128, "c": False},
        # a batch of requests, one token each
        {"name": "product_requests", "op": "product", "m": 48, "n": 8192, "k": 8192, "out": "bf16", "b_rows": 128, "c": False},
        # sizes that end inside a tile, with a residual added
        {"name": "product_ragged", "op": "product", "m": 4000, "n": 3000, "k": 2064, "out": "f16", "b_rows": 128, "c": True},
        # a weight's gradient, summed over the tokens into 32 bits
        {"name": "product_gradient", "op": "product", "m": 4096, "n": 4096, "k": 8192, "out": "f32", "b_rows": 1, "c": True},
        # the forward product of a large layer
        {"name": "product_forward", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16", "b_rows": 128, "c": False},
        # the update of a small weight
        {"name": "orthogonalize_small", "op": "orthogonalize", "type": "bf16", "batch": 1, "m": 96, "n": 128},
        # the updates of one weight of each of 16 layers, taller than wide and odd
        {"name": "orthogonalize_batch", "op": "orthogonalize", "type": "f16", "batch": 16, "m": 1000, "n": 520},
        # a wide projection's update
        {"name": "orthogonalize_wide", "op": "orthogonalize", "type": "bf16", "batch": 1, "m": 1024, "n": 4096},
        # a large layer's update
        {"name": "orthogonalize_large", "op": "orthogonalize", "type": "bf16", "batch": 1, "m": 8192, "n": 8192},
    ]


def spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "orthogonalize"])
    if op == "quantize":
        return {"op": op, "type": rng.choice(["f16", "bf16", "f32"]), "rows": spread(rng, 1, 8192),
                "cols": spread(rng, 16, 8192), "block_rows": rng.choice([1, 128]), "both": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "m": spread(rng, 1, 8192), "n": spread(rng, 16, 8192), "k": 16 * spread(rng, 1, 512),
                "out": rng.choice(["f16", "bf16", "f32"]), "b_rows": rng.choice([1, 128]), "c": rng.random() < 0.4}
    m, n = spread(rng, 16, 4096), spread(rng, 16, 4096)
    most = max(1, min(32, 4096 * 4096 // (m * n)))
    return {"op": op, "type": rng.choice(["f16", "bf16"]), "batch": spread(rng, 1, most), "m": m, "n": n}


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def to_codes(x, block_rows):
    """Codes, and scales of one value per (block_rows x 128) block stored with the rows contiguous."""
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), blocks(cols)
    full = torch.zeros(br * block_rows, bc * BLOCK, device=x.device)
    full[:rows, :cols] = x
    tiles = full.view(br, block_rows, bc, BLOCK)
    top = tiles.abs().amax(dim=(1, 3)).clamp_min(TINY)
    bad = ~torch.isfinite(top)
    scale = torch.where(bad, torch.nan, top / TOP)
    codes = (tiles * TOP / top[:, None, :, None]).clamp(-TOP, TOP)
    codes = torch.where(bad[:, None, :, None], torch.nan, codes).view(br * block_rows, bc * BLOCK)
    kept = -(-cols // 16) * 16
    codes = torch.nn.functional.pad(codes[:rows, :cols], (0, kept - cols))
    return codes.to(torch.float8_e4m3fn), scale.t().contiguous().t()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        # activations whose features differ in size, a few of them large
        x = normal(gen, rows, cols) * torch.exp(0.5 * normal(gen, cols))
        x[:, :: 97] *= 8.0
        return {"case": case, "x": x.to(TYPES[case["type"]])}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = to_codes(normal(gen, m, k) * torch.exp(0.5 * normal(gen, k)), 1)
        b, sb = to_codes(normal(gen, n, k) * (k ** -0.5), case["b_rows"])
        c = normal(gen, m, n).to(TYPES[case["out"]]) if case["c"] else None
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb, "c": c}
    batch, m, n = case["batch"], case["m"], case["n"]
    # a gradient's momentum: a few strong directions in noise
    r = min(8, m, n)
    x = normal(gen, batch, m, r) @ normal(gen, batch, r, n) * 0.5 + normal(gen, batch, m, n)
    x = (x * 1e-3).to(TYPES[case["type"]])
    return {"case": case, "x": x if batch > 1 else x[0]}


def decoded(codes, scales, block_rows):
    """The real values of codes and scales, in 32 bits."""
    rows, cols = codes.shape
    s = scales.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scales
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :cols]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from stride_layouts_lds_amd import api
        if op == "quantize":
            return api.quantize(state["x"], block_rows=case["block_rows"], transposed=case["both"])
        if op == "product":
            return api.gemm(state["a"], state["b"], state["c"], sfa=state["sa"], sfb=state["sb"], block_k=BLOCK,
                            dtype=TYPES[case["out"]])
        return api.orthogonalize(state["x"])
    if op == "quantize":
        x = state["x"].float()
        out = to_codes(x, case["block_rows"])
        return out + to_codes(x.t(), case["block_rows"]) if case["both"] else out
    if op == "product":
        a = decoded(state["a"], state["sa"], 1)
        b = decoded(state["b"], state["sb"], case["b_rows"])
        d = a @ b.t()
        return (d if state["c"] is None else d + state["c"].float()).to(TYPES[case["out"]])
    x = state["x"].float()
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if tall else x
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + 1e-7)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        g = x @ x.transpose(-2, -1).contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    x = x.transpose(-2, -1) if tall else x
    return x.to(TYPES[case["type"]])


def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols, br = case["rows"], case["cols"], case["block_rows"]
        size = {"f16": 2, "bf16": 2, "f32": 4}[case["type"]]
        n = rows * cols
        moved = size * n + n + 4 * -(-rows // br) * blocks(cols)
        if case["both"]:
            moved += n + 4 * -(-cols // br) * blocks(rows)
        return {"bytes": moved, "flops": (4 if case["both"] else 2) * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = {"f16": 2, "bf16": 2, "f32": 4}[case["out"]]
        moved = m * k + n * k + 4 * blocks(k) * (m + -(-n // case["b_rows"])) + (2 if case["c"] else 1) * out * m * n
        return {"bytes": moved, "flops": 2 * m * n * k}
    batch, m, n = case["batch"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # G and G^2 are symmetric: half of their products
    step = m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n
    return {"bytes": 2 * 2 * batch * m * n, "flops": batch * STEPS * step}


def nearest_e4m3(v):
    """64-bit values rounded to the nearest E4M3 value, ties to even."""
    _, e = torch.frexp(v.abs())
    step = torch.exp2((e.double() - 1).clamp_min(-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def exact_codes(x, block_rows):
    rows, cols = x.shape
    r = torch.arange(rows, device=x.device) // block_rows
    c = torch.arange(cols, device=x.device) // BLOCK
    along = torch.zeros(rows, blocks(cols), device=x.device, dtype=torch.float64)
    along = along.scatter_reduce(1, c.expand(rows, cols), x.abs(), "amax")
    top = torch.zeros(-(-rows // block_rows), blocks(cols), device=x.device, dtype=torch.float64)
    top = top.scatter_reduce(0, r[:, None].expand(rows, blocks(cols)), along, "amax")
    top = torch.maximum(top, torch.full_like(top, TINY))
    q = nearest_e4m3(x * TOP / top[r][:, c])
    kept = -(-cols // 16) * 16
    return torch.cat([q, q.new_zeros(rows, kept - cols)], 1), top / TOP


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = state["x"].double()
        out = exact_codes(x, case["block_rows"])
        if case["both"]:
            out += exact_codes(x.t().contiguous(), case["block_rows"])
        return out
    if op == "product":
        a, b = state["a"].double(), state["b"].double()
        d = torch.zeros(case["m"], case["n"], device=a.device, dtype=torch.float64)
        sa, sb = state["sa"].double(), state["sb"].double()
        rows = torch.arange(case["n"], device=a.device) // case["b_rows"]
        for j in range(blocks(case["k"])):
            at = slice(j * BLOCK, (j + 1) * BLOCK)
            d.addmm_(a[:, at] * sa[:, j : j + 1], (b[:, at] * sb[rows, j : j + 1]).t())
        return d if state["c"] is None else d + state["c"].double()
    x = state["x"].double()
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT if flip else x
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + 1e-7)
    a, b, c = COEFFICIENTS
    eye = torch.eye(x.shape[-2], device=x.device, dtype=torch.float64)
    for _ in range(STEPS):
        g = torch.matmul(x, x.mT.contiguous())
        x = torch.matmul(a * eye + torch.matmul(g, b * eye + c * g), x)
    return x.mT.contiguous() if flip else x
