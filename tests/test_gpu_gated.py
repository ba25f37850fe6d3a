"""Row quantisation to int8, the int8 product, the gated feed-forward block and
its backward pass on the GPU, against plain implementations in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and e = finfo(type).eps / 2 (half
a step of the result's type):
  int8 product   the int32 sum rounded once, two products: 3 u of sa sb S; C's
                 addition u, the result's rounding e
  16-bit sums    K products added in fp32 in any order: K 2 u of sum |x w| (an
                 addition in the matrix core may drop rather than round)
  activation     1.2 is above every slope; the functions' own error is stated in fn()
"""

import math

import pytest

pytestmark = pytest.mark.gpu

TOP, TINY = 127.0, 2.0 ** -100
U = 2.0 ** -24
# The hardware's exponential and reciprocal give zero for results below 2^-126: the
# s of act(v) = v s is then 0, off by less than 2^-126, and act(v) by that times |v|.
FLUSH = 2.0 ** -126
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from stride_layouts_lds_amd import api as A
    A.lib()
    return A


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape):
    import torch
    return torch.randn(shape, generator=gen(seed), device="cuda")


def integers(seed, low, high, *shape):
    import torch
    return torch.randint(low, high + 1, shape, generator=gen(seed), device="cuda")


def dtype_of(name):
    import torch
    return getattr(torch, name)


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half a step of the type's subnormals."""
    import torch
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def strided(x, how):
    """x's values in another storage: "cols" column-major, "padded" row-major with
    rows off 16 bytes, "sparse" no unit stride, "wide" 16-byte rows far apart."""
    import torch
    if how == "rows":
        return x.contiguous()
    if how == "cols":
        return x.mT.contiguous().mT
    if how == "wide":
        store = torch.full(x.shape[:-1] + (x.shape[-1] + 64,), 7, dtype=x.dtype, device=x.device)
        v = store[..., 16:16 + x.shape[-1]]
    else:
        pad, step = (3, 1) if how == "padded" else (5, 2)
        store = torch.full(x.shape[:-1] + (step * x.shape[-1] + pad,), 7, dtype=x.dtype, device=x.device)
        v = store[..., 1:1 + step * x.shape[-1]:step]
    v.copy_(x)
    return v


def within(got, want, tol, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst by {float((off / tol).nan_to_num(9e9).max()):.3g} of "
                                 f"its tolerance, first at {bad.nonzero()[0].tolist()}")


# ---------------------------------------------------------------------------
# row quantisation
# ---------------------------------------------------------------------------

def check_rows(q, s, x):
    """Scales bit for bit, codes the nearest integers to 127 x / top, ties to even:
    the quotient in 64 bits decides them (a 24-bit x lies on a tie or 2^-25 off)."""
    import torch
    x = x.double()
    top = x.abs().amax(-1, keepdim=True).clamp_min(TINY) if x.shape[-1] else torch.full(x.shape[:-1] + (1,), TINY, device=x.device,
                                                                                         dtype=torch.float64)
    assert torch.equal(s, (top / TOP).float())
    C = x.shape[-1]
    assert q.shape == x.shape[:-1] + (-(-C // 16) * 16,)
    assert not q[..., C:].any()
    assert torch.equal(q[..., :C], torch.round(x * TOP / top).to(torch.int8))


SIZES = [(1, 1), (1, 16), (1, 4096), (1, 5000), (3, 7), (5, 1000), (64, 1024), (65, 1025), (127, 4096), (1100, 4096), (1100, 4097),
         (1030, 520), (7, 16384), (3, 16400), (2, 40000)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_quantize_rows(api, size, dtype):
    import torch
    x = (normal(1, *size) * torch.exp(normal(2, size[1]))).to(dtype_of(dtype))
    check_rows(*api.quantize_rows(x), x)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_quantize_rows_ties(api, dtype):
    """Rows whose quotients are exact ties, and fp32 values one step off them."""
    import torch
    k = torch.arange(-127, 127, device="cuda", dtype=torch.float64) + 0.5
    rows = []
    for scale in (1.0, 2.0 ** -20, 2.0 ** 10, 3.0 * 2.0 ** -9):
        top = 127.0 * scale
        rows.append(torch.cat([torch.tensor([top], device="cuda", dtype=torch.float64), k * scale]))
    x = torch.stack(rows)
    t = dtype_of(dtype)
    x = x[:, (x.to(t).double() == x).all(0)]  # those that the type holds
    assert x.shape[1] > 80  # bf16: 3 |2 k + 1| has eight bits up to |2 k + 1| = 85
    check_rows(*api.quantize_rows(x.to(t)), x)
    if t == torch.float32:
        y = x.float()
        for toward in (float("inf"), -float("inf")):
            z = torch.nextafter(y, torch.full_like(y, toward))
            z[:, 0] = y[:, 0]
            check_rows(*api.quantize_rows(z), z)
        # a top that 127 does not divide: ties of x = (k + 1/2) top / 127 rounded
        top = torch.tensor(1.2345678, dtype=torch.float32).item()
        z = torch.cat([torch.tensor([top], device="cuda"), ((k * top) / 127.0).float()])[None]
        check_rows(*api.quantize_rows(z), z)


@pytest.mark.parametrize("how", ["cols", "padded", "sparse"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_quantize_rows_strides_and_batches(api, how, dtype):
    import torch
    x = strided(normal(3, 3, 150, 333).to(dtype_of(dtype)), how)
    q, s = api.quantize_rows(x)
    check_rows(q, s, x)
    # one matrix read for all, codes and scales of other strides
    out = (torch.full((3, 150, 400), 9, dtype=torch.int8, device="cuda")[..., :384], torch.full((3, 150, 2), 9.0, device="cuda")[..., 1:])
    api.quantize_rows(x[:1].expand(3, -1, -1), out=out)
    for b in range(3):
        assert torch.equal(out[0][b, :, :336], q[0]) and not out[0][b, :, 336:].any() and torch.equal(out[1][b], s[0])


@pytest.mark.parametrize("how", ["rows", "cols"])
@pytest.mark.parametrize("cols", [100, 3000, 20000])
def test_quantize_rows_extremes(api, how, cols):
    """Zeros, the smallest and the largest values; a NaN or an infinity makes its
    row's scale NaN and its codes 0, and leaves the others."""
    import torch
    x = normal(4, 70, cols)
    x[0] = 0
    x[1] *= 1e-38
    x[2, 1] = 3.4e38
    x[3, 2] = 1e-45
    x = strided(x, how)
    clean = api.quantize_rows(x)
    check_rows(*clean, x)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = strided(x.clone(), how)
        y[5, cols - 1] = bad
        q, s = api.quantize_rows(y)
        assert torch.isnan(s[5]).all() and not q[5].any()
        keep = torch.arange(70, device="cuda") != 5
        assert torch.equal(q[keep], clean[0][keep]) and torch.equal(s[keep], clean[1][keep])
    b = torch.full((2, 40), 3.0e38, dtype=torch.bfloat16, device="cuda")
    check_rows(*api.quantize_rows(b), b)


def test_quantize_rows_many(api):
    """More than 2^32 elements: offsets pass 32 bits."""
    import torch
    rows = (1 << 32) // 4096 + 130
    x = torch.zeros((rows, 4096), dtype=torch.float16, device="cuda")
    x[-200:] = normal(5, 200, 4096).half()
    q, s = api.quantize_rows(x)
    check_rows(q[-256:], s[-256:], x[-256:])
    assert not q[:-200][::1009].any()


def test_quantize_rows_empty(api):
    import torch
    q, s = api.quantize_rows(torch.zeros(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1)
    x = torch.zeros(70, 0, device="cuda")
    q, s = api.quantize_rows(x)
    check_rows(q, s, x)


# ---------------------------------------------------------------------------
# the int8 product
# ---------------------------------------------------------------------------

def codes(seed, *shape):
    import torch
    return integers(seed, -128, 127, *shape).to(torch.int8)


def scales(seed, *shape):
    return (normal(seed, *shape, 1).abs() + 0.1) * 0.01


def check_int8(api, a, b, sa, sb, c=None, dtype="bfloat16", **kw):
    import torch
    t = dtype_of(dtype)
    got = api.gemm(a, b, c, sfa=sa, sfb=sb, dtype=t, **kw)
    part = torch.matmul(a.double(), b.double().mT.contiguous()) * sa.double() * sb.double().mT
    want = part if c is None else part + c.double()
    tol = 3.01 * U * part.abs() + (1.01 * U + half_step(t)) * want.abs() + smallest(t)
    within(got, want, tol, f"{tuple(a.shape)} x {tuple(b.shape)}")
    return got


SHAPES = [(1, 1, 16), (1, 4096, 1024), (3, 100, 48), (16, 257, 144), (17, 64, 128), (32, 200, 2064), (33, 130, 1040), (48, 8192, 512),
          (64, 300, 384), (65, 4100, 256), (130, 700, 512), (200, 1000, 4096), (1000, 1030, 272), (1300, 1500, 528), (2100, 2300, 128),
          (4100, 4200, 144), (5000, 130, 80)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_int8_product(api, shape, dtype):
    M, N, K = shape
    a, b = codes(1, M, K), codes(2, N, K)
    sa, sb = scales(3, M), scales(4, N)
    check_int8(api, a, b, sa, sb, dtype=dtype)
    check_int8(api, a, b, sa, sb, normal(5, M, N).to(dtype_of(dtype)), dtype)


@pytest.mark.parametrize("shape", [(1, 40, 131056), (20, 24, 131056), (300, 400, 8192)])
def test_int8_sums_are_exact(api, shape):
    """The largest sums there are, of one sign: -128 x -128 up to 131056 times."""
    import torch
    M, N, K = shape
    a, b = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    one = lambda n: torch.ones(n, 1, device="cuda")
    got = api.gemm(a, b, sfa=one(M), sfb=one(N), dtype=torch.float32)
    assert torch.equal(got, torch.full((M, N), float(K) * 16384.0, device="cuda"))


@pytest.mark.parametrize("M", [1, 40, 300, 2100])
def test_int8_strides_batches_and_broadcasts(api, M):
    import torch
    N, K = 260, 272
    a, b = codes(1, 3, M, K), codes(2, 3, N, K)
    sa, sb = scales(3, 3, M), scales(4, 3, N)
    plain = check_int8(api, a, b, sa, sb)
    wide = lambda x: strided(x, "wide")
    out = strided(torch.zeros(3, M, N, dtype=torch.bfloat16, device="cuda"), "sparse")
    got = check_int8(api, wide(a), wide(b), strided(sa, "sparse"), strided(sb, "sparse"), out=out)
    assert got is out and torch.equal(out, plain)
    out = strided(torch.zeros(3, M, N, dtype=torch.float32, device="cuda"), "cols")
    c = strided(normal(6, 3, M, N), "padded")
    check_int8(api, a, b, sa, sb, c, "float32", out=out)
    # one weight for every matrix, one scale for every row, one row of C for all
    # (a bias), and C in D's place
    bias = normal(7, 1, 1, N).bfloat16().expand(3, M, N)
    got = check_int8(api, a, b[0].expand(3, N, K), sa[:, :1].expand(3, M, 1), sb[0].expand(3, N, 1), bias)
    again = api.gemm(a, b[0], bias, sfa=sa[:, :1].expand(3, M, 1), sfb=sb[0], dtype=torch.bfloat16)
    assert torch.equal(got, again)
    d = c.clone().bfloat16()
    want = check_int8(api, a, b, sa, sb, d.clone())
    api.gemm(a, b, d, out=d, sfa=sa, sfb=sb)
    assert torch.equal(d, want)


def test_int8_row_of_one_with_any_stride(api):
    """A single row's stride is never stepped along: it may be anything."""
    import torch
    store = codes(1, 64 * 1024)
    a = store[:1024].as_strided((1, 1024), (16, 1))
    b = store[1024:].view(63, 1024)
    check_int8(api, a, b, scales(2, 1), scales(3, 63))
    check_int8(api, b, a, scales(3, 63), scales(2, 1))
    # rows that overlap
    a = store.as_strided((300, 1024), (16, 1))
    check_int8(api, a, b, scales(4, 300), scales(3, 63))
    check_int8(api, b[:1].expand(300, -1), b, scales(4, 300), scales(3, 63))


def test_int8_nan_scale(api):
    """A row with a NaN scale (quantize_rows of a row with a NaN) gives NaN there alone."""
    import torch
    for M in (5, 50, 700):
        a, b, sa, sb = codes(1, M, 256), codes(2, 300, 256), scales(3, M), scales(4, 300)
        want = api.gemm(a, b, sfa=sa, sfb=sb)
        sa[3] = float("nan")
        a[3] = 0
        got = api.gemm(a, b, sfa=sa, sfb=sb)
        keep = torch.arange(M, device="cuda") != 3
        assert torch.isnan(got[3]).all() and torch.equal(got[keep], want[keep])


def test_int8_empty(api):
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")
    o = lambda *s: torch.ones(*s, device="cuda")
    assert api.gemm(z(0, 64), z(5, 64), sfa=o(0, 1), sfb=o(5, 1)).shape == (0, 5)
    c = normal(1, 20, 5).half()
    assert torch.equal(api.gemm(z(20, 0), z(5, 0), c, sfa=o(20, 1), sfb=o(5, 1)), c)
    assert not api.gemm(z(300, 0), z(500, 0), sfa=o(300, 1), sfb=o(500, 1)).any()


# ---------------------------------------------------------------------------
# the gated block
# ---------------------------------------------------------------------------

def activation(kind, v):
    """act(v) and act'(v) in 64 bits."""
    import torch
    if kind == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if kind == "gelu":
        p = torch.special.ndtr(v)
        return v * p, p + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))
        return v * s, s + v * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * v * v)
    return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).double()


def fn(kind, v):
    """What the fp32 functions may be off by, of act(v): the exponential's
    argument t is rounded a few times (each U |t|, t = v or 1.6 v (1 + 0.045 v^2)),
    exponential, reciprocal and products 2 U each, erfc 8 U."""
    t = v.abs() if kind == "silu" else 1.6 * v.abs() * (1 + 0.045 * v * v) if kind == "gelu_tanh" else v * v
    return 0 * v if kind == "relu" else (16 + 4 * t) * 2 * U


def matmul(a, b):
    """a b^T of (batches of) 64-bit matrices."""
    import torch
    return torch.matmul(a, b.mT.contiguous())


def check_gated(kind, got, x, wg, wu, sx=None, sg=None, su=None):
    """h, or (h, gate, up)."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = matmul(x, wg), matmul(x, wu)
    if sx is not None:  # (scales after the sums: sums of integers that are zero stay so)
        g, u = g * sx.double() * sg.double().mT, u * sx.double() * su.double().mT
        eg, eu = 3.01 * U * g.abs(), 3.01 * U * u.abs()
    else:
        ax, K = x.abs(), x.shape[-1]
        eg, eu = K * 2 * U * matmul(ax, wg.abs()), K * 2 * U * matmul(ax, wu.abs())
    a, _ = activation(kind, g)
    ea = 1.2 * eg + a.abs() * fn(kind, g.abs() + eg) + FLUSH * g.abs()
    outs = got if isinstance(got, tuple) else (got,)
    e = half_step(outs[0].dtype)
    tiny = smallest(outs[0].dtype)
    h = a * u
    eh = a.abs() * eu + u.abs() * ea + ea * eu + U * h.abs()
    within(outs[0], h, eh * 1.01 + e * (h.abs() + eh) + tiny, "h")
    for o, v, ev, name in zip(outs[1:], (g, u), (eg, eu), ("gate", "up")):
        within(o, v, ev * 1.01 + e * (v.abs() + ev) + tiny, name)


def block(seed, shape, dtype, batch=(), shared=False):
    import torch
    M, F, K = shape
    t = dtype_of(dtype)
    x = normal(seed, *batch, M, K).to(t)
    w = normal(seed + 1, 2, *(() if shared else batch), F, K) * K ** -0.5
    return x, w[0].to(t), w[1].to(t)


# (M, F, K): every tile, whole and ragged, K whole, ending inside a K-tile and off 8
GATED = [(1, 1, 8), (1, 8192, 512), (1, 300, 4096), (5, 40, 1000), (16, 130, 72), (17, 40, 128), (32, 1000, 512), (33, 100, 1032),
         (48, 8192, 256), (64, 333, 640), (65, 2100, 256), (130, 500, 520), (200, 64, 2000), (257, 1500, 200), (600, 1000, 64),
         (1300, 1100, 320), (2100, 2200, 136), (4100, 1030, 192)]


@pytest.mark.parametrize("shape", GATED)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated(api, shape, dtype, kind):
    x, wg, wu = block(1, shape, dtype)
    check_gated(kind, api.gated(x, wg, wu, kind), x, wg, wu)


@pytest.mark.parametrize("shape", [(1, 300, 4096), (40, 100, 264), (200, 500, 136), (1300, 1100, 320)])
@pytest.mark.parametrize("kind", ACTS)
def test_gated_keeps_both_projections(api, shape, kind):
    import torch
    x, wg, wu = block(1, shape, "bfloat16")
    got = api.gated(x * 3, wg, wu, kind, keep=True)
    check_gated(kind, got, x * 3, wg, wu)
    assert torch.equal(api.gated(x * 3, wg, wu, kind), got[0])


@pytest.mark.parametrize("shape", GATED)
def test_gated_integers_bit_for_bit(api, shape):
    """relu of small integers: every sum is exact, so only the last rounding is left."""
    import torch
    M, F, K = shape
    x = integers(1, -2, 2, M, K).half()
    w = integers(2, -2, 2, 2, F, K).half()
    h, g, u = api.gated(x, w[0], w[1], "relu", keep=True)
    ge, ue = matmul(x.double(), w[0].double()), matmul(x.double(), w[1].double())
    assert torch.equal(g, ge.half()) and torch.equal(u, ue.half())
    assert torch.equal(h, (ge.clamp_min(0) * ue).float().half())
    assert torch.equal(api.gated(x, w[0], w[1], "relu"), h)


@pytest.mark.parametrize("shape", [(1, 300, 1001), (7, 40, 7), (40, 65, 333), (1000, 250, 1001), (600, 1030, 65)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated_odd_rows(api, shape, dtype):
    """K off 8: the operands are copied to whole 16-byte rows first."""
    x, wg, wu = block(1, shape, dtype)
    check_gated("silu", api.gated(x, wg, wu), x, wg, wu)


@pytest.mark.parametrize("how", ["cols", "padded", "sparse", "wide"])
@pytest.mark.parametrize("M", [3, 50, 200])
def test_gated_strides(api, how, M):
    import torch
    x, wg, wu = block(1, (M, 72, 136), "float16")
    want = api.gated(x, wg, wu, "gelu", keep=True)
    check_gated("gelu", want, x, wg, wu)
    for views in ((strided(x, how), wg, wu), (x, strided(wg, how), strided(wu, how)), (x, wg, strided(wu, how)),
                  (strided(x, how), strided(wg, how), strided(wu, how))):
        for a, b in zip(api.gated(*views, "gelu", keep=True), want):
            assert torch.equal(a, b)
    out = tuple(strided(torch.zeros_like(t), how) for t in want)
    for a, b in zip(api.gated(x, wg, wu, "gelu", keep=True, out=out), want):
        assert torch.equal(a, b)
    # both projections in one matrix, side by side and in turns of rows
    both = torch.zeros((M, 144), dtype=torch.float16, device="cuda")
    turns = torch.zeros((2 * M, 72), dtype=torch.float16, device="cuda")
    for pair in ((both[:, :72], both[:, 72:]), (both[:, 72:], both[:, :72]), (turns[0::2], turns[1::2]), (both[:, 0::2], both[:, 1::2])):
        got = api.gated(x, wg, wu, "gelu", keep=True, out=(out[0],) + pair)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    h = strided(torch.zeros_like(want[0]), how)
    assert api.gated(x, wg, wu, "gelu", out=h) is h and torch.equal(h, want[0])


@pytest.mark.parametrize("shape", [(1, 200, 264), (9, 100, 136), (70, 150, 100), (300, 400, 72)])
def test_gated_batches(api, shape):
    """Experts of their own weights; one weight for all, as a batch that is one
    matrix of all its rows and as one that is not."""
    import torch
    x, wg, wu = block(1, shape, "bfloat16", (3,))
    got = api.gated(x, wg, wu, keep=True)
    check_gated("silu", got, x, wg, wu)
    for b in range(3):
        for g, w in zip(got, api.gated(x[b], wg[b], wu[b], keep=True)):
            check_gated("silu", got[0][b], x[b], wg[b], wu[b])
    want = api.gated(x, wg[0].contiguous(), wu[0].contiguous(), keep=True)
    check_gated("silu", want, x, wg[0], wu[0])
    spread = torch.zeros((3, shape[0] + 5, shape[2]), dtype=x.dtype, device="cuda")[:, 2:-3]
    spread.copy_(x)
    check_gated("silu", api.gated(spread, wg[0], wu[0], keep=True), x, wg[0], wu[0])
    check_gated("silu", api.gated(x, wg[:1].expand(3, -1, -1), wu[:1].expand(3, -1, -1), keep=True), x, wg[0], wu[0])
    # one x for every expert
    check_gated("silu", api.gated(x[0], wg, wu, keep=True), x[0], wg, wu)
    # gate shared, up not
    check_gated("silu", api.gated(x, wg[0], wu, keep=True), x, wg[0], wu)


def test_gated_many_sequences_of_one_token(api):
    import torch
    x, wg, wu = block(1, (1, 320, 264), "bfloat16", (75,), shared=True)
    h = api.gated(x, wg, wu)
    check_gated("silu", h, x, wg, wu)
    assert torch.equal(h[:, 0], api.gated(x[:, 0], wg, wu))
    # of a longer one, the last token of each
    long = normal(7, 75, 9, 264).bfloat16()
    check_gated("silu", api.gated(long[:, -1:], wg, wu), long[:, -1:], wg, wu)


@pytest.mark.parametrize("shape", [(1, 1, 16), (1, 8192, 512), (16, 130, 80), (17, 40, 128), (48, 8192, 256), (64, 333, 656), (65, 2100, 256),
                                   (200, 64, 2000), (600, 1000, 64), (1300, 1100, 320), (2100, 2200, 144)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_gated_int8(api, shape, dtype):
    M, F, K = shape
    x, w = codes(1, M, K), codes(2, 2, F, K)
    sx, sw = scales(3, M) * 0.3, scales(4, 2, F) * K ** -0.5
    got = api.gated(x, w[0], w[1], sx=sx, s_gate=sw[0], s_up=sw[1], keep=True, dtype=dtype_of(dtype))
    check_gated("silu", got, x, w[0], w[1], sx, sw[0], sw[1])


def test_gated_int8_batches_and_strides(api):
    import torch
    for M in (1, 30, 200):
        x, w = codes(1, 3, M, 144), codes(2, 2, 3, 100, 144)
        sx, sw = scales(3, 3, M), scales(4, 2, 3, 100)
        args = dict(sx=sx, s_gate=sw[0], s_up=sw[1], dtype=torch.bfloat16, keep=True)
        got = api.gated(x, w[0], w[1], "gelu", **args)
        check_gated("gelu", got, x, w[0], w[1], sx, sw[0], sw[1])
        other = dict(args, sx=strided(sx, "sparse"), s_gate=strided(sw[0], "sparse"), s_up=strided(sw[1], "cols"))
        for a, b in zip(api.gated(strided(x, "wide"), strided(w[0], "wide"), w[1], "gelu", **other), got):
            assert torch.equal(a, b)
        shared = api.gated(x, w[0][0], w[1][0], "gelu", **dict(args, s_gate=sw[0][0], s_up=sw[1][0]))
        check_gated("gelu", shared, x, w[0][0], w[1][0], sx, sw[0][0], sw[1][0])
        one = api.gated(x, w[0][0], w[1][0], "gelu", **dict(args, sx=sx[0], s_gate=sw[0][0], s_up=sw[1][0]))
        check_gated("gelu", one, x, w[0][0], w[1][0], sx[0], sw[0][0], sw[1][0])


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_activation_far_out(api, kind, M):
    """Gates from far below zero to far above, zero among them: x is the gate
    itself (an identity for its weight)."""
    import torch
    v = torch.cat([torch.linspace(-60, 60, 200, device="cuda"), torch.tensor([0.0, -0.0, 1e-7, -1e-7, 300.0, -300.0, -3e4, 3e4], device="cuda")])
    x = v.expand(M, -1).contiguous().half()
    eye = torch.eye(208, device="cuda", dtype=torch.float16)
    ones = torch.zeros(208, 208, device="cuda", dtype=torch.float16)
    ones[:, 100:101] = 1.0 / float(x[0, 100])  # up is 1 or close to it
    h, g, u = api.gated(x, eye, ones, kind, keep=True)
    assert torch.equal(g, x)
    want = activation(kind, x.double())[0] * float(x[0, 100]) * float(ones[0, 100])
    tol = want.abs() * (fn(kind, x.double().abs()) + half_step(torch.float16) + 4 * U) + FLUSH * x.double().abs() + smallest(torch.float16)
    within(h, want, tol, kind)


def test_gated_nan_and_infinity(api):
    """A NaN in one token stays in its row; in one weight row in its column; relu
    passes it on."""
    import torch
    for M in (3, 40, 300):
        x, wg, wu = block(1, (M, 200, 136), "bfloat16")
        want = api.gated(x, wg, wu, "relu")
        x2 = x.clone()
        x2[2, 5] = float("nan")
        h = api.gated(x2, wg, wu, "relu")
        keep = torch.arange(M, device="cuda") != 2
        assert torch.isnan(h[2]).all() and torch.equal(h[keep], want[keep])
        w2 = wg.clone()
        w2[7, 0] = float("nan")
        h = api.gated(x, w2, wu, "relu")
        keep = torch.arange(200, device="cuda") != 7
        assert torch.isnan(h[:, 7]).all() and torch.equal(h[:, keep], want[:, keep])


def test_gated_empty(api):
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.float16)
    assert api.gated(z(0, 64), z(8, 64), z(8, 64)).shape == (0, 8)
    assert api.gated(z(5, 64), z(0, 64), z(0, 64)).shape == (5, 0)
    for M in (3, 40, 600):
        for t in api.gated(z(M, 0), z(300, 0), z(300, 0), keep=True, out=tuple(normal(1, M, 300).half() for _ in range(3))):
            assert not t.any()


# ---------------------------------------------------------------------------
# its backward pass
# ---------------------------------------------------------------------------

def check_backward(kind, got, dh, x, wg, wu, g, u):
    """dg and du are off by their own rounding and the functions'; the products'
    sums by that times the other operand, and by their additions."""
    import torch
    t = x.dtype
    e, tiny = half_step(t), smallest(t)
    dh, x, wg, wu, g, u = (v.double() for v in (dh, x, wg, wu, g, u))
    a, slope = activation(kind, g)
    dg, du = dh * u * slope, dh * a
    # the slope is a sum of terms up to 1 + |t|: its error is absolute
    ef = fn(kind, g)
    edg = (dh * u).abs() * (ef * (2 + g.abs()) + 4 * U + FLUSH * (2 + g.abs())) + e * dg.abs() + tiny
    edu = dh.abs() * (a.abs() * ef + 4 * U * a.abs() + FLUSH * g.abs()) + e * du.abs() + tiny
    edg, edu = edg * (1 + e), edu * (1 + e)
    shared = wg.dim() == 2 and x.dim() == 3
    F, M = wg.shape[-2], x.shape[-2] * (x.shape[0] if shared else 1)
    if got[0] is not None:
        want = torch.matmul(dg, wg) + torch.matmul(du, wu)
        size = torch.matmul(dg.abs() + edg, wg.abs()) + torch.matmul(du.abs() + edu, wu.abs())
        tol = torch.matmul(edg, wg.abs()) + torch.matmul(edu, wu.abs()) + (2 * F + 8) * 2 * U * size
        within(got[0], want, tol + e * (want.abs() + tol) + tiny, "dx")
    if got[1] is not None:
        flat = (lambda v: v.reshape(-1, v.shape[-1])) if shared else (lambda v: v)
        for d, ed, o, name in ((dg, edg, got[1], "dw_gate"), (du, edu, got[2], "dw_up")):
            left, el, right = flat(d).mT.contiguous(), flat(ed).mT.contiguous(), flat(x)
            want = torch.matmul(left, right)
            tol = torch.matmul(el, right.abs()) + (M + 8) * 2 * U * torch.matmul(left.abs() + el, right.abs())
            within(o, want, tol + e * (want.abs() + tol) + tiny, name)


def state(seed, shape, dtype, kind, batch=(), shared=False):
    """Inputs of the backward pass: what a forward call had and kept."""
    import torch
    x, wg, wu = block(seed, shape, dtype, batch, shared)
    t = dtype_of(dtype)
    g, u = matmul(x.double(), wg.double()).to(t), matmul(x.double(), wu.double()).to(t)
    dh = normal(seed + 5, *batch, shape[0], shape[1]).to(t)
    return dh, x, wg, wu, g, u


BACKWARD = [(1, 1, 1), (1, 300, 520), (5, 40, 1000), (16, 130, 72), (63, 64, 65), (64, 64, 64), (65, 66, 129), (130, 500, 520), (200, 64, 2000),
            (257, 1500, 200), (600, 1000, 63), (1300, 1100, 320), (700, 2500, 1001)]


@pytest.mark.parametrize("shape", BACKWARD)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated_backward(api, shape, dtype):
    import torch
    s = state(1, shape, dtype, "silu")
    got = api.gated_backward(*s, "silu")
    check_backward("silu", got, *s)
    one = api.gated_backward(*s, "silu", need_dw=False)
    two = api.gated_backward(*s, "silu", need_dx=False)
    assert one[1] is None and one[2] is None and two[0] is None
    # (a call for one of them may take another tile, which adds in another order)
    check_backward("silu", one, *s)
    check_backward("silu", two, *s)


@pytest.mark.parametrize("kind", ACTS)
def test_gated_backward_activations(api, kind):
    s = state(1, (150, 200, 136), "float16", kind)
    s[4].mul_(3)
    s[4][0, :50] = 0
    s[4][1, :20] = 30
    s[4][2, :20] = -30
    check_backward(kind, api.gated_backward(*s, kind), *s)


@pytest.mark.parametrize("shape", [(1, 40, 72), (70, 100, 136), (300, 260, 65), (200, 520, 264), (430, 1000, 520)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated_backward_batches(api, shape, dtype):
    """Experts; weights shared by a batch, whose gradients are summed over it, as
    one matrix of all rows and as rows apart."""
    import torch
    s = state(1, shape, dtype, "gelu", (3,))
    check_backward("gelu", api.gated_backward(*s, "gelu"), *s)
    s = state(1, shape, dtype, "gelu", (3,), shared=True)
    got = api.gated_backward(*s, "gelu")
    check_backward("gelu", got, *s)
    apart = torch.zeros((3, shape[0] + 3, shape[2]), dtype=s[1].dtype, device="cuda")[:, 1:-2]
    apart.copy_(s[1])
    got = api.gated_backward(s[0], apart, *s[2:], "gelu")
    check_backward("gelu", got, *s)
    # a batch of one
    s = state(2, shape, dtype, "gelu", (1,))
    check_backward("gelu", api.gated_backward(*s, "gelu"), *s)


@pytest.mark.parametrize("how", ["cols", "padded", "sparse", "wide"])
def test_gated_backward_strides(api, how):
    import torch
    s = state(1, (130, 100, 72), "bfloat16", "silu")
    want = api.gated_backward(*s)
    check_backward("silu", want, *s)
    for a, b in zip(api.gated_backward(*(strided(v, how) for v in s)), want):
        assert torch.equal(a, b)
    out = tuple(strided(torch.zeros_like(t), how) for t in want)
    api.gated_backward(*s, out=out)
    for a, b in zip(out, want):
        within(a, b.double(), 2.1 * half_step(a.dtype) * b.double().abs() + 1e-30)  # another tile may sum in another order
    # the weights' gradients the other way round in one buffer, and interleaved by rows
    both = torch.zeros((2,) + want[1].shape, dtype=want[1].dtype, device="cuda")
    api.gated_backward(*s, out=(out[0], both[1], both[0]))
    check_backward("silu", (out[0], both[1], both[0]), *s)
    rows = torch.zeros((200, 72), dtype=want[1].dtype, device="cuda")
    api.gated_backward(*s, out=(out[0], rows[0::2], rows[1::2]))
    check_backward("silu", (out[0], rows[0::2], rows[1::2]), *s)


def test_gated_backward_integers_bit_for_bit(api):
    """relu with small integers: dg, du and every sum are exact."""
    import torch
    for M, F, K in ((70, 130, 72), (300, 520, 264), (513, 300, 600)):
        x, w = integers(1, -2, 2, M, K).half(), integers(2, -2, 2, 2, F, K).half()
        g, u, dh = integers(3, -3, 3, M, F).half(), integers(4, -3, 3, M, F).half(), integers(5, -2, 2, M, F).half()
        dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp_min(0)).double()
        dx, dwg, dwu = api.gated_backward(dh, x, w[0], w[1], g, u, "relu")
        assert torch.equal(dx, (dg @ w[0].double() + du @ w[1].double()).float().half())
        assert torch.equal(dwg, (dg.t() @ x.double()).float().half()) and torch.equal(dwu, (du.t() @ x.double()).float().half())


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_gated_backward_against_differences(api, kind):
    """Along random directions, (h(p + t d) - h(p - t d)) / 2t in 64 bits: the formula
    itself.  With t = 1e-4 the differences are off by t^2 times the third derivative (order
    1 times the values), next to which e-sized roundings of the gradients are large:
    the tolerance is theirs, e = 2^-11 on sums of M F values added in quadrature, six
    of them."""
    import torch
    M, F, K = 40, 50, 60
    dh, x, wg, wu, g, u = state(3, (M, F, K), "float16", kind)
    # gates as the forward pass has them before rounding
    grads = api.gated_backward(dh, x, wg, wu, g, u, kind)
    value = lambda x, a, b: float((activation(kind, matmul(x, a))[0] * matmul(x, b) * dh.double()).sum())
    p = [t.double() for t in (x, wg, wu)]
    for i, grad in enumerate(grads):
        d = normal(10 + i, *p[i].shape).double()
        at = lambda t: value(*[v + t * d if j == i else v for j, v in enumerate(p)])
        want = (at(1e-4) - at(-1e-4)) / 2e-4
        got = float((grad.double() * d).sum())
        # roundings of g, u, dg, du and of the gradient, relative e each: independent over the entries
        noise = 6 * 2.0 ** -11 * float((grad.double() * d).square().sum().sqrt()) * math.sqrt(5) * 4
        assert abs(got - want) <= noise, (i, got, want, noise)


def test_gated_backward_empty(api):
    """No tokens: the weights' gradients are zeros; no columns of h: x's is."""
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.float16)
    f = lambda *s: torch.ones(*s, device="cuda", dtype=torch.float16)
    for lead in ((), (3,), (0,)):
        M = 0 if lead != (0,) else 5
        dw = f(2, 8, 64)
        out = (f(*lead, M, 64), dw[0], dw[1])
        api.gated_backward(z(*lead, M, 8), z(*lead, M, 64), z(8, 64), z(8, 64), z(*lead, M, 8), z(*lead, M, 8), out=out)
        assert not dw.any()
    dw = f(2, 3, 8, 64)
    api.gated_backward(z(3, 0, 8), z(3, 0, 64), z(3, 8, 64), z(3, 8, 64), z(3, 0, 8), z(3, 0, 8), out=(f(3, 0, 64), dw[0], dw[1]))
    assert not dw.any()
    dx = f(70, 64)
    api.gated_backward(z(70, 0), z(70, 64), z(0, 64), z(0, 64), z(70, 0), z(70, 0), out=(dx, z(0, 64), z(0, 64)))
    assert not dx.any()


# ---------------------------------------------------------------------------
# how they are called: streams, workspaces, graphs, together
# ---------------------------------------------------------------------------

def served(api, x, wq, ws, dq, ds):
    """A block in 8-bit integers: codes, the gated pair, codes, the product out."""
    import torch
    q, s = api.quantize_rows(x)
    h = api.gated(q, wq[0], wq[1], "silu", sx=s, s_gate=ws[0], s_up=ws[1], dtype=torch.bfloat16)
    q, s = api.quantize_rows(h)
    return api.gemm(q, dq, x, sfa=s, sfb=ds, dtype=torch.bfloat16)


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_a_served_block(api, tokens):
    """Against the block in 64 bits on the codes' values: int8 activations are off by
    half a scale each, so the result by what that makes of sums of F terms."""
    import torch
    K, F = 256, 768
    x = normal(1, tokens, K).bfloat16()
    w = (normal(2, 2, F, K) * K ** -0.5).bfloat16()
    down = (normal(3, K, F) * F ** -0.5).bfloat16()
    (gq, gs), (uq, us), (dq, ds) = (api.quantize_rows(v) for v in (w[0], w[1], down))
    y = served(api, x, (gq, uq), (gs, us), dq, ds)
    q, s = api.quantize_rows(x)
    value = lambda q, s: q.double() * s.double()
    h = activation("silu", matmul(value(q, s), value(gq, gs)))[0] * matmul(value(q, s), value(uq, us))
    # h's codes: half a step of 1/127 of the row's largest, and bf16's rounding before
    step = h.abs().amax(-1, keepdim=True) / 127 * 0.51 + h.abs() * 2.0 ** -8 * 1.1
    want = x.double() + matmul(h, value(dq, ds))
    tol = matmul(step, value(dq, ds).abs()) + 1e-4 * matmul(h.abs(), value(dq, ds).abs())
    within(y, want, tol + 2.0 ** -8 * (want.abs() + tol))


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_a_served_block_captured(api, tokens):
    """A graph of the block, replayed with other inputs between eager calls."""
    import torch
    K, F = 256, 768
    wq, ws = zip(*(api.quantize_rows((normal(i, F, K) * K ** -0.5).bfloat16()) for i in (2, 3)))
    dq, ds = api.quantize_rows((normal(4, K, F) * F ** -0.5).bfloat16())
    x = normal(1, tokens, K).bfloat16()
    served(api, x, wq, ws, dq, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        y = served(api, x, wq, ws, dq, ds)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.copy_(normal(20 + i, tokens, K).bfloat16())
        want = served(api, x, wq, ws, dq, ds)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("shape", [(40, 100, 65), (300, 520, 264), (20, 2048, 2048), (1000, 2304, 2048)])
def test_a_training_step_captured(api, shape):
    """Forward and backward in one graph, its workspaces the graph's own."""
    import torch
    M, F, K = shape
    dh, x, wg, wu, _, _ = state(1, shape, "bfloat16", "silu")

    def step():
        h, g, u = api.gated(x, wg, wu, keep=True)
        return (h,) + tuple(api.gated_backward(dh, x, wg, wu, g, u))
    step()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = step()
    with torch.cuda.graph(other):
        second = step()
    for i in range(4):
        x.copy_(normal(30 + i, M, K).bfloat16())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, want, second):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_on_another_stream(api):
    """stream=: the call and what it allocates belong to that stream."""
    import torch
    side = torch.cuda.Stream()
    s = state(1, (200, 130, 65), "float16", "silu")
    want = api.gated(*s[1:4], keep=True) + tuple(api.gated_backward(*s)) + tuple(api.quantize_rows(s[1]))
    torch.cuda.synchronize()
    got = (api.gated(*s[1:4], keep=True, stream=side.cuda_stream) + tuple(api.gated_backward(*s, stream=side.cuda_stream)) +
           tuple(api.quantize_rows(s[1], stream=side.cuda_stream)))
    q, sc = api.quantize_rows(s[1])
    with torch.cuda.stream(side):
        also = api.gated(*s[1:4], keep=True) + tuple(api.gated_backward(*s)) + tuple(api.quantize_rows(s[1]))
    side.synchronize()
    for a, b, c in zip(got, want, also):
        assert torch.equal(a, b) and torch.equal(c, b)
    d = api.gemm(q, q, sfa=sc, sfb=sc)
    torch.cuda.synchronize()
    e = api.gemm(q, q, sfa=sc, sfb=sc, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(d, e)


def test_callers_workspace_and_neighbours(api):
    """A workspace of exactly the bytes asked for, its contents of no matter, and
    nothing written behind it or behind any output."""
    import torch
    M, F, K = 130, 100, 65
    s = state(1, (M, F, K), "bfloat16", "silu")
    want = api.gated(*s[1:4], keep=True) + tuple(api.gated_backward(*s))

    def guarded(like):
        """A view of like's shape in the middle of a buffer of 77s, and the buffer."""
        store = torch.full((like.numel() + 512,), 77, dtype=like.dtype, device="cuda")
        return store[256:256 + like.numel()].view(like.shape), store

    def untouched(store, n):
        return bool((store[:256] == 77).all()) and bool((store[256 + n:] == 77).all())

    args = api.sl_gated_args()
    outs = [guarded(t) for t in want]
    for name, t in zip(("x", "w_gate", "w_up"), s[1:4]):
        setattr(args, name, api.tensor_desc(t))
    for name, (t, _) in zip(("h", "gate", "up"), outs):
        setattr(args, name, api.tensor_desc(t))
    for name in ("sx", "s_gate", "s_up"):
        getattr(args, name).layout.rank = 2
    args.activation = 1
    n = api.sl_gated_workspace_bytes(args)
    assert n >= 2 * K * (M + 2 * F)
    ws, wstore = guarded(torch.zeros(n, dtype=torch.uint8, device="cuda"))
    ws.fill_(255)  # NaNs
    api.gated(*s[1:4], keep=True, out=tuple(o for o, _ in outs[:3]), workspace=ws)
    for (o, store), w in zip(outs[:3], want):
        assert torch.equal(o, w) and untouched(store, o.numel())
    assert untouched(wstore, n)

    back = api.sl_gated_backward_args()
    for name, t in zip(("dh", "x", "w_gate", "w_up", "gate", "up"), s):
        setattr(back, name, api.tensor_desc(t))
    for name, (t, _) in zip(("dx", "dw_gate", "dw_up"), outs[3:]):
        setattr(back, name, api.tensor_desc(t))
    back.activation = 1
    n = api.sl_gated_backward_workspace_bytes(back)
    ws, wstore = guarded(torch.zeros(n, dtype=torch.uint8, device="cuda"))
    ws.fill_(255)
    got = api.gated_backward(*s, out=tuple(o for o, _ in outs[3:]), workspace=ws)
    check_backward("silu", got, *s)
    assert all(untouched(store, o.numel()) for o, store in outs[3:]) and untouched(wstore, n)


def test_calls_do_not_vary(api):
    import torch
    s = state(1, (300, 520, 264), "float16", "silu")
    first = api.gated(*s[1:4], keep=True) + tuple(api.gated_backward(*s))
    for _ in range(3):
        for a, b in zip(api.gated(*s[1:4], keep=True) + tuple(api.gated_backward(*s)), first):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# large products: operands read as they lie, and the tiles that only they take
# ---------------------------------------------------------------------------

def backward_workspace(api, s, got):
    args = api.sl_gated_backward_args()
    for name, t in zip(("dh", "x", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up"), tuple(s) + tuple(got)):
        if t is not None:
            setattr(args, name, api.tensor_desc(t))
        else:
            getattr(args, name).layout.rank = 2
    args.activation = 1
    return api.sl_gated_backward_workspace_bytes(args)


def as_they_lie(M, F, n=1):
    """Bytes of dg and du side by side: the workspace of a call that copies nothing."""
    return -(-n * M * 2 * (-(-F // 64) * 64) * 2 // 256) * 256


# x's gradient on a large tile: F and the output's sides end inside tiles
@pytest.mark.parametrize("shape", [(3900, 200, 3504), (4001, 264, 3400), (4090, 65, 3608), (4000, 323, 4096)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_large_input_gradient(api, shape, dtype):
    M, F, K = shape
    s = state(1, shape, dtype, "silu")
    got = api.gated_backward(*s, need_dw=False)
    assert backward_workspace(api, s, got) == as_they_lie(M, F)
    check_backward("silu", got, *s)
    # the same values in rows further apart, and a result in such rows
    wide = [strided(v, "wide") for v in s]
    out = strided(got[0].clone().zero_(), "wide")
    api.gated_backward(*wide, need_dw=False, out=(out, None, None))
    assert backward_workspace(api, wide, (out, None, None)) == as_they_lie(M, F)
    assert (out == got[0]).all()
    # weights that cannot be read as they lie: the other way, whose sums run in another order
    off = [strided(v, "padded") if i in (2, 3) else v for i, v in enumerate(s)]
    assert backward_workspace(api, off, got) > as_they_lie(M, F)
    check_backward("silu", api.gated_backward(*off, need_dw=False), *s)


# the weights' gradients on a large tile: tokens that end inside a K-tile
@pytest.mark.parametrize("shape", [(384, 2040, 3600), (330, 2048, 4096), (1, 2048, 4096), (67, 2040, 3600)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_large_weight_gradients(api, shape, dtype):
    import torch
    M, F, K = shape
    s = state(1, shape, dtype, "gelu")
    got = api.gated_backward(*s, "gelu", need_dx=False)
    check_backward("gelu", got, *s)
    lies = backward_workspace(api, s, got) == as_they_lie(M, F)
    assert lies == (M > 256)  # few tokens take smaller tiles
    both = torch.zeros((F, 2, K), dtype=s[1].dtype, device="cuda")
    wide = [strided(v, "wide") for v in s]
    api.gated_backward(*wide, "gelu", need_dx=False, out=(None, both[:, 0], both[:, 1]))
    assert (both[:, 0] == got[1]).all() and (both[:, 1] == got[2]).all()


@pytest.mark.parametrize("shared", [False, True])
def test_large_backward_of_a_batch(api, shared):
    """Experts, each with tokens and weights of its own, and sequences that share them."""
    M, F, K, n = (1000, 264, 3400, 4) if shared else (1030, 1024, 2040, 4)
    s = state(1, (M, F, K), "bfloat16", "silu", (n,), shared=shared)
    check_backward("silu", api.gated_backward(*s), *s)
    one = api.gated_backward(*s, need_dw=False)
    two = api.gated_backward(*s, need_dx=False)
    check_backward("silu", one, *s)
    check_backward("silu", two, *s)


def test_large_backward_integers_bit_for_bit(api):
    """relu with small integers: dg, du and every sum are exact, on whichever way."""
    import torch
    for M, F, K in ((4096, 330, 3600), (330, 2048, 3608), (1100, 2100, 2056)):
        x, w = integers(1, -2, 2, M, K).bfloat16(), integers(2, -2, 2, 2, F, K).bfloat16()
        g, u, dh = integers(3, -3, 3, M, F).bfloat16(), integers(4, -3, 3, M, F).bfloat16(), integers(5, -2, 2, M, F).bfloat16()
        dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp_min(0)).double()
        for wg, wu, v in ((w[0], w[1], x), (strided(w[0], "padded"), strided(w[1], "padded"), strided(x, "cols"))):
            dx, dwg, dwu = api.gated_backward(dh, v, wg, wu, g, u, "relu")
            assert torch.equal(dx, (dg @ w[0].double() + du @ w[1].double()).float().bfloat16())
            assert torch.equal(dwg, (dg.t() @ x.double()).float().bfloat16()) and torch.equal(dwu, (du.t() @ x.double()).float().bfloat16())


def test_large_backward_infinities_stay_in_their_rows(api):
    """Rows and columns past an operand's end are not read as its values: what is
    next to a view in memory is NaN throughout."""
    import torch
    M, F, K = 4001, 202, 3400

    def among_nans(v):
        store = torch.full((v.shape[0] + 200, v.shape[1] + 64), float("nan"), dtype=v.dtype, device="cuda")
        view = store[100:100 + v.shape[0], 32:32 + v.shape[1]]
        view.copy_(v)
        return view
    s = state(1, (M, F, K), "bfloat16", "silu")
    got = api.gated_backward(*(among_nans(v) for v in s))
    check_backward("silu", got, *s)
    s = state(2, (330, 2048, 3608), "float16", "silu")
    got = api.gated_backward(*(among_nans(v) for v in s))
    check_backward("silu", got, *s)


# the 256 x 128 tile and tiles of two products in one launch, next to each alone
@pytest.mark.parametrize("shape", [(512, 1024, 512), (64, 360, 256), (700, 130, 2500), (1000, 1000, 1000), (2050, 1030, 1030), (33, 40, 2000), (4000, 500, 3000), (300, 3000, 3500), (1000, 2304, 2048), (260, 1500, 2056)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated_backward_tiles(api, shape, dtype):
    s = state(1, shape, dtype, "gelu_tanh")
    check_backward("gelu_tanh", api.gated_backward(*s, "gelu_tanh"), *s)
    check_backward("gelu_tanh", api.gated_backward(*s, "gelu_tanh", need_dx=False), *s)
    check_backward("gelu_tanh", api.gated_backward(*s, "gelu_tanh", need_dw=False), *s)


@pytest.mark.parametrize("shape", [(1000, 2500, 256), (1000, 2500, 4100), (256, 4096, 1000), (2048, 2048, 1032), (512, 1024, 4100), (4000, 3000, 264), (3500, 2900, 1000)])
def test_middle_tiles(api, shape):
    x, wg, wu = block(1, shape, "bfloat16")
    check_gated("silu", api.gated(x, wg, wu, keep=True), x, wg, wu)
    M, N, K = shape
    K = -(-K // 16) * 16
    check_int8(api, codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N), c=normal(5, M, N).bfloat16())


def test_two_streams_at_once(api):
    """Calls in flight on two streams, each with its own allocations, give what they give alone."""
    import torch
    s, r = state(1, (300, 520, 264), "bfloat16", "silu"), state(2, (257, 1100, 520), "bfloat16", "silu")

    def steps(v):
        q, sc = api.quantize_rows(v[1])
        return api.gated(*v[1:4], keep=True) + tuple(api.gated_backward(*v)) + (api.gemm(q, q, sfa=sc, sfb=sc),)
    want = steps(s), steps(r)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(one):
            a = steps(s)
        with torch.cuda.stream(two):
            b = steps(r)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        for x, y in zip(a + b, want[0] + want[1]):
            assert torch.equal(x, y)


def test_the_same_operand_twice(api):
    """One tensor in several places that are only read."""
    import torch
    x = normal(1, 130, 136).bfloat16()
    w = (normal(2, 200, 136) * 0.1).bfloat16()
    check_gated("silu", api.gated(x, w, w, keep=True), x, w, w)
    check_gated("gelu", api.gated(w, w, w, "gelu"), w, w, w)
    g = matmul(x.double(), w.double()).bfloat16()
    check_backward("silu", api.gated_backward(g, x, w, w, g, g), g, x, w, w, g, g)
    q, s = api.quantize_rows(w)
    check_int8(api, q, q, s, s)


# ---------------------------------------------------------------------------
# offsets past 32 bits, gradients that broadcast
# ---------------------------------------------------------------------------

def test_large_offsets(api):
    """Operands and results of more than 2^32 bytes, their last rows against the formula."""
    import torch
    K, n = 8192, 300
    rows = (1 << 32) // K + n
    a = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    a[-n:] = codes(1, n, K)
    b, sa, sb = codes(2, 64, K), scales(3, rows), scales(4, 64)
    got = api.gemm(a, b, sfa=sa, sfb=sb, dtype=torch.float32)
    part = a[-n:].double() @ b.double().t() * sa[-n:].double() * sb.double().t()
    within(got[-n:], part, 3.01 * U * part.abs())
    assert not got[:-n].any()
    # and as the weight
    got = api.gemm(b, a, sfa=sb, sfb=sa, dtype=torch.float32)
    within(got[:, -n:], part.t(), 3.01 * U * part.abs().t())
    del a, got
    rows = (1 << 31) // K + n
    x, wg, wu = block(5, (n, 64, K), "bfloat16")
    big = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    big[-n:] = x
    h, g, u = api.gated(big, wg, wu, keep=True)
    check_gated("silu", (h[-n:], g[-n:], u[-n:]), x, wg, wu)
    assert not h[:-n].any()
    # backward: the other rows' gradients are zero
    dh = torch.zeros_like(h)
    dh[-n:] = normal(6, n, 64).bfloat16()
    dx, dwg, dwu = api.gated_backward(dh, big, wg, wu, g, u)
    check_backward("silu", (dx[-n:], dwg, dwu), dh[-n:], x, wg, wu, g[-n:], u[-n:])
    assert not dx[:-n].any()
    # as the weights
    few = normal(7, 20, K).bfloat16()
    h = api.gated(few, big, big)
    check_gated("silu", h[:, -n:], few, x, x)


@pytest.mark.parametrize("shape", [(40, 100, 72), (300, 520, 264), (1100, 1000, 520)])
def test_gated_backward_of_a_sum(api, shape):
    """h's gradient as a sum gives it, one value for all (strides 0), and a row for all."""
    import torch
    M, F, K = shape
    for batch in ((), (3,)):
        for shared in (False, True):
            s = state(1, shape, "bfloat16", "silu", batch, shared and bool(batch))
            for dh in (torch.ones((), device="cuda", dtype=torch.bfloat16).expand(s[0].shape),
                       s[0][..., :1, :].expand(s[0].shape)):
                check_backward("silu", api.gated_backward(dh, *s[1:]), dh, *s[1:])


# few rows, large weights: x's gradient straight from the weights, the rows of them shared by workgroups
@pytest.mark.parametrize("shape", [(1, 2048, 2048), (16, 2100, 2056), (17, 4096, 1032), (33, 3001, 2312), (64, 2048, 2048), (65, 4100, 1032),
                                   (150, 4096, 1032), (40, 8192, 4104)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_input_gradient_of_few_rows(api, shape, dtype):
    import torch
    M, F, K = shape
    s = state(1, shape, dtype, "silu")
    got = api.gated_backward(*s, need_dw=False)
    lies = as_they_lie(M, F)
    assert lies < backward_workspace(api, s, got) <= lies + 16 * 4 * M * K  # sums of up to 16 workgroups, no copies
    check_backward("silu", got, *s)
    check_backward("silu", api.gated_backward(*s), *s)
    for a in (api.gated_backward(*s, need_dw=False), api.gated_backward(*(strided(v, "wide") for v in s), need_dw=False)):
        assert torch.equal(a[0], got[0])
    out = strided(torch.zeros_like(got[0]), "sparse")
    api.gated_backward(*s, need_dw=False, out=(out, None, None))
    assert torch.equal(out, got[0])


def test_input_gradient_of_few_rows_of_a_batch(api):
    """Experts of a few rows each; weights among NaNs; integers bit for bit."""
    import torch
    s = state(1, (20, 1500, 2056), "bfloat16", "silu", (3,))
    check_backward("silu", api.gated_backward(*s, need_dw=False), *s)
    s = state(2, (7, 2048, 2056), "float16", "silu")
    store = torch.full((2, 2300, 2200), float("nan"), dtype=torch.float16, device="cuda")
    w = store[:, 100:2148, 64:2120]
    w[0].copy_(s[2]), w[1].copy_(s[3])
    s = s[:2] + (w[0], w[1]) + s[4:]
    check_backward("silu", api.gated_backward(*s, need_dw=False), *s)
    for M in (1, 30, 60, 100):
        F, K = 2080, 2056
        x, w = integers(1, -2, 2, M, K).bfloat16(), integers(2, -2, 2, 2, F, K).bfloat16()
        g, u, dh = integers(3, -3, 3, M, F).bfloat16(), integers(4, -3, 3, M, F).bfloat16(), integers(5, -2, 2, M, F).bfloat16()
        dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp_min(0)).double()
        dx, _, _ = api.gated_backward(dh, x, w[0], w[1], g, u, "relu", need_dw=False)
        assert torch.equal(dx, (dg @ w[0].double() + du @ w[1].double()).float().bfloat16())


# how results are written: by eights, fours and single columns, and what is left of a row
@pytest.mark.parametrize("N", [129, 130, 132, 136, 267, 1036])
@pytest.mark.parametrize("how", ["rows", "wide", "padded", "sparse"])
def test_result_rows(api, N, how):
    import torch
    M, K = 300, 272
    a, b, sa, sb = codes(1, M, K), codes(2, N, K), scales(3, M), scales(4, N)
    for dtype in ("float16", "bfloat16", "float32"):
        t = dtype_of(dtype)
        c = strided(normal(5, M, N).to(t), how)
        for given in (None, c):
            out = strided(torch.full((M, N), 9, dtype=t, device="cuda"), how)
            check_int8(api, a, b, sa, sb, given, dtype, out=out)
    x, wg, wu = block(6, (M, N, K), "bfloat16")
    outs = tuple(strided(torch.full((M, N), 9, dtype=torch.bfloat16, device="cuda"), how) for _ in range(3))
    check_gated("gelu", api.gated(x, wg, wu, "gelu", keep=True, out=outs), x, wg, wu)
    check_gated("gelu", api.gated(x, wg, wu, "gelu"), x, wg, wu)
    s = state(7, (M, 200, N), "float16", "silu")
    outs = tuple(strided(torch.full_like(v, 9), how) for v in s[1:4])
    check_backward("silu", api.gated_backward(*s, out=outs), *s)


@pytest.mark.parametrize("K", [30, 64, 128, 200])
def test_many_experts_of_few_rows(api, K):
    """Few K-tiles and many matrices: larger tiles than few rows alone would take."""
    x, wg, wu = block(1, (4, 4171, K), "float16", (15,))
    check_gated("silu", api.gated(x, wg, wu, keep=True), x, wg, wu)
    n = -(-K // 16) * 16
    a, b = codes(1, 15, 16, n), codes(2, 15, 5000, n)
    check_int8(api, a, b, scales(3, 15, 16), scales(4, 15, 5000))


def test_input_gradient_of_few_rows_of_shared_weights(api):
    """Sequences that share their weights, as one matrix of all rows and as rows apart."""
    import torch
    s = state(1, (20, 2048, 2056), "bfloat16", "gelu", (3,), shared=True)
    got = api.gated_backward(*s, "gelu", need_dw=False)
    check_backward("gelu", got, *s)
    apart = [torch.zeros((3, 24, v.shape[2]), dtype=v.dtype, device="cuda")[:, 1:21] for v in (s[0], s[1], s[4], s[5])]
    for a, v in zip(apart, (s[0], s[1], s[4], s[5])):
        a.copy_(v)
    t = (apart[0], apart[1], s[2], s[3], apart[2], apart[3])
    check_backward("gelu", api.gated_backward(*t, "gelu", need_dw=False), *s)
    check_backward("gelu", api.gated_backward(*t, "gelu"), *s)
    out = torch.full((3, 30, 2056), 7, dtype=s[1].dtype, device="cuda")
    api.gated_backward(*t, "gelu", need_dw=False, out=(out[:, 5:25], None, None))
    check_backward("gelu", (out[:, 5:25], None, None), *s)
    assert (out[:, :5] == 7).all() and (out[:, 25:] == 7).all()


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_gated_backward_far_out(api, kind, dtype):
    """Gates as large as the type holds, where the slope is 0 or 1 to the last
    bit: with x and w_gate identities the gradients are dg and du themselves, and
    with dh and u powers of two those are exact."""
    import torch
    t = dtype_of(dtype)
    top = [1e3, 3e4, 65504.0] if dtype == "float16" else [1e3, 1e10, 8e18, 9e19, 1e30, 3e38]
    v = torch.tensor((top + [-a for a in top] + [0.0] * 16)[:16], dtype=torch.float64, device="cuda").to(t)
    g = v.expand(16, 16).contiguous()
    dh, u = torch.full_like(g, 2.0 ** -3), torch.full_like(g, 2.0 ** -5)
    eye, zero = torch.eye(16, device="cuda", dtype=t), torch.zeros(16, 16, device="cuda", dtype=t)
    a, slope = activation(kind, g.double())
    dg, du = (dh.double() * u.double() * slope).to(t), (dh.double() * a).to(t)
    dx, dwg, dwu = api.gated_backward(dh, eye, eye, zero, g, u, kind)
    assert torch.equal(dwg, dg.t()) and torch.equal(dwu, du.t()) and torch.equal(dx, dg)


@pytest.mark.parametrize("size", [(1 << 22, 64, 64), (1 << 22, 40, 61), (64, 1 << 21, 64), (3, (1 << 21) + 40, 61)])
def test_gated_backward_of_many_tokens_and_wide_blocks(api, size):
    """Whole numbers whose sums fp32 holds exactly (below 2^24): bit for bit."""
    import torch
    M, F, K = size
    bits = lambda seed, *shape: integers(seed, -1, 1, *shape).to(torch.int8).bfloat16()
    dh, x, wg, wu = bits(1, M, F), bits(2, M, K), bits(3, F, K), bits(4, F, K)
    g, u = bits(5, M, F), bits(6, M, F)
    dx, dwg, dwu = api.gated_backward(dh, x, wg, wu, g, u, "relu")
    dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp_min(0)).double()
    assert torch.equal(dwg, (dg.t() @ x.double()).bfloat16()) and torch.equal(dwu, (du.t() @ x.double()).bfloat16())
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).bfloat16())


def test_gated_backward_of_many_sequences_apart(api):
    """2^16 sequences of two tokens with a row between them, weights shared."""
    import torch
    B, M, F, K = 1 << 16, 2, 64, 48
    bits = lambda seed, *shape: integers(seed, -1, 1, *shape).to(torch.int8).bfloat16()
    dh, wg, wu, g, u = bits(1, B, M, F), bits(3, F, K), bits(4, F, K), bits(5, B, M, F), bits(6, B, M, F)
    x = bits(2, B, M + 1, K)[:, 1:]
    dx, dwg, dwu = api.gated_backward(dh, x, wg, wu, g, u, "relu")
    dg, du = ((dh * u * (g > 0)).double().view(-1, F), (dh * g.clamp_min(0)).double().view(-1, F))
    flat = x.double().reshape(-1, K)
    assert torch.equal(dwg, (dg.t() @ flat).bfloat16()) and torch.equal(dwu, (du.t() @ flat).bfloat16())
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).bfloat16().view(B, M, K))


def test_gated_longest_rows(api):
    """K of 2^30 - 8: rows that end 16 bytes short of 2^31.  Whole numbers whose
    sums fp32 holds exactly."""
    import torch
    K = (1 << 30) - 8

    def bits(seed):
        out = torch.empty(1, K, dtype=torch.bfloat16, device="cuda")
        generator = gen(seed)
        for part in out[0].split(1 << 26):
            part.copy_(torch.randint(-1, 2, part.shape, generator=generator, device="cuda", dtype=torch.int8))
        return out
    x, wg, wu = bits(1), bits(2), bits(3)
    x[0, -8:], wg[0, -8:], wu[0, -8:] = 1, 30, 60      # the last chunk counts
    h, g, u = api.gated(x, wg, wu, "relu", keep=True)
    dot = lambda w: sum(int((a.int() * b.int()).sum()) for a, b in zip(x[0].split(1 << 26), w[0].split(1 << 26)))
    G, V = dot(wg), dot(wu)
    assert abs(G) < 1 << 20 and abs(V) < 1 << 20
    of = lambda v: float(torch.tensor(v, dtype=torch.float32).bfloat16())
    assert float(g) == of(G) and float(u) == of(V) and float(h) == of(float(max(G, 0) * V))


@pytest.mark.parametrize("rows,cols,how", [(5, 100, "rows"), (5, 3000, "rows"), (1100, 3000, "rows"), (5, 9000, "rows"), (5, 20000, "rows"), (70, 100, "cols")])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_quantize_rows_of_no_numbers(api, dtype, rows, cols, how):
    """Rows of NaN alone, of infinities alone and of both among numbers: scale NaN, codes 0."""
    import torch
    x = normal(6, rows, cols).to(dtype_of(dtype))
    clean = api.quantize_rows(x)
    x[0], x[1], x[2, ::2], x[2, 1::4], x[3, cols // 2] = float("nan"), -float("inf"), float("inf"), float("nan"), float("inf")
    q, s = api.quantize_rows(strided(x, how))
    assert torch.isnan(s[:4]).all() and not q[:4].any()
    assert torch.equal(q[4:], clean[0][4:]) and torch.equal(s[4:], clean[1][4:])


def test_gated_backward_past_fp16(api):
    """A dg from 65520 on is infinite: with it go its row of dx and its row of
    dw_gate, and nothing else."""
    import torch
    for shape in ((5, 40, 72), (300, 520, 264)):
        s = list(state(3, shape, "float16", "relu"))
        s[4][2, 7], s[0][2, 7], s[5][2, 7] = 0.5, 0.25, 0.125
        want = api.gated_backward(*s, "relu")
        s[0][2, 7], s[5][2, 7] = 300.0, 300.0        # dg 90000, du 150
        dx, dwg, dwu = api.gated_backward(*s, "relu")
        m, f = torch.arange(shape[0], device="cuda") != 2, torch.arange(shape[1], device="cuda") != 7
        assert not torch.isfinite(dx[2]).any() and not torch.isfinite(dwg[7]).any()
        assert torch.equal(dx[m], want[0][m]) and torch.equal(dwg[f], want[1][f]) and torch.equal(dwu[f], want[2][f])
        assert torch.isfinite(dwu).all()


@pytest.mark.parametrize("batch,M,N,K", [(16, 1, 8190, 1040), (16, 16, 8190, 1040), (16, 17, 8190, 144), (24, 33, 2100, 528), (16, 64, 8190, 1040),
                                         (1, 17, 70001, 256), (1, 64, 140000, 80)])
def test_few_rows_in_large_tiles(api, batch, M, N, K):
    """Up to 64 rows where reading B once does not bound the call."""
    a, b, sa, sb = codes(1, batch, M, K), codes(2, batch, N, K), scales(3, batch, M), scales(4, batch, N)
    d = normal(5, batch, M, N).bfloat16()
    args = api.make_args(a, b, None, d, sa, sb)
    assert api.sl_gemm_plan(args)["tile_m"] >= 128
    check_int8(api, a, b, sa, sb)
    check_int8(api, a, b, sa, sb, d)
    if batch > 1:
        for dtype in ("float16", "bfloat16"):
            x, wg, wu = block(1, (M, N // 2, K // 2), dtype, (batch,))
            check_gated("gelu", api.gated(x, wg, wu, "gelu", keep=True), x, wg, wu)
            s = state(2, (M, N // 8, K // 2), dtype, "silu", (batch,))
            check_backward("silu", api.gated_backward(*s, "silu"), *s)
