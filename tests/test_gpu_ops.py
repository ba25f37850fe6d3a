"""Block quantisation, the block-scaled 8-bit product and the orthogonalised
update on the GPU, against plain implementations in 64 bits."""

import math

import pytest

pytestmark = pytest.mark.gpu

BLOCK = 128
TOP = 448.0
TINY = 2.0 ** -100


@pytest.fixture(scope="module")
def api():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from stride_layouts_lds_amd import api as A
    A.lib()
    return A


def blocks(n):
    return -(-n // BLOCK)


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def same_bytes(x, y):
    import torch
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def strided(x, how):
    """x's values in another storage: "rows" row-major, "cols" column-major,
    "padded" row-major with rows off 16 bytes, "sparse" no unit stride."""
    import torch
    if how == "rows":
        return x.contiguous()
    if how == "cols":
        return x.mT.contiguous().mT
    pad = 3 if how == "padded" else 5
    step = 1 if how == "padded" else 2
    store = torch.full(x.shape[:-1] + (step * x.shape[-1] + pad,), 7.0, dtype=x.dtype, device=x.device)
    v = store[..., 1:1 + step * x.shape[-1]:step]
    v.copy_(x)
    return v


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def e4m3_steps(v):
    """E4M3's spacing at the 64-bit values v."""
    import torch
    _, e = torch.frexp(v.abs())
    return torch.exp2((e.double() - 1).clamp_min(-6.0) - 3.0)


def block_tops(x, block_rows):
    """Largest magnitudes of x's blocks (64-bit), at least TINY."""
    import torch
    batch, (R, C) = x.shape[:-2], x.shape[-2:]
    br, bc = -(-R // block_rows), blocks(C)
    full = torch.zeros(batch + (br * block_rows, bc * BLOCK), dtype=torch.float64, device=x.device)
    full[..., :R, :C] = x.abs()
    return full.view(batch + (br, block_rows, bc, BLOCK)).amax(dim=(-3, -1)).clamp_min(TINY)


def spread_scales(s, block_rows, R, C):
    """Block values at every element."""
    return s.repeat_interleave(block_rows, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :C]


def check_codes(q, s, x, block_rows):
    """q and s against their definition: scales bit for bit, codes the nearest
    value to 448 x / top in 64 bits, or, where that quotient rounded to fp32
    is a tie, one of the tie's two."""
    import torch
    x = x.double()
    R, C = x.shape[-2:]
    top = block_tops(x, block_rows)
    assert torch.equal(s, (top / 448.0).float())
    assert q.shape[-1] == -(-C // 16) * 16 and q.shape[-2] == R
    assert not q[..., C:].view(torch.uint8).any()
    v = x * TOP / spread_scales(top, block_rows, R, C)
    step = e4m3_steps(v)
    want = (torch.round(v / step) * step).clamp(-TOP, TOP)
    got = q[..., :C].double()
    off = got != want
    # fp32 x: 448 x and the quotient are each rounded, 2^-24 apiece
    near_tie = (((v / step) - torch.floor(v / step) - 0.5).abs() <= 2.0 ** -22 * (v / step).abs())
    ok = ~off | (near_tie & ((got - want).abs() <= step * 1.0001))
    assert bool(ok.all()), f"{int((~ok).sum())} codes differ"
    if x.dtype != torch.float32:
        assert float(off.double().mean()) < 1e-3


SIZES = [(1, 1), (1, 128), (1, 4096), (3, 16), (7, 100), (64, 129), (127, 127), (128, 128), (129, 257), (200, 640),
         (1000, 72), (515, 1023)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(api, size, dtype, block_rows):
    import torch
    x = torch.randn(size, generator=gen(1), device="cuda") * torch.exp(torch.randn(size[1], generator=gen(2), device="cuda"))
    x = x.to(getattr(torch, dtype))
    q, s = api.quantize(x, block_rows=block_rows)
    check_codes(q, s, x, block_rows)
    q2, s2, qt, st = api.quantize(x, block_rows=block_rows, transposed=True)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    check_codes(qt, st, x.t(), block_rows)
    qt3, st3 = api.quantize(x, block_rows=block_rows, transposed=True, direct=False)
    assert torch.equal(qt3.view(torch.uint8), qt.view(torch.uint8)) and torch.equal(st3, st)


@pytest.mark.parametrize("how", ["cols", "padded", "sparse"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_strides_and_batches(api, how, dtype, block_rows):
    import torch
    x = strided(torch.randn((3, 150, 333), generator=gen(3), device="cuda").to(getattr(torch, dtype)), how)
    q, s, qt, st = api.quantize(x, block_rows=block_rows, transposed=True)
    check_codes(q, s, x, block_rows)
    check_codes(qt, st, x.mT, block_rows)
    q1, s1 = api.quantize(x, block_rows=block_rows)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, s)
    # one batch read for all (stride 0), and scales of other strides
    shared = x[:1].expand(3, -1, -1)
    out = (torch.empty((3, 150, 384), dtype=torch.float8_e4m3fn, device="cuda"),
           torch.empty((3, -(-150 // block_rows), 3), device="cuda"))
    api.quantize(shared, block_rows=block_rows, out=out)
    for b in range(3):
        assert torch.equal(out[0][b, :, :336].view(torch.uint8), q[0].view(torch.uint8))
        assert not out[0][b, :, 336:].view(torch.uint8).any()
        assert torch.equal(out[1][b], s[0])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_extremes(api, block_rows, transposed):
    """Zeros, the smallest and largest values, a NaN and infinities: a block
    that holds one of those is NaN throughout, the others are untouched."""
    import torch
    x = torch.randn((256, 384), generator=gen(4), device="cuda")
    x[0:128, 0:128] = 0
    x[128, 130] = 3.0e38
    x[130, 131] = 1e-45
    x[200:, 256:] *= 1e-38
    clean = api.quantize(x, block_rows=block_rows, transposed=transposed)
    check_codes(clean[0], clean[1], x, block_rows)
    if transposed:
        check_codes(clean[2], clean[3], x.t(), block_rows)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[5, 300] = bad
        out = api.quantize(y, block_rows=block_rows, transposed=transposed)
        for q, s, q0, s0, v in [(out[0], out[1], clean[0], clean[1], y)] + ([(out[2], out[3], clean[2], clean[3], y.t())] if transposed else []):
            hit = torch.zeros_like(s, dtype=torch.bool)
            r, c = (5, 300) if v is y else (300, 5)
            hit[r // block_rows, c // 128] = True
            assert torch.equal(torch.isnan(s), hit)
            assert torch.equal(s[~hit], s0[~hit])
            every = spread_scales(hit, block_rows, *v.shape)
            codes = q[:, :v.shape[1]].float()
            assert torch.equal(torch.isnan(codes), every)
            assert torch.equal(codes[~every], q0[:, :v.shape[1]].float()[~every])


def test_quantize_many_rows(api):
    """More than 2^32 elements: offsets pass 32 bits."""
    import torch
    rows = (1 << 32) // 4096 + 130
    x = torch.zeros((rows, 4096), dtype=torch.float16, device="cuda")
    x[-200:] = torch.randn((200, 4096), generator=gen(5), device="cuda").half()
    q, s = api.quantize(x)
    check_codes(q[-256:], s[-256:], x[-256:], 1)
    assert not q[:-200].view(torch.uint8)[::1009].any()


def test_quantize_on_another_stream(api):
    import torch
    x = torch.randn((300, 500), generator=gen(6), device="cuda").half()
    want = api.quantize(x, transposed=True)
    out = tuple(torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.quantize(x, transposed=True, out=out)
    side.synchronize()
    for a, b in zip(out, want):
        assert same_bytes(a, b)


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------

def int_codes(shape, seed, most=4):
    import torch
    return torch.randint(-most, most + 1, shape, generator=gen(seed), device="cuda").to(torch.float8_e4m3fn)


def scales(batch, rows, k, block_rows, seed, powers=True):
    import torch
    shape = batch + (-(-rows // block_rows), blocks(k))
    if powers:
        return torch.exp2(torch.randint(-3, 4, shape, generator=gen(seed), device="cuda").float())
    return torch.exp(torch.randn(shape, generator=gen(seed), device="cuda"))


def product64(a, sa, ra, b, sb, rb, c):
    """(D, sum of magnitudes) in 64 bits."""
    import torch
    K = a.shape[-1]
    av = a.double() * spread_scales(sa.double(), ra, a.shape[-2], K)
    bv = b.double() * spread_scales(sb.double(), rb, b.shape[-2], K)
    d = torch.matmul(av, bv.mT.contiguous())
    size = torch.matmul(av.abs(), bv.abs().mT.contiguous())
    return (d if c is None else d + c.double()), size


OUTS = ["float16", "bfloat16", "float32"]
# M, N, K: every tile's edges, one row, K from one sixteenth of a block up
SHAPES = [(1, 16, 16), (1, 1, 128), (1, 4096, 4096), (2, 33, 144), (15, 100, 256), (17, 48, 1024), (33, 64, 2064),
          (48, 513, 640), (64, 257, 112), (65, 65, 384), (100, 3, 512), (129, 130, 272), (200, 1000, 1040),
          (300, 264, 128), (513, 200, 4096), (600, 770, 2064)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("blocks_of", [(1, 128), (1, 1), (128, 128)])
def test_product_exact(api, shape, out, blocks_of):
    """Small integers and powers of two: every sum is exact in fp32, so D is
    the exact result rounded once."""
    import torch
    M, N, K = shape
    ra, rb = blocks_of
    a, b = int_codes((M, K), 11, 2), int_codes((N, K), 12, 2)
    sa, sb = scales((), M, K, ra, 13), scales((), N, K, rb, 14)
    c = torch.randint(-8, 9, (M, N), generator=gen(15), device="cuda").to(getattr(torch, out)) if M % 2 else None
    got = api.gemm(a, b, c, sfa=sa, sfb=sb, block_k=128, dtype=getattr(torch, out))
    want, _ = product64(a, sa, ra, b, sb, rb, c)
    assert torch.equal(got, want.to(torch.float32).to(getattr(torch, out)))


@pytest.mark.parametrize("shape", [(1, 4096, 4096), (48, 1000, 2064), (300, 520, 4096), (1030, 1100, 1040)])
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("rb", [1, 128])
def test_product_close(api, shape, out, rb):
    """Codes and scales over their whole range.  A block's sum on the 8-bit
    instruction (16-bit D) keeps bits down to 2^-16 of its largest product or
    better, over at most 128 products: 2^-11 of the sum of magnitudes covers
    it; on the fp16 instruction (fp32 D) 2^-24 for each of the additions."""
    import torch
    M, N, K = shape
    dt = getattr(torch, out)
    wide = lambda shp, seed: (torch.randn(shp, generator=gen(seed), device="cuda") *
                              torch.exp(torch.randn(shp, generator=gen(seed + 1), device="cuda")) * 8).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    a, b = wide((M, K), 21), wide((N, K), 23)
    sa, sb = scales((), M, K, 1, 25, False), scales((), N, K, rb, 26, False)
    c = torch.randn((M, N), generator=gen(27), device="cuda").to(dt)
    got = api.gemm(a, b, c, sfa=sa, sfb=sb, block_k=128, dtype=dt).double()
    want, size = product64(a, sa, 1, b, sb, rb, c)
    share = 2.0 ** -11 if out != "float32" else (8 + 2 * blocks(K)) * 2.0 ** -24
    bound = torch.finfo(dt).eps / 2 * want.abs() + share * (size + c.double().abs()) * (1 + torch.finfo(dt).eps)
    over = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + bound > torch.finfo(dt).max)
    assert bool((((got - want).abs() <= bound) | over).all())


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("shape", [(33, 72, 400), (150, 140, 272)])
def test_product_batches_strides_and_c(api, out, shape):
    import torch
    M, N, K = shape
    dt = getattr(torch, out)
    a, b = int_codes((3, M, K), 31, 2), int_codes((3, N, K), 32, 2)
    sa, sb = scales((3,), M, K, 1, 33), scales((3,), N, K, 128, 34)
    c = torch.randint(-8, 9, (3, M, N), generator=gen(35), device="cuda").to(dt)
    want = product64(a, sa, 1, b, sb, 128, c)[0].float().to(dt)
    assert torch.equal(api.gemm(a, b, c, sfa=sa, sfb=sb, block_k=128, dtype=dt), want)
    # C is D; scales with the rows contiguous; D column-major and with gaps
    buf = c.clone()
    api.gemm(a, b, buf, out=buf, sfa=sa.mT.contiguous().mT, sfb=sb.mT.contiguous().mT, block_k=128)
    assert torch.equal(buf, want)
    for how in ("cols", "padded", "sparse"):
        d = strided(torch.zeros((3, M, N), dtype=dt, device="cuda"), how)
        api.gemm(a, b, strided(c, how), out=d, sfa=sa, sfb=sb, block_k=128)
        assert torch.equal(d, want)
    # a weight shared by the batch (rank 2 and stride 0), C one row for all rows
    row = c[:1, :1].expand(3, M, N)
    want = product64(a, sa, 1, b[:1].expand(3, N, K), sb[:1].expand(3, -1, -1), 128, row)[0].float().to(dt)
    assert torch.equal(api.gemm(a, b[0], row, sfa=sa, sfb=sb[0], block_k=128, dtype=dt), want)
    assert torch.equal(api.gemm(a, b[:1].expand(3, N, K), row, sfa=sa, sfb=sb[:1].expand(3, -1, -1), block_k=128, dtype=dt), want)
    # rows of A inside a larger buffer whose other bytes are NaN codes
    store = torch.full((M, K + 64), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    store[:, 16:16 + K] = a[0]
    want = product64(a[0], sa[0], 1, b[0], sb[0], 128, None)[0].float().to(dt)
    assert torch.equal(api.gemm(store[:, 16:16 + K], b[0], sfa=sa[0], sfb=sb[0], block_k=128, dtype=dt), want)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("M", [5, 100])
def test_product_nan_and_empty(api, out, M):
    """A NaN code or scale reaches its row alone; K = 0 gives C; M or N = 0
    nothing."""
    import torch
    dt = getattr(torch, out)
    a, b = int_codes((M, 512), 41, 2), int_codes((80, 512), 42, 2)
    sa, sb = scales((), M, 512, 1, 43), scales((), 80, 512, 1, 44)
    clean = api.gemm(a, b, sfa=sa, sfb=sb, block_k=128, dtype=dt)
    a2 = a.float()
    a2[3, 200] = float("nan")
    got = api.gemm(a2.to(torch.float8_e4m3fn), b, sfa=sa, sfb=sb, block_k=128, dtype=dt)
    sb2 = sb.clone()
    sb2[7, 1] = float("nan")
    got2 = api.gemm(a, b, sfa=sa, sfb=sb2, block_k=128, dtype=dt)
    for g, dim, at in ((got, 0, 3), (got2, 1, 7)):
        assert bool(torch.isnan(g.select(dim, at)).all())
        keep = [i for i in range(g.shape[dim]) if i != at]
        assert torch.equal(g.index_select(dim, torch.tensor(keep, device="cuda")),
                           clean.index_select(dim, torch.tensor(keep, device="cuda")))
    c = torch.randn((M, 80), generator=gen(45), device="cuda").to(dt)
    z = api.gemm(a[:, :0], b[:, :0], c, sfa=sa[:, :0], sfb=sb[:, :0], block_k=128, dtype=dt)
    assert torch.equal(z, c)
    assert api.gemm(a[:0], b, sfa=sa[:0], sfb=sb, block_k=128, dtype=dt).shape == (0, 80)
    # overflow of D's type gives infinities, as for every other product
    if dt == torch.float16:
        big = torch.full((M, 1), 2.0 ** 10, device="cuda").expand(M, 4).contiguous()
        inf = api.gemm(torch.full((M, 512), 448.0, device="cuda").to(torch.float8_e4m3fn), b.float().abs().add(1).to(torch.float8_e4m3fn),
                       sfa=big, sfb=torch.ones_like(sb), block_k=128, dtype=dt)
        assert bool(torch.isinf(inf).all())


def test_product_far_rows(api):
    """Operands whose rows lie past 2^32 bytes."""
    import torch
    N, K = (1 << 32) // 4096 + 300, 4096
    b = torch.zeros((N, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    b[-300:] = int_codes((300, K), 51, 2)
    sb = torch.ones((N, 1), device="cuda").expand(N, 32)
    a, sa = int_codes((4, K), 52, 2), scales((), 4, K, 1, 53)
    got = api.gemm(a, b, sfa=sa, sfb=sb, block_k=128, dtype=torch.float32)
    want, _ = product64(a, sa, 1, b[-300:], sb[-300:], 1, None)
    assert torch.equal(got[:, -300:], want.float())
    assert not got[:, :-300].any()
    # the same rows as A of a large product
    sc = scales((), 200, K, 128, 54)
    w = int_codes((200, K), 55, 2)
    got = api.gemm(b[-70000:], w, sfa=sb[-70000:], sfb=sc, block_k=128, dtype=torch.float32)
    want, _ = product64(b[-300:], sb[-300:], 1, w, sc, 128, None)
    assert torch.equal(got[-300:], want.float()) and not got[:-300].any()


def test_quantize_then_product(api):
    """The chain a linear layer runs: the product of quantised operands is the
    product of the values their codes and scales stand for, and those lie
    within half a step of E4M3 (2^-4) of the inputs."""
    import torch
    x = torch.randn((300, 700), generator=gen(61), device="cuda").bfloat16()
    w = (torch.randn((520, 700), generator=gen(62), device="cuda") / 26).bfloat16()
    q, s, qt, st = api.quantize(x, transposed=True)
    wq, ws, wqt, wst = api.quantize(w, block_rows=128, transposed=True)
    y = api.gemm(q, wq, sfa=s, sfb=ws, block_k=128, dtype=torch.float32)
    want, _ = product64(q, s, 1, wq, ws, 128, None)
    plain = torch.matmul(x.double(), w.double().t().contiguous())
    assert float((y.double() - want).norm() / want.norm()) < 1e-6
    assert float((y.double() - plain).norm() / plain.norm()) < 2 * 2.0 ** -4
    # the gradients' products read the transposes' codes
    g = torch.randn((300, 520), generator=gen(63), device="cuda").bfloat16()
    gq, gs, gqt, gst = api.quantize(g, transposed=True)
    dx = api.gemm(gq, wqt, sfa=gs, sfb=wst, block_k=128, dtype=torch.bfloat16)
    dw = api.gemm(gqt, qt, sfa=gst, sfb=st, block_k=128, dtype=torch.float32)
    for got, ref in ((dx, g.double() @ w.double()), (dw, g.double().t().contiguous() @ x.double())):
        assert got.shape == ref.shape
        assert float((got.double() - ref).norm() / ref.norm()) < 2 * 2.0 ** -4 + 2.0 ** -8


# ---------------------------------------------------------------------------
# the orthogonalised update
# ---------------------------------------------------------------------------

DEFAULT = (3.4445, -4.7750, 2.0315)


def orthogonalize64(x, steps=5, coefficients=None):
    import torch
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + 1e-7)
    co = coefficients or [DEFAULT] * steps
    for a, b, c in co:
        g = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.mT if tall else x


def gradient_like(shape, seed, dtype):
    import torch
    m, n = shape[-2:]
    r = min(8, m, n)
    x = torch.matmul(torch.randn(shape[:-1] + (r,), generator=gen(seed), device="cuda"),
                     torch.randn(shape[:-2] + (r, n), generator=gen(seed + 1), device="cuda"))
    return ((0.5 * x + torch.randn(shape, generator=gen(seed + 2), device="cuda")) * 1e-3).to(getattr(torch, dtype))


def ortho_tolerance(dt):
    """Relative, 2-norm.  The result's own rounding is half a step at most.
    bf16 results: the matrices between products are fp16, which costs up to
    1.8e-3 in a 64-bit simulation of those roundings (16 x 16 to 1000 x 1000),
    below another half step; fp16 results: pairs of fp16, 3e-7 there, 2^-17
    allowed."""
    import torch
    return torch.finfo(dt).eps / 2 + (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -17)


ORTHO_SIZES = [(1, 1), (1, 300), (16, 16), (17, 40), (64, 64), (65, 63), (96, 128), (128, 129), (100, 1000), (1000, 100),
               (130, 520), (300, 256), (513, 640), (1000, 520), (257, 2100)]


@pytest.mark.parametrize("size", ORTHO_SIZES)
@pytest.mark.parametrize("dtype,out", [("bfloat16", "bfloat16"), ("float16", "float16"), ("float32", "bfloat16"),
                                       ("float32", "float16")])
def test_orthogonalize(api, size, dtype, out):
    import torch
    dt = getattr(torch, out)
    x = gradient_like(size, 71, dtype)
    keep = x.clone()
    d = torch.full(size, 7.0, dtype=dt, device="cuda")
    assert api.orthogonalize(x, out=d) is d
    want = orthogonalize64(x)
    assert torch.equal(x, keep)
    assert float((d.double() - want).norm() / want.norm()) <= ortho_tolerance(dt)
    assert torch.equal(api.orthogonalize(x, out=torch.empty_like(d)), d)  # the same from call to call


@pytest.mark.parametrize("how", ["rows", "cols", "padded", "sparse"])
@pytest.mark.parametrize("shape", [(4, 96, 72), (3, 60, 200), (2, 330, 260)])
def test_orthogonalize_batches_and_strides(api, how, shape):
    import torch
    for dtype in ("bfloat16", "float16"):
        dt = getattr(torch, dtype)
        x = strided(gradient_like(shape, 81, dtype), how)
        x[1] *= 100.0  # each matrix by its own norm
        d = strided(torch.zeros(shape, dtype=dt, device="cuda"), how)
        api.orthogonalize(x, out=d)
        want = orthogonalize64(x)
        for b in range(shape[0]):
            assert float((d[b].double() - want[b]).norm() / want[b].norm()) <= ortho_tolerance(dt)
            one = api.orthogonalize(x[b])
            assert float((one.double() - want[b]).norm() / want[b].norm()) <= ortho_tolerance(dt)
        api.orthogonalize(x, out=x)  # in place
        assert torch.equal(x, d)


def test_orthogonalize_steps_and_coefficients(api):
    import torch
    x = gradient_like((90, 200), 91, "float16")
    co = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    for steps, given in ((1, None), (3, co), (3, (1.875, -1.25, 0.375)), (12, None)):
        d = api.orthogonalize(x, steps=steps, coefficients=given)
        each = None if given is None else (given if isinstance(given, list) else [given] * steps)
        want = orthogonalize64(x, steps, each)
        # twelve steps carry a rounding further than five: a singular value's
        # error grows by the polynomial's slope, up to 3.45 a step while it is small
        assert float((d.double() - want).norm() / want.norm()) <= 4 * ortho_tolerance(torch.float16)


def test_orthogonalize_spectrum(api):
    """Singular values from 1 to 0.02 of the largest come out within the
    polynomial's band."""
    import torch
    u, _ = torch.linalg.qr(torch.randn((200, 200), generator=gen(95), device="cuda"))
    v, _ = torch.linalg.qr(torch.randn((300, 200), generator=gen(96), device="cuda"))
    s = torch.logspace(0, math.log10(0.02), 200, device="cuda")
    d = api.orthogonalize((torch.matmul(u * s, v.t().contiguous())).half())
    got = torch.linalg.svdvals(d.float())
    assert 0.6 < float(got.min()) and float(got.max()) < 1.3


@pytest.mark.parametrize("size", [(40, 60), (200, 300)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_orthogonalize_extremes(api, size, dtype):
    import torch
    dt = getattr(torch, dtype)
    assert not api.orthogonalize(torch.zeros(size, dtype=dt, device="cuda")).any()
    for bad in (float("nan"), float("inf")):
        x = gradient_like((2,) + size, 97, dtype)
        clean = api.orthogonalize(x)
        x[0, 3, 4] = bad
        d = api.orthogonalize(x)
        assert bool(torch.isnan(d[0]).all()) and torch.equal(d[1], clean[1])
    # the largest and the smallest values: the norm neither overflows nor vanishes
    x = torch.randn(size, generator=gen(98), device="cuda").sign()
    for scale in ((3e38, 1.0, 1e-4) if dt == torch.bfloat16 else (60000.0, 1.0, 2.0 ** -14)):
        y = (x * scale).to(dt)
        want = orthogonalize64(y)
        assert float((api.orthogonalize(y).double() - want).norm() / want.norm()) <= ortho_tolerance(dt)
    assert api.orthogonalize(torch.zeros((0, 5), dtype=dt, device="cuda")).shape == (0, 5)


def test_orthogonalize_in_a_graph(api):
    """Captured, replayed with the program's own work between, on new values."""
    import torch
    x = gradient_like((3, 200, 150), 101, "float16")
    d = torch.empty_like(x)
    q, s, qt, st = api.quantize(x[0], transposed=True)
    args = api.sl_orthogonalize_args()
    args.x, args.d, args.steps = api.tensor_desc(x), api.tensor_desc(d), 5
    ws = torch.empty(api.sl_orthogonalize_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    y = torch.empty((200, 200), dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.orthogonalize(x, out=d, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.orthogonalize(x, out=d, workspace=ws)
        api.quantize(d[0], transposed=True, out=(q, s, qt, st))
        api.gemm(q, q, sfa=s, sfb=s, block_k=128, out=y)
    for seed in (102, 103, 104, 105):
        x.copy_(gradient_like((3, 200, 150), seed, "float16"))
        ws.fill_(255)  # the workspace's contents do not matter
        graph.replay()
        torch.cuda.synchronize()
        want = api.orthogonalize(x)
        assert torch.equal(d, want)
        wq = api.quantize(want[0], transposed=True)
        for got, ref in zip((q, s, qt, st), wq):
            assert same_bytes(got, ref)
        assert torch.equal(y, api.gemm(wq[0], wq[0], sfa=wq[1], sfb=wq[1], block_k=128, dtype=torch.float32))
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# the tiles of large results
# ---------------------------------------------------------------------------

# 256 x 256 tiles (16-bit D) and 128 x 128 ones two to a CU; 128 x 128 tiles
# four K-tiles deep
@pytest.mark.parametrize("shape", [(2100, 4300, 16), (2100, 4300, 400), (4090, 2310, 2064), (1290, 1500, 128),
                                   (1290, 1500, 1040), (1025, 1030, 656)])
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("rb", [1, 128])
def test_product_large_tiles(api, shape, out, rb):
    import torch
    M, N, K = shape
    dt = getattr(torch, out)
    a, b = int_codes((M, K), 111, 2), int_codes((N, K), 112, 2)
    sa, sb = scales((), M, K, 1, 113), scales((), N, K, rb, 114)
    c = torch.randint(-8, 9, (M, N), generator=gen(115), device="cuda").to(dt)
    want = product64(a, sa, 1, b, sb, rb, c)[0].float().to(dt)
    d = torch.zeros((M, N), dtype=dt, device="cuda")
    plan = api.sl_gemm_plan(api.make_args(a, b, c, d, sa, sb, 128))
    assert plan["tile_m"] in (128, 256)
    assert torch.equal(api.gemm(a, b, c, out=d, sfa=sa, sfb=sb, block_k=128), want)
    t = strided(torch.zeros((M, N), dtype=dt, device="cuda"), "cols")
    api.gemm(a, b, strided(c, "cols"), out=t, sfa=sa, sfb=sb, block_k=128)
    assert torch.equal(t, want)
    # codes over their whole range, and a NaN's row
    wide = (torch.randn((M, K), generator=gen(116), device="cuda") * 60).clamp(-TOP, TOP)
    wide[7, 3] = float("nan")
    got = api.gemm(wide.to(torch.float8_e4m3fn), b, sfa=sa, sfb=sb, block_k=128, dtype=dt).double()
    ref, size = product64(wide.to(torch.float8_e4m3fn), sa, 1, b, sb, rb, None)
    assert bool(torch.isnan(got[7]).all())
    rest = torch.arange(M, device="cuda") != 7
    share = 2.0 ** -11 if out != "float32" else (8 + 2 * blocks(K)) * 2.0 ** -24
    bound = torch.finfo(dt).eps / 2 * ref.abs() + share * size * (1 + torch.finfo(dt).eps)
    over = torch.isinf(got) & (got.sign() == ref.sign()) & (ref.abs() + bound > torch.finfo(dt).max)
    assert bool((((got - ref).abs() <= bound) | over)[rest].all())


@pytest.mark.parametrize("shape,dtype,out", [
    ((3900, 4090), "bfloat16", "bfloat16"),   # direct, one plane: ring tiles, edges and what is left of a round
    ((4090, 3900), "float16", "float16"),     # Gram, pairs, ring tiles, x and d tall
    ((3840, 4200), "float32", "float16"),     # x itself a pair
    ((1100, 5000), "bfloat16", "bfloat16"),   # Gram for a wide matrix
    ((2, 2050, 2100), "float16", "float16"),
])
def test_orthogonalize_large_tiles(api, shape, dtype, out):
    import torch
    dt = getattr(torch, out)
    x = gradient_like(shape, 121, dtype)
    d = api.orthogonalize(x, out=torch.empty(shape, dtype=dt, device="cuda"))
    want = orthogonalize64(x)
    for b in range(shape[0] if len(shape) == 3 else 1):
        g, w = (d[b], want[b]) if len(shape) == 3 else (d, want)
        assert float((g.double() - w).norm() / w.norm()) <= ortho_tolerance(dt)


def test_orthogonalize_large_direct_pairs(api):
    """Steps that amplify too much for the Gram matrix, on ring tiles."""
    import torch
    x = gradient_like((3900, 4090), 131, "float16")
    co = [DEFAULT] * 6
    d = api.orthogonalize(x, steps=6, coefficients=co)
    want = orthogonalize64(x, 6, co)
    assert float((d.double() - want).norm() / want.norm()) <= 4 * ortho_tolerance(torch.float16)


# ---------------------------------------------------------------------------
# inputs with directions in which x has (almost) nothing
# ---------------------------------------------------------------------------

def poor_rank(kind, shape, seed, dtype):
    """Of few strong directions, of singular values over decades, or with most
    rows zero."""
    import torch
    m, n = shape
    normal = lambda s, *shp: torch.randn(shp, generator=gen(s), device="cuda", dtype=torch.float64)
    if kind.startswith("rank"):
        r = int(kind[4:])
        x = torch.matmul(normal(seed, m, r), normal(seed + 1, r, n))
    elif kind.startswith("decades"):
        k = min(m, n)
        u, _ = torch.linalg.qr(normal(seed, m, k))
        v, _ = torch.linalg.qr(normal(seed + 1, n, k))
        x = torch.matmul(u * torch.logspace(0, -int(kind[7:]), k, device="cuda", dtype=torch.float64), v.t().contiguous())
    else:
        x = normal(seed, m, n)
        x[m // 8:] = 0
    return (x * 1e-3).to(getattr(torch, dtype))


# 2-norm, relative.  A bf16 result's rounding is uniform within half a step, which is at most 2^-8 of
# the value: 2^-8 / sqrt(3) = 2.26e-3 at most.  Next to it stand, for five default steps, what a 64-bit
# simulation of the fp16 roundings of X (as a factor), G and B gave, 2.8e-3 at most (few equal rows
# among zeros), and, for steps that amplify more and run on pairs, 1e-4.
BF16_ROUNDING = 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("kind", ["rank1", "rank8", "rank64", "decades2", "decades4", "rows"])
@pytest.mark.parametrize("shape,dtype", [((300, 400), "bfloat16"), ((300, 400), "float32"), ((1000, 1000), "bfloat16"),
                                         ((2100, 530), "float32"), ((3900, 4090), "bfloat16")])
@pytest.mark.parametrize("steps", [5, 6])
def test_orthogonalize_poor_rank(api, kind, shape, dtype, steps):
    import torch
    x = poor_rank(kind, shape, 141, dtype)
    d = api.orthogonalize(x, out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"), steps=steps)
    want = orthogonalize64(x, steps)
    inside = 2.9e-3 if steps == 5 else 1.1e-4
    assert float((d.double() - want).norm() / want.norm()) <= (BF16_ROUNDING ** 2 + inside ** 2) ** 0.5


@pytest.mark.parametrize("norm", [1e-6, 1e-8, 3e-10, 1e-11, 1e-13, 1e-16, 1e-24, 1e-33])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shape,steps", [((96, 128), 5), ((300, 400), 5), ((300, 400), 6), ((140, 1000), 5), ((1500, 1600), 5)])
def test_orthogonalize_small_norms(api, norm, dtype, shape, steps):
    """Norms about and far below the 1e-7 that is added to them: the result is
    small then, and as accurate as any other."""
    import torch
    x = torch.randn((2,) + shape, generator=gen(151), device="cuda", dtype=torch.float64)
    x[0] *= norm / x[0].norm()  # the other matrix is ordinary
    x = x.to(getattr(torch, dtype))
    d = api.orthogonalize(x, out=torch.empty(x.shape, dtype=torch.bfloat16, device="cuda"), steps=steps)
    want = orthogonalize64(x, steps)
    for b in range(2):
        assert float((d[b].double() - want[b]).norm() / want[b].norm()) <= (BF16_ROUNDING ** 2 + 2.9e-3 ** 2) ** 0.5


# ---------------------------------------------------------------------------
# the `stream` argument
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("op", ["orthogonalize", "gemm", "quantize"])
def test_allocations_belong_to_the_stream(api, op, monkeypatch):
    """A call on another stream than torch's current one takes what it
    allocates from that stream's pool: while its kernels wait there, tensors
    of the same size allocated on the current stream are other memory."""
    import torch
    x = gradient_like((300, 400), 161, "bfloat16")
    a, b = (torch.randn(s, generator=gen(162), device="cuda").half() for s in ((64, 8192), (64, 8192)))
    seen = []
    keep = api.set_workspace

    def record(args, workspace):
        seen.append((workspace.data_ptr(), workspace.numel()))
        keep(args, workspace)
    monkeypatch.setattr(api, "set_workspace", record)
    call = {"orthogonalize": lambda **kw: api.orthogonalize(x, **kw), "gemm": lambda **kw: api.gemm(a, b, **kw),
            "quantize": lambda **kw: api.quantize(x, transposed=True, **kw)}[op]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, 0):
        seen.clear()
        with torch.cuda.stream(side if stream else torch.cuda.default_stream()):
            torch.cuda._sleep(20_000_000)  # some milliseconds; the call's kernels run after it
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            got = call(stream=stream)
            assert (len(seen) > 0) == (op != "quantize")
            outs = got if isinstance(got, tuple) else (got,)
            taken = seen + [(t.data_ptr(), t.numel() * t.element_size()) for t in outs]
            fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _, n in taken for _ in range(3)]
            for f in fill:
                for at, n in taken:
                    assert f.data_ptr() + f.numel() <= at or at + n <= f.data_ptr()
        torch.cuda.synchronize()
        for g, w in zip(outs, want if isinstance(want, tuple) else (want,)):
            assert same_bytes(g, w)


@pytest.mark.parametrize("kind", ["rank64", "decades4"])
@pytest.mark.parametrize("shape", [(140, 1000), (5000, 1100)])
def test_orthogonalize_wide_float32(api, kind, shape):
    """fp32 values with bf16 results, through the Gram matrix: pairs of fp16,
    4e-4 next to the rounding."""
    import torch
    x = poor_rank(kind, shape, 181, "float32")
    d = api.orthogonalize(x)
    want = orthogonalize64(x)
    assert d.dtype == torch.bfloat16
    assert float((d.double() - want).norm() / want.norm()) <= (BF16_ROUNDING ** 2 + 4e-4 ** 2) ** 0.5


@pytest.mark.parametrize("kind", ["rank1", "rank8", "rank64", "decades4", "rows"])
@pytest.mark.parametrize("shape", [(140, 1000), (5000, 1100), (40, 500)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("out", ["bfloat16", "float16"])
def test_orthogonalize_poor_rank_wide(api, kind, shape, dtype, out):
    """Through the Gram matrix (small, wide, or fp16 results): pairs of fp16,
    4e-4 next to the rounding."""
    import torch
    dt = getattr(torch, out)
    x = poor_rank(kind, shape, 181, dtype)
    d = api.orthogonalize(x, out=torch.empty(shape, dtype=dt, device="cuda"))
    want = orthogonalize64(x)
    bound = ((torch.finfo(dt).eps / 2) ** 2 / 3 + 4e-4 ** 2) ** 0.5
    assert float((d.double() - want).norm() / want.norm()) <= bound


# ---------------------------------------------------------------------------
# schedules: other coefficients each step, steep ones first
# ---------------------------------------------------------------------------

SCHEDULE = [(8.287212, -23.595887, 17.300387), (4.107059, -2.947850, 0.544843), (3.948691, -2.908902, 0.551819),
            (3.318420, -2.488488, 0.510049), (2.300652, -1.668904, 0.418807), (1.891301, -1.267996, 0.376804),
            (1.875, -1.25, 0.375), (1.875, -1.25, 0.375)]


@pytest.mark.parametrize("kind", ["rank8", "decades4", "rows"])
@pytest.mark.parametrize("shape", [(96, 128), (300, 400), (1000, 140)])
@pytest.mark.parametrize("out", ["bfloat16", "float16"])
@pytest.mark.parametrize("steps", [3, 4, 8])
def test_orthogonalize_schedules(api, kind, shape, out, steps):
    """Steps that amplify a lot run on pairs of fp16 with fp32 sums: next to
    the result's rounding (uniform within half a step) an iteration in 32 bits
    alone is off by up to 2.4e-4 for these coefficients; twice that."""
    import torch
    dt = getattr(torch, out)
    x = poor_rank(kind, shape, 171, "float32")
    co = [tuple(torch.tensor(c, dtype=torch.float32).tolist()) for c in SCHEDULE[:steps]]  # as the library takes them
    d = api.orthogonalize(x, out=torch.empty(shape, dtype=dt, device="cuda"), steps=steps, coefficients=co)
    want = orthogonalize64(x, steps, co)
    bound = ((torch.finfo(dt).eps / 2) ** 2 / 3 + 4.8e-4 ** 2) ** 0.5
    assert float((d.double() - want).norm() / want.norm()) <= bound


# ---------------------------------------------------------------------------
# codes of 16-bit values, bit for bit
# ---------------------------------------------------------------------------

def exact_codes64(x, block_rows):
    """The nearest E4M3 value to 448 x / top in 64 bits, ties to even.  With
    16-bit x the quotient, if it is not a tie, is further from one than its
    rounding to fp32 moves it: 448 x and the tie times top are whole multiples
    of one unit and have at most 16 bits."""
    import torch
    x = x.double()
    v = x * TOP / spread_scales(block_tops(x, block_rows), block_rows, *x.shape[-2:])
    step = e4m3_steps(v)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def tie_rows(dtype):
    """Rows whose largest value is 7 j 2^e and whose others are m j 2^i: 448
    times such a quotient is m 2^i', for odd m from 17 to 31 halfway between two
    codes, and below 2^-6, where the codes are 2^-9 apart, for every odd m."""
    import torch
    dt = getattr(torch, dtype)
    rows = []
    for j in (1, 3, 5, 7, 9, 11, 13, 29, 33, 61, 65):
        for e in (-9, -3, 0, 4):
            row = [7.0 * j * 2.0 ** e]
            for m in range(1, 32, 2):
                for i in range(-17, 3):
                    for sign in (1, -1):
                        v = sign * m * j * 2.0 ** (e + i)
                        if abs(v) <= row[0] and float(torch.tensor(v, dtype=torch.float64).to(dt)) == v:
                            row.append(v)
            if float(torch.tensor(row[0], dtype=torch.float64).to(dt)) == row[0]:
                rows += [([row[0]] + row[1 + at:128 + at]) for at in range(0, len(row) - 1, 127)]
    x = torch.zeros((len(rows), 128), dtype=torch.float64)
    for r, row in enumerate(rows):
        x[r, :len(row)] = torch.tensor(row, dtype=torch.float64)
    return x.to(dt).cuda()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantize_ties(api, dtype):
    import torch
    x = tie_rows(dtype)
    v = x.double() * TOP / spread_scales(block_tops(x.double(), 1), 1, *x.shape)
    step = e4m3_steps(v)
    ties = (v / step - torch.floor(v / step)) == 0.5
    assert int(ties.sum()) > 1000
    want = exact_codes64(x, 1)
    q, s = api.quantize(x)
    assert torch.equal(q[:, :128].double(), want)
    # both outputs of one pass, along the rows and of the transpose
    q, s, qt, st = api.quantize(x.t().contiguous(), transposed=True)
    assert torch.equal(qt[:, :128].double(), want)
    square = torch.zeros((128 * len(x), 128), dtype=x.dtype, device="cuda")
    square[::128] = x
    q, s = api.quantize(square, block_rows=128)
    assert torch.equal(q[::128, :128].double(), want)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_codes_exact(api, dtype, block_rows):
    """Few bits, so that ties are many, and values over the whole range."""
    import torch
    dt = getattr(torch, dtype)
    for seed, x in ((191, torch.randint(-255, 256, (700, 900), generator=gen(191), device="cuda").to(dt)),
                    (192, torch.randn((700, 900), generator=gen(192), device="cuda").to(dt)),
                    (193, (torch.randn((700, 900), generator=gen(193), device="cuda") *
                           torch.exp(3 * torch.randn((700, 900), generator=gen(194), device="cuda"))).clamp(-6e4, 6e4).to(dt))):
        q, s, qt, st = api.quantize(x, block_rows=block_rows, transposed=True)
        assert torch.equal(q[:, :900].double(), exact_codes64(x, block_rows)), seed
        assert torch.equal(qt[:, :700].double(), exact_codes64(x.t(), block_rows)), seed
        q1, s1 = api.quantize(x, block_rows=block_rows)
        assert same_bytes(q1, q) and torch.equal(s1, s)
