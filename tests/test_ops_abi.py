"""sl_quantize, sl_orthogonalize and the block-scaled form of sl_gemm on the
host (no GPU): every check of their arguments runs before any HIP call, so a
refusal is seen here; what passes the checks is planned, not run."""

import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def api():
    from stride_layouts_lds_amd import api as A
    if not os.path.exists(A.LIB_PATH):
        from stride_layouts_lds_amd import build
        build.build(verbose=False)
    A.lib()
    return A


F16, F32, F8, E8M0, BF16 = 1, 2, 3, 4, 5
X, Q, S, QT, ST, D, WS = (i << 36 for i in range(1, 8))


def rm(ptr, shape, dtype, strides=None):
    """A row-major descriptor's fields, or one with the given strides."""
    if strides is None:
        strides, acc = [0] * len(shape), 1
        for i in reversed(range(len(shape))):
            strides[i], acc = acc, acc * shape[i]
    return ptr, dtype, shape, strides


def refused(api, call, args, what):
    with pytest.raises(api.SLError) as e:
        call(args, 0)
    assert api.STATUS[e.value.status] == what, str(e.value)
    assert str(e.value)


# ------------------------------------------------------------------ quantize

def quantize_args(api, x, q=None, s=None, qt=None, st=None, block_rows=1):
    a = api.sl_quantize_args()
    for name, v in (("x", x), ("q", q), ("s", s), ("qt", qt), ("st", st)):
        if v is not None:
            setattr(a, name, api.desc(*v))
        else:
            getattr(a, name).layout.rank = 2
    a.block_rows = block_rows
    return a


GOOD_Q = dict(x=rm(X, (256, 512), F16), q=rm(Q, (256, 512), F8), s=rm(S, (256, 4), F32),
              qt=rm(QT, (512, 256), F8), st=rm(ST, (512, 2), F32))


@pytest.mark.parametrize("change,what", [
    (dict(x=rm(X, (256, 512), F8)), "SL_ERR_DTYPE"),
    (dict(q=rm(Q, (256, 512), F16)), "SL_ERR_DTYPE"),
    (dict(s=rm(S, (256, 4), F16)), "SL_ERR_DTYPE"),
    (dict(block_rows=64), "SL_ERR_ARG"),
    (dict(block_rows=0), "SL_ERR_ARG"),
    (dict(x=rm(X, (512,), F16)), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (256, 512), F16, (-512, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (256, -512), F16, (512, 1))), "SL_ERR_SHAPE"),
    (dict(q=rm(Q, (256, 496), F8)), "SL_ERR_SHAPE"),                     # fewer columns than x
    (dict(q=rm(Q, (256, 528), F8)), "SL_ERR_SHAPE"),                     # past the last block
    (dict(q=rm(Q, (255, 512), F8)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (256, 3), F32)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (2, 4), F32)), "SL_ERR_SHAPE"),                        # the square blocks' shape
    (dict(qt=rm(QT, (256, 512), F8)), "SL_ERR_SHAPE"),                   # not transposed
    (dict(st=rm(ST, (4, 256), F32)), "SL_ERR_SHAPE"),
    (dict(q=rm(Q, (1, 256, 512), F8), x=rm(X, (2, 256, 512), F16)), "SL_ERR_SHAPE"),
    (dict(x=rm(0, (256, 512), F16)), "SL_ERR_NULL"),
    (dict(q=rm(0, (256, 512), F8), qt=rm(0, (512, 256), F8)), "SL_ERR_NULL"),
    (dict(s=rm(0, (256, 4), F32)), "SL_ERR_NULL"),
    (dict(x=rm(X + 1, (256, 512), F16)), "SL_ERR_ALIGN"),
    (dict(s=rm(S + 2, (256, 4), F32)), "SL_ERR_ALIGN"),
    (dict(q=rm(Q, (256, 512), F8, (1, 256))), "SL_ERR_LAYOUT"),          # columns not contiguous
    (dict(q=rm(Q, (256, 512), F8, (520, 1))), "SL_ERR_LAYOUT"),          # rows off 16 bytes
    (dict(q=rm(Q + 8, (256, 512), F8)), "SL_ERR_LAYOUT"),
    (dict(q=rm(Q, (256, 512), F8, (0, 1))), "SL_ERR_LAYOUT"),            # broadcast output
    (dict(s=rm(S, (256, 4), F32, (1, 0))), "SL_ERR_LAYOUT"),
    (dict(q=rm(X, (256, 512), F8)), "SL_ERR_ALIAS"),
    (dict(qt=rm(Q + 4096, (512, 256), F8)), "SL_ERR_ALIAS"),
    (dict(st=rm(S + 16, (512, 2), F32)), "SL_ERR_ALIAS"),
    (dict(x=rm(X, ((1 << 31) - 128, 1), F16)), "SL_ERR_SHAPE"),
])
def test_quantize_refuses(api, change, what):
    refused(api, api.sl_quantize, quantize_args(api, **{**GOOD_Q, **change}), what)


def test_quantize_null_args_and_empty(api):
    assert api.lib().sl_quantize(None, None) == -1
    for shape in ((0, 512), (256, 0)):
        R, C = shape
        kb = lambda n: (n + 127) // 128
        api.sl_quantize(quantize_args(api, rm(0, shape, F16), rm(0, shape, F8), rm(0, (R, kb(C)), F32)), 0)
        api.sl_quantize(quantize_args(api, rm(X, shape, F16), rm(Q, shape, F8), rm(S, (R, kb(C)), F32),
                                      rm(QT, (C, R), F8), rm(ST, (C, kb(R)), F32)), 0)


def test_quantize_python_refuses(api):
    import torch
    with pytest.raises(ValueError):
        api.quantize(torch.zeros(128))
    with pytest.raises(ValueError):
        api.quantize(torch.zeros(4, 128), direct=False)
    with pytest.raises(ValueError):
        api.quantize(torch.zeros(4, 128), out=(1, 2, 3, 4))
    with pytest.raises(TypeError):
        api.quantize(torch.zeros(4, 128, dtype=torch.float64))


# ------------------------------------------------------------ orthogonalize

def ortho_args(api, x, d, steps=5, coefficients=None, ws=WS, ws_bytes=1 << 40):
    a = api.sl_orthogonalize_args()
    a.x, a.d, a.steps = api.desc(*x), api.desc(*d), steps
    if coefficients is not None:
        a.keep = (ctypes.c_float * len(coefficients))(*coefficients)
        a.coefficients = ctypes.cast(a.keep, ctypes.POINTER(ctypes.c_float))
    a.workspace, a.workspace_bytes = ws, ws_bytes
    return a


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,what", [
    (dict(x=rm(X, (96, 128), F8)), "SL_ERR_DTYPE"),
    (dict(d=rm(D, (96, 128), F32)), "SL_ERR_DTYPE"),
    (dict(steps=0), "SL_ERR_ARG"),
    (dict(steps=65), "SL_ERR_ARG"),
    (dict(steps=1, coefficients=(1.0, NAN, 0.0)), "SL_ERR_ARG"),
    (dict(steps=1, coefficients=(INF, 0.0, 0.0)), "SL_ERR_ARG"),
    (dict(steps=1, coefficients=(17.0, 0.0, 0.0)), "SL_ERR_ARG"),
    (dict(d=rm(D, (128, 96), BF16)), "SL_ERR_SHAPE"),
    (dict(d=rm(D, (2, 96, 128), BF16)), "SL_ERR_SHAPE"),
    (dict(d=rm(D, (96, 128), BF16, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(d=rm(D, (96, 128), BF16, (1, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (96, 128), BF16, (-128, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(0, (96, 128), BF16)), "SL_ERR_NULL"),
    (dict(d=rm(0, (96, 128), BF16)), "SL_ERR_NULL"),
    (dict(x=rm(X + 1, (96, 128), BF16)), "SL_ERR_ALIGN"),
    (dict(d=rm(X + 2, (96, 128), BF16)), "SL_ERR_ALIAS"),                 # neither x itself nor apart from it
    (dict(d=rm(X, (96, 128), BF16), x=rm(X, (96, 128), F32)), "SL_ERR_ALIAS"),
    (dict(ws=0), "SL_ERR_NULL"),
    (dict(ws_bytes=64), "SL_ERR_SHAPE"),
    (dict(ws_bytes=-1), "SL_ERR_SHAPE"),
    (dict(ws=WS + 8), "SL_ERR_ALIGN"),
    (dict(ws=X), "SL_ERR_ALIAS"),
    (dict(ws=D), "SL_ERR_ALIAS"),
    (dict(x=rm(X, (70000, 4, 4), BF16), d=rm(D, (70000, 4, 4), BF16)), "SL_ERR_SHAPE"),
    # more bytes than a product's 32-bit offsets reach: 20 default steps amplify
    # too much for the Gram matrix, so this goes the direct way
    (dict(x=rm(X, (128, 1 << 24), BF16), d=rm(D, (128, 1 << 24), BF16), steps=20), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (129, 1 << 23), BF16), d=rm(D, (129, 1 << 23), BF16)), "SL_ERR_SHAPE"),
])
def test_orthogonalize_refuses(api, change, what):
    good = dict(x=rm(X, (96, 128), BF16), d=rm(D, (96, 128), BF16))
    refused(api, api.sl_orthogonalize, ortho_args(api, **{**good, **change}), what)


def test_orthogonalize_null_empty_and_workspace(api):
    assert api.lib().sl_orthogonalize(None, None) == -1
    assert api.lib().sl_orthogonalize_workspace_bytes(None, None) == -1
    empty = ortho_args(api, rm(0, (0, 128), BF16), rm(0, (0, 128), BF16), ws=0, ws_bytes=0)
    assert api.sl_orthogonalize_workspace_bytes(empty) == 0
    api.sl_orthogonalize(empty, 0)
    size = lambda m, n, t=BF16: api.sl_orthogonalize_workspace_bytes(ortho_args(api, rm(X, (m, n), t), rm(D, (m, n), t)))
    assert size(1000, 520) == size(520, 1000)  # a tall x is worked on transposed
    assert size(2048, 4096) > size(1024, 4096) > 0


def test_orthogonalize_python_refuses(api):
    import torch
    for c in ((1.0, 2.0), [(1.0, 2.0, 3.0)] * 4):
        with pytest.raises(ValueError):
            api.orthogonalize(torch.zeros(4, 4, dtype=torch.bfloat16), coefficients=c, steps=5)


# ------------------------------------------------- the block-scaled product

def gemm_args(api, a, b, d, sfa, sfb, c=None, block_k=128):
    D_ = lambda v: api.desc(*v) if v is not None else None
    return api.make_args(D_(a), D_(b), D_(c), D_(d), D_(sfa), D_(sfb), block_k)


GOOD_P = dict(a=rm(X, (300, 512), F8), b=rm(Q, (200, 512), F8), d=rm(D, (300, 200), BF16), sfa=rm(S, (300, 4), F32),
              sfb=rm(ST, (2, 4), F32))


@pytest.mark.parametrize("change,what", [
    (dict(b=rm(Q, (200, 512), F16)), "SL_ERR_DTYPE"),
    (dict(sfb=rm(ST, (200, 4), E8M0)), "SL_ERR_DTYPE"),
    (dict(d=rm(D, (300, 200), F8)), "SL_ERR_DTYPE"),
    (dict(c=rm(QT, (300, 200), F16)), "SL_ERR_DTYPE"),
    (dict(block_k=32), "SL_ERR_SHAPE"),
    (dict(b=rm(Q, (200, 528), F8)), "SL_ERR_SHAPE"),
    (dict(d=rm(D, (200, 300), BF16)), "SL_ERR_SHAPE"),
    (dict(c=rm(QT, (300, 100), BF16)), "SL_ERR_SHAPE"),
    (dict(sfa=rm(S, (300, 5), F32)), "SL_ERR_SHAPE"),
    (dict(sfa=rm(S, (2, 4), F32)), "SL_ERR_SHAPE"),                        # 3 blocks of rows
    (dict(sfb=rm(ST, (3, 4), F32)), "SL_ERR_SHAPE"),
    (dict(a=rm(X, (2, 300, 512), F8)), "SL_ERR_SHAPE"),                    # d has one batch
    (dict(a=rm(0, (300, 512), F8)), "SL_ERR_NULL"),
    (dict(sfa=rm(0, (300, 4), F32)), "SL_ERR_NULL"),
    (dict(d=rm(0, (300, 200), BF16)), "SL_ERR_NULL"),
    (dict(d=rm(D + 1, (300, 200), BF16)), "SL_ERR_ALIGN"),
    (dict(sfb=rm(ST + 2, (2, 4), F32)), "SL_ERR_ALIGN"),
    (dict(a=rm(X, (300, 512), F8, (1, 300))), "SL_ERR_LAYOUT"),
    (dict(a=rm(X, (300, 512), F8, (520, 1))), "SL_ERR_LAYOUT"),
    (dict(a=rm(X + 8, (300, 512), F8)), "SL_ERR_LAYOUT"),
    (dict(a=rm(X, (300, 504), F8, (512, 1)), b=rm(Q, (200, 504), F8, (512, 1))), "SL_ERR_LAYOUT"),
    (dict(d=rm(D, (300, 200), BF16, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(d=rm(X, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(d=rm(ST, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(c=rm(D + 2, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(a=rm(X, (300, 512), F8, (1 << 24, 1))), "SL_ERR_SHAPE"),         # a tile spans 2^31 bytes
])
def test_block_product_refuses(api, change, what):
    args = gemm_args(api, **{**GOOD_P, **change})
    for call in (api.sl_gemm, api.sl_gemm_no_alloc):
        refused(api, call, args, what)


def test_block_product_plans(api):
    p = api.sl_gemm_plan(gemm_args(api, **GOOD_P))
    assert p["kernel"] == api.K_BLOCK8 and p["tile_k"] == 128 and p["m"] == 300 and p["n"] == 200
    # C may be D itself, broadcast, or absent; K = 0 and empty products are planned
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_P, "c": GOOD_P["d"]}))
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_P, "c": rm(QT, (300, 200), BF16, (0, 1))}))
    api.sl_gemm_plan(gemm_args(api, rm(0, (300, 0), F8), rm(0, (200, 0), F8), GOOD_P["d"], rm(0, (300, 0), F32),
                               rm(0, (2, 0), F32)))
    api.sl_gemm(gemm_args(api, rm(X, (0, 512), F8), GOOD_P["b"], rm(D, (0, 200), BF16), rm(S, (0, 4), F32),
                          GOOD_P["sfb"]), 0)
    # the other 8-bit form is as before
    mx = gemm_args(api, GOOD_P["a"], GOOD_P["b"], rm(D, (300, 200), F16), rm(S, (300, 16), E8M0),
                   rm(ST, (200, 16), E8M0), block_k=32)
    assert api.sl_gemm_plan(mx)["kernel"] in (api.K_MX, api.K_MX_W8, api.K_MX_W4R)


# ------------------------------------------- a launch's grid: below 2^32 work items

def test_quantize_grid_limit(api):
    # 2^24 workgroups of 256 threads: 64 rows x 128 columns each, or tiles of 128 x 128
    R = 1 << 30
    refused(api, api.sl_quantize, quantize_args(api, rm(X, (R, 1), F16), rm(1 << 50, (R, 16), F8), rm(1 << 51, (R, 1), F32)),
            "SL_ERR_SHAPE")
    refused(api, api.sl_quantize, quantize_args(api, rm(X, (2, R, 1), F16), qt=rm(1 << 52, (2, 1, R), F8),
                                                st=rm(1 << 53, (2, 1, R // 128), F32)), "SL_ERR_SHAPE")
    refused(api, api.sl_quantize, quantize_args(api, rm(X, (2, R, 1), F16), rm(1 << 50, (2, R, 16), F8),
                                                rm(1 << 51, (2, R // 128, 1), F32), block_rows=128), "SL_ERR_SHAPE")


def test_orthogonalize_grid_limit(api):
    size = lambda shape, **kw: api.sl_orthogonalize_workspace_bytes(ortho_args(api, rm(X, shape, BF16), rm(D, shape, BF16), **kw))
    # up to 128 rows: 128 columns a workgroup of 256 threads
    assert size((65535, 1, 32767)) > 0 and size((1, (1 << 31) - 128)) > 0
    # 64 x 64 values a workgroup of 256 threads
    assert size((255, 200, 64 * 16383)) > 0
    for shape in ((65535, 1, 65536), (65535, 128, 32769), (1, (1 << 31) - 1), (257, 200, 64 * 16384)):
        with pytest.raises(api.SLError) as e:
            size(shape)
        assert e.value.name == "SL_ERR_SHAPE", shape


def test_product_grid_limit(api):
    def block(M, N, K=16):
        return gemm_args(api, rm(X, (M, K), F8), rm(Q, (N, K), F8), rm(D, (M, N), BF16, (N, 1)), rm(S, (M, 1), F32, (1, 1)),
                         rm(ST, (-(-N // 128), 1), F32, (1, 1)))
    # one row: 32 columns a workgroup of 512 threads; 40 rows: of 256
    ok = api.sl_gemm_plan(block(1, (1 << 28) - 32))
    assert ok["workgroups"] * ok["threads"] == (1 << 32) - 512
    ok = api.sl_gemm_plan(block(40, (1 << 29) - 32))
    assert ok["workgroups"] * ok["threads"] < 1 << 32
    for M, N in ((1, 1 << 28), (40, 1 << 29), (1 << 21, 1 << 20)):
        with pytest.raises(api.SLError) as e:
            api.sl_gemm_plan(block(M, N))
        assert e.value.name == "SL_ERR_SHAPE"
    # the other forms
    f16 = lambda M, N: api.sl_gemm_plan(gemm_args(api, rm(X, (M, 64), F16), rm(Q, (N, 64), F16), rm(D, (M, N), F16, (N, 1)),
                                                  None, None))
    ok = f16(1 << 21, 1 << 18)
    assert ok["workgroups"] * ok["threads"] < 1 << 32
    with pytest.raises(api.SLError) as e:
        f16(1 << 21, 1 << 20)
    assert e.value.name == "SL_ERR_SHAPE"


def test_orthogonalize_coefficient_limits(api):
    size = lambda *co: api.sl_orthogonalize_workspace_bytes(ortho_args(api, rm(X, (96, 128), BF16), rm(D, (96, 128), BF16),
                                                                       steps=len(co) // 3, coefficients=co))
    assert size(8.2872, -23.5959, 17.3004) > 0 and size(16.0, -64.0, 64.0) > 0
    for co in ((16.5, 0.0, 0.0), (1.0, 64.5, 0.0), (1.0, 0.0, -65.0), (1.0, 0.0, NAN)):
        with pytest.raises(api.SLError) as e:
            size(*co)
        assert e.value.name == "SL_ERR_ARG"


@pytest.mark.parametrize("M,N,out", [(1, 4096, BF16), (48, 8192, F16), (48, 8192, F32), (30, 100, BF16), (300, 200, F16),
                                     (1290, 1500, BF16), (1290, 1500, F32), (8192, 8192, BF16), (4000, 3000, F32)])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_block_product_is_described(api, M, N, out, b_rows):
    """The trace of every kernel of the block-scaled form: of the plan that
    sl_gemm_plan gives, its layouts ones that the algebra reads back."""
    K = 2064
    kb = 17
    args = gemm_args(api, rm(X, (M, K), F8), rm(Q, (N, K), F8), rm(D, (M, N), out), rm(S, (M, kb), F32, (1, M)),
                     rm(ST, (-(-N // b_rows), kb), F32), c=rm(QT, (M, N), out))
    plan = api.sl_gemm_plan(args)
    text = api.describe_plan(args)
    stages = api.describe_stages(text)
    assert text.startswith(f"# kernel {api.K_BLOCK8}:")
    assert f"{plan['workgroups']} workgroups of {plan['threads']} threads" in text
    assert f"{plan['lds_bytes']} LDS bytes" in text
    for name in ("A_instr", "A", "A_tiles", "B", "B_tiles", "A_frag", "B_frag", "SFA", "SFB", "D_instr", "acc", "D_lane0", "D", "C",
                 "D_tiles"):
        api.layout_op("parse", stages[name])
    assert ("A_lds" in stages) == (M > 16)
    size = lambda l: int(api.layout_op("size", l))
    assert size(stages["A"]) == M * K and size(stages["B"]) == N * K and size(stages["D"]) == M * N
    # m, block -> offset of the scale: one row of scales for each row of A, b_rows of B's share one
    at = lambda l, row, rows, j: int(api.layout_op("eval", l, str(row + rows * j)))
    assert at(stages["SFA"], M - 1, M, 3) == M - 1 + 3 * M
    rows_b = N if b_rows == 1 else -(-N // 128) * 128
    for n in (0, N // 2, N - 1):
        assert at(stages["SFB"], n, rows_b, 5) == n // b_rows * kb + 5
    # a lane's 32 codes, twice 16 in a row 64 apart
    assert [int(api.layout_op("eval", stages["A_instr"], str(64 * v))) // 16 for v in (0, 15, 16, 31)] == [0, 15, 64, 79]
    assert ("v_mfma_f32_16x16x32_f16" in text) == (out == F32)
    # accumulators: as many fp32 registers as the tile's part of a lane
    tile_m = plan["tile_m"] if plan["tile_m"] != 64 else (16 if M <= 16 else 32 if M <= 32 else 64)
    waves = plan["threads"] // 64 if plan["tile_m"] != 64 else 1
    assert size(stages["acc"]) == tile_m * plan["tile_n"] // 64 // waves


def test_block_product_description_refuses(api):
    for change, what in ((dict(block_k=32), "SL_ERR_SHAPE"), (dict(sfb=rm(ST, (3, 4), F32)), "SL_ERR_SHAPE"),
                         (dict(a=rm(X, (300, 512), F8, (520, 1))), "SL_ERR_LAYOUT")):
        with pytest.raises(api.SLError) as e:
            api.describe_plan(gemm_args(api, **{**GOOD_P, **change}))
        assert e.value.name == what
    empty = gemm_args(api, rm(X, (0, 512), F8), GOOD_P["b"], rm(D, (0, 200), BF16), rm(S, (0, 4), F32), GOOD_P["sfb"])
    assert "nothing is launched" in api.describe_plan(empty)
    no_k = gemm_args(api, rm(0, (300, 0), F8), rm(0, (200, 0), F8), GOOD_P["d"], rm(0, (300, 0), F32), rm(0, (2, 0), F32))
    assert api.describe_plan(no_k).startswith("# kernel 9")


def test_current_stream_without_torchs_private_call(api, monkeypatch):
    """torch's private call for a stream's handle is a short cut, not needed."""
    import torch

    class Stream:
        cuda_stream = 4711
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    assert api._stream(None).value == 103 and api._stream(7).value == 7 and not api._stream(0).value
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert api._stream(None).value == 4711


def test_host_tensors_are_refused(api):
    """Before any call: a kernel that reads host memory faults the GPU."""
    import torch
    h, q, s = torch.zeros(64, 128).half(), torch.zeros(64, 128).to(torch.float8_e4m3fn), torch.ones(64, 1)
    for call in (lambda **kw: api.gemm(h, h, **kw), lambda **kw: api.gemm(q, q, sfa=s, sfb=s, block_k=128, **kw),
                 lambda **kw: api.quantize(h, **kw), lambda **kw: api.quantize(h, transposed=True, **kw),
                 lambda **kw: api.orthogonalize(h, **kw)):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    packed = api.PackedTensor(torch.zeros(64 * 96, dtype=torch.uint8), api.SL_F6_E2M3, (64, 128), (128, 1))
    with pytest.raises(ValueError, match="GPU tensors"):
        api.gemm(packed, packed, out=h)
