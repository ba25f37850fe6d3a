"""sl_quantize_rows, the int8 form of sl_gemm, sl_gated and sl_gated_backward on
the host (no GPU): every check of their arguments runs before any HIP call, so a
refusal is seen here; what passes the checks is planned, not run."""

import ctypes

import pytest

from test_ops_abi import BF16, D, F16, F32, F8, Q, QT, S, ST, WS, X, api, gemm_args, refused, rm  # noqa: F401

I8 = 9
SILU, RELU = 1, 4
Z = [i << 36 for i in range(10, 20)]   # further addresses, 64 GiB apart


def filled(api, args, tensors):  # noqa: F811
    for name, _ in args._fields_:
        if _ is not api.sl_tensor:
            continue
        if tensors.get(name) is not None:
            setattr(args, name, api.desc(*tensors[name]))
        else:
            getattr(args, name).layout.rank = 2
    return args


# --------------------------------------------------------------- quantize_rows

def rows_args(api, **t):  # noqa: F811
    return filled(api, api.sl_quantize_rows_args(), t)


GOOD_R = dict(x=rm(X, (256, 500), F16), q=rm(Q, (256, 512), I8), s=rm(S, (256, 1), F32))


@pytest.mark.parametrize("change,what", [
    (dict(x=rm(X, (256, 500), I8)), "SL_ERR_DTYPE"),
    (dict(q=rm(Q, (256, 512), F8)), "SL_ERR_DTYPE"),
    (dict(s=rm(S, (256, 1), F16)), "SL_ERR_DTYPE"),
    (dict(x=rm(X, (500,), F16)), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (256, 500), F16, (500, -1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (256, -500), F16, (512, 1))), "SL_ERR_SHAPE"),
    (dict(q=rm(Q, (256, 496), I8)), "SL_ERR_SHAPE"),                     # fewer columns than x
    (dict(q=rm(Q, (256, 528), I8)), "SL_ERR_SHAPE"),                     # past the next multiple of 128
    (dict(q=rm(Q, (255, 512), I8)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (255, 1), F32)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (256, 4), F32)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (1, 256), F32)), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (2, 256, 500), F16)), "SL_ERR_SHAPE"),                 # q and s have one matrix
    (dict(x=rm(X, (2, 256, 500), F16), q=rm(Q, (2, 256, 512), I8)), "SL_ERR_SHAPE"),
    (dict(s=rm(S, (2, 256, 1), F32)), "SL_ERR_SHAPE"),
    (dict(x=rm(0, (256, 500), F16)), "SL_ERR_NULL"),
    (dict(q=rm(0, (256, 512), I8)), "SL_ERR_NULL"),
    (dict(s=rm(0, (256, 1), F32)), "SL_ERR_NULL"),
    (dict(x=rm(X + 1, (256, 500), F16)), "SL_ERR_ALIGN"),
    (dict(s=rm(S + 2, (256, 1), F32)), "SL_ERR_ALIGN"),
    (dict(q=rm(Q, (256, 512), I8, (1, 256))), "SL_ERR_LAYOUT"),          # columns not contiguous
    (dict(q=rm(Q, (256, 512), I8, (520, 1))), "SL_ERR_LAYOUT"),          # rows off 16 bytes
    (dict(q=rm(Q + 8, (256, 512), I8)), "SL_ERR_LAYOUT"),
    (dict(q=rm(Q, (256, 512), I8, (0, 1))), "SL_ERR_LAYOUT"),            # every row the same memory
    (dict(s=rm(S, (256, 1), F32, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(q=rm(X, (256, 512), I8)), "SL_ERR_ALIAS"),
    (dict(s=rm(X + 64, (256, 1), F32)), "SL_ERR_ALIAS"),
    (dict(s=rm(Q + 512 * 256 - 4, (256, 1), F32)), "SL_ERR_ALIAS"),
    (dict(x=rm(X, ((1 << 31) - 128, 1), F16), q=rm(Q, ((1 << 31) - 128, 16), I8), s=rm(S, ((1 << 31) - 128, 1), F32)), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (1 << 16, 1 << 16, 1), F16), q=rm(Q, (1 << 16, 1 << 16, 16), I8), s=rm(S, (1 << 16, 1 << 16, 1), F32)), "SL_ERR_SHAPE"),
])
def test_quantize_rows_refuses(api, change, what):  # noqa: F811
    refused(api, api.sl_quantize_rows, rows_args(api, **{**GOOD_R, **change}), what)


def test_quantize_rows_null_and_empty(api):  # noqa: F811
    assert api.lib().sl_quantize_rows(None, None) == -1
    # nothing to write: no memory either
    api.sl_quantize_rows(rows_args(api, x=rm(0, (0, 512), F16), q=rm(0, (0, 512), I8), s=rm(0, (0, 1), F32)), 0)
    api.sl_quantize_rows(rows_args(api, x=rm(0, (0, 4, 512), F16), q=rm(0, (0, 4, 512), I8), s=rm(0, (0, 4, 1), F32)), 0)
    # rows without columns still have scales
    refused(api, api.sl_quantize_rows, rows_args(api, x=rm(0, (4, 0), F16), q=rm(0, (4, 0), I8), s=rm(0, (4, 1), F32)), "SL_ERR_NULL")


# ------------------------------------------------------------ the int8 product

GOOD_I = dict(a=rm(X, (300, 512), I8), b=rm(Q, (200, 512), I8), d=rm(D, (300, 200), BF16),
              sfa=rm(S, (300, 1), F32), sfb=rm(ST, (200, 1), F32), block_k=0)


@pytest.mark.parametrize("change,what", [
    (dict(b=rm(Q, (200, 512), F8)), "SL_ERR_DTYPE"),
    (dict(d=rm(D, (300, 200), I8)), "SL_ERR_DTYPE"),
    (dict(c=rm(QT, (300, 200), F32)), "SL_ERR_DTYPE"),
    (dict(sfa=rm(S, (300, 1), BF16)), "SL_ERR_DTYPE"),
    (dict(sfb=rm(ST, (200, 1), 4)), "SL_ERR_DTYPE"),
    (dict(b=rm(Q, (200, 528), I8)), "SL_ERR_SHAPE"),
    (dict(d=rm(D, (200, 300), BF16)), "SL_ERR_SHAPE"),
    (dict(c=rm(QT, (300, 1), BF16)), "SL_ERR_SHAPE"),
    (dict(sfa=rm(S, (300, 4), F32)), "SL_ERR_SHAPE"),                      # the block-scaled form's
    (dict(sfb=rm(ST, (300, 1), F32)), "SL_ERR_SHAPE"),
    (dict(a=rm(X, (2, 300, 512), I8)), "SL_ERR_SHAPE"),                    # d has one batch
    (dict(sfb=rm(ST, (2, 200, 1), F32)), "SL_ERR_SHAPE"),
    (dict(a=rm(X, (300, 131072), I8), b=rm(Q, (200, 131072), I8)), "SL_ERR_SHAPE"),   # sums past 31 bits
    (dict(a=rm(0, (300, 512), I8)), "SL_ERR_NULL"),
    (dict(sfa=rm(0, (300, 1), F32)), "SL_ERR_NULL"),
    (dict(d=rm(0, (300, 200), BF16)), "SL_ERR_NULL"),
    (dict(d=rm(D + 1, (300, 200), BF16)), "SL_ERR_ALIGN"),
    (dict(sfb=rm(ST + 2, (200, 1), F32)), "SL_ERR_ALIGN"),
    (dict(a=rm(X, (300, 512), I8, (1, 300))), "SL_ERR_LAYOUT"),
    (dict(a=rm(X, (300, 512), I8, (520, 1))), "SL_ERR_LAYOUT"),
    (dict(b=rm(Q + 8, (200, 512), I8)), "SL_ERR_LAYOUT"),
    (dict(a=rm(X, (300, 504), I8, (512, 1)), b=rm(Q, (200, 504), I8, (512, 1))), "SL_ERR_LAYOUT"),
    (dict(d=rm(D, (300, 200), BF16, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(d=rm(X, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(d=rm(ST, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(c=rm(D + 2, (300, 200), BF16)), "SL_ERR_ALIAS"),
    (dict(a=rm(X, (300, 512), I8, (1 << 24, 1))), "SL_ERR_SHAPE"),         # a tile spans 2^31 bytes
    (dict(a=rm(X, (1 << 25, 1, 16), I8), b=rm(Q, (16, 16), I8), sfa=rm(S, (1, 1), F32), sfb=rm(ST, (16, 1), F32),
          d=rm(D, (1 << 25, 1, 16), BF16)), "SL_ERR_SHAPE"),               # more tiles than a grid holds
])
def test_int8_product_refuses(api, change, what):  # noqa: F811
    args = gemm_args(api, **{**GOOD_I, **change})
    for call in (api.sl_gemm, api.sl_gemm_no_alloc):
        refused(api, call, args, what)
    with pytest.raises(api.SLError) as e:
        api.describe_plan(args)
    assert e.value.name == what


def test_int8_product_plans(api):  # noqa: F811
    p = api.sl_gemm_plan(gemm_args(api, **GOOD_I))
    assert p["kernel"] == api.K_I8 and p["tile_k"] == 128 and (p["m"], p["n"], p["k"]) == (300, 200, 512)
    assert p["split_k"] == 1 and p["workspace_bytes"] == 0
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_I, "c": GOOD_I["d"]}))
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_I, "c": rm(QT, (300, 200), BF16, (0, 1))}))
    # the longest sums that are exact
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_I, "a": rm(X, (300, 131056), I8), "b": rm(Q, (200, 131056), I8)}))
    # K = 0 reads neither operand; an empty D is planned and nothing runs
    api.sl_gemm_plan(gemm_args(api, **{**GOOD_I, "a": rm(0, (300, 0), I8), "b": rm(0, (200, 0), I8)}))
    api.sl_gemm(gemm_args(api, rm(0, (0, 512), I8), GOOD_I["b"], rm(0, (0, 200), BF16), rm(0, (0, 1), F32), GOOD_I["sfb"], block_k=0), 0)


@pytest.mark.parametrize("M,N,out", [(1, 4096, BF16), (48, 8192, F16), (64, 100, F32), (300, 200, F16), (1290, 1500, BF16), (1000, 2500, F32),
                                     (8192, 8192, BF16), (4000, 1000, F32),
                                     (4000, 3000, F16), (512, 1024, BF16)])
@pytest.mark.parametrize("K", [2064, 16384])
def test_int8_product_is_described(api, M, N, out, K):  # noqa: F811
    args = gemm_args(api, rm(X, (M, K), I8), rm(Q, (N, K), I8), rm(D, (M, N), out), rm(S, (M, 1), F32), rm(ST, (N, 1), F32),
                     c=rm(QT, (M, N), out), block_k=0)
    plan = api.sl_gemm_plan(args)
    text = api.describe_plan(args)
    stages = api.describe_stages(text)
    assert text.startswith(f"# kernel {api.K_I8}:") and "v_mfma_i32_16x16x64_i8" in text
    assert f"{plan['workgroups']} workgroups of {plan['threads']} threads" in text
    assert f"{plan['lds_bytes']} LDS bytes" in text
    assert plan["lds_bytes"] <= 160 * 1024
    if plan["tile_m"] >= 128:  # a ring of five operand K-tiles, or of nine
        slots = plan["lds_bytes"] // (128 * plan["tile_m"])
        assert slots in (5, 9) and f"a ring of {slots} operand K-tiles" in text
    for name in ("A", "B", "D", "C"):
        api.layout_op("parse", stages[name])
    size = lambda l: int(api.layout_op("size", l))
    assert size(stages["A"]) == M * K and size(stages["B"]) == N * K and size(stages["D"]) == M * N
    # tiles cover the product
    tm, tn = -(-M // plan["tile_m"]), -(-N // plan["tile_n"])
    assert plan["workgroups"] == tm * tn


# -------------------------------------------------------------- the gated block

def gated_args(api, activation=SILU, ws=0, ws_bytes=0, **t):  # noqa: F811
    a = filled(api, api.sl_gated_args(), t)
    a.activation, a.workspace, a.workspace_bytes = activation, ws, ws_bytes
    return a


M, F, K = 72, 96, 64
GOOD_G = dict(x=rm(X, (M, K), BF16), w_gate=rm(Z[0], (F, K), BF16), w_up=rm(Z[1], (F, K), BF16), h=rm(D, (M, F), BF16),
              gate=rm(Z[2], (M, F), BF16), up=rm(Z[3], (M, F), BF16))
GOOD_G8 = dict(x=rm(X, (M, K), I8), w_gate=rm(Z[0], (F, K), I8), w_up=rm(Z[1], (F, K), I8), h=rm(D, (M, F), F16),
               sx=rm(S, (M, 1), F32), s_gate=rm(ST, (F, 1), F32), s_up=rm(Z[4], (F, 1), F32))


@pytest.mark.parametrize("change,what", [
    (dict(x=rm(X, (M, K), F32)), "SL_ERR_DTYPE"),
    (dict(x=rm(X, (M, K), F16)), "SL_ERR_DTYPE"),
    (dict(w_up=rm(Z[1], (F, K), F16)), "SL_ERR_DTYPE"),
    (dict(h=rm(D, (M, F), F32)), "SL_ERR_DTYPE"),
    (dict(gate=rm(Z[2], (M, F), F32)), "SL_ERR_DTYPE"),
    (dict(sx=rm(S, (M, 1), F32)), "SL_ERR_DTYPE"),                         # scales of 16-bit values
    (dict(activation=0), "SL_ERR_ARG"),
    (dict(activation=5), "SL_ERR_ARG"),
    (dict(x=rm(X, (K,), BF16)), "SL_ERR_LAYOUT"),
    (dict(w_gate=rm(Z[0], (F, K), BF16, (-64, 1))), "SL_ERR_LAYOUT"),
    (dict(w_gate=rm(Z[0], (F, K + 8), BF16)), "SL_ERR_SHAPE"),
    (dict(w_up=rm(Z[1], (F + 1, K), BF16)), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (M + 1, K), BF16)), "SL_ERR_SHAPE"),
    (dict(up=rm(Z[3], (F, M), BF16)), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (2, M, K), BF16)), "SL_ERR_SHAPE"),                      # h is one matrix
    (dict(h=rm(D, (2, M, F), BF16)), "SL_ERR_SHAPE"),                      # and so are gate and up
    (dict(h=rm(D, (2, M, F), BF16), gate=rm(Z[2], (2, M, F), BF16), up=rm(Z[3], (2, M, F), BF16), x=rm(X, (3, M, K), BF16)), "SL_ERR_SHAPE"),
    (dict(x=rm(0, (M, K), BF16)), "SL_ERR_NULL"),
    (dict(w_up=rm(0, (F, K), BF16)), "SL_ERR_NULL"),
    (dict(h=rm(0, (M, F), BF16)), "SL_ERR_NULL"),
    (dict(gate=rm(0, (M, F), BF16)), "SL_ERR_NULL"),                       # one of the two
    (dict(x=rm(X + 1, (M, K), BF16)), "SL_ERR_ALIGN"),
    (dict(h=rm(D, (M, F), BF16, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(up=rm(Z[3], (M, F), BF16, (F, 0))), "SL_ERR_LAYOUT"),
    (dict(h=rm(X, (M, F), BF16)), "SL_ERR_ALIAS"),
    (dict(gate=rm(D, (M, F), BF16)), "SL_ERR_ALIAS"),
    (dict(gate=rm(D + 2 * F, (M, F), BF16, (2 * F - 8, 1)), h=rm(D, (M, F), BF16, (2 * F - 8, 1))), "SL_ERR_ALIAS"),
    (dict(up=rm(Z[1] + 128, (M, F), BF16)), "SL_ERR_ALIAS"),
    (dict(x=rm(X, (M, 1 << 30), BF16), w_gate=rm(Z[0], (F, 1 << 30), BF16), w_up=rm(Z[1], (F, 1 << 30), BF16)), "SL_ERR_SHAPE"),
    (dict(w_gate=rm(Z[0], (F, 1 << 24), BF16, (1, F)), x=rm(X, (M, 1 << 24), BF16), w_up=rm(Z[1], (F, 1 << 24), BF16)), "SL_ERR_SHAPE"),
    # copies are needed
    (dict(x=rm(X, (M, K), BF16, (1, M))), "SL_ERR_NULL"),
    (dict(x=rm(X, (M, K), BF16, (1, M)), ws=WS, ws_bytes=M * K * 2 - 1), "SL_ERR_SHAPE"),
    (dict(x=rm(X, (M, K), BF16, (1, M)), ws=WS + 8, ws_bytes=1 << 30), "SL_ERR_ALIGN"),
    (dict(x=rm(X, (M, K), BF16, (1, M)), ws=D + 16, ws_bytes=1 << 30), "SL_ERR_ALIAS"),
    (dict(x=rm(X, (M, K), BF16, (1, M)), ws=X - (1 << 12), ws_bytes=1 << 30), "SL_ERR_ALIAS"),
])
def test_gated_refuses(api, change, what):  # noqa: F811
    refused(api, api.sl_gated, gated_args(api, **{**GOOD_G, **change}), what)


@pytest.mark.parametrize("change,what", [
    (dict(w_gate=rm(Z[0], (F, K), F16)), "SL_ERR_DTYPE"),
    (dict(h=rm(D, (M, F), I8)), "SL_ERR_DTYPE"),
    (dict(sx=rm(S, (M, 1), F16)), "SL_ERR_DTYPE"),
    (dict(s_up=None), "SL_ERR_DTYPE"),
    (dict(s_gate=rm(ST, (M, 1), F32)), "SL_ERR_SHAPE"),
    (dict(s_gate=rm(0, (F, 1), F32)), "SL_ERR_NULL"),
    (dict(s_gate=rm(ST + 2, (F, 1), F32)), "SL_ERR_ALIGN"),
    (dict(x=rm(X, (M, K), I8, (1, M))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (M, K), I8, (72, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (M, 40), I8, (64, 1)), w_gate=rm(Z[0], (F, 40), I8, (64, 1)), w_up=rm(Z[1], (F, 40), I8, (64, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (M, 131072), I8), w_gate=rm(Z[0], (F, 131072), I8), w_up=rm(Z[1], (F, 131072), I8)), "SL_ERR_SHAPE"),
    (dict(w_up=rm(Z[1], (F, K), I8, (1 << 25, 1))), "SL_ERR_SHAPE"),       # a tile spans 2^31 bytes
    (dict(h=rm(S, (M, F), F16)), "SL_ERR_ALIAS"),
])
def test_gated_int8_refuses(api, change, what):  # noqa: F811
    refused(api, api.sl_gated, gated_args(api, **{**GOOD_G8, **change}), what)


def workspace(api, call, args):  # noqa: F811
    n = ctypes.c_int64(-1)
    api._check(call(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def test_gated_plans(api):  # noqa: F811
    L = api.lib()
    assert L.sl_gated(None, None) == -1 and L.sl_gated_workspace_bytes(None, None) == -1
    need = lambda **t: workspace(api, L.sl_gated_workspace_bytes, gated_args(api, **{**GOOD_G, **t}))
    assert need() == 0 and need(gate=None, up=None) == 0
    assert workspace(api, L.sl_gated_workspace_bytes, gated_args(api, **GOOD_G8)) == 0
    # weights that are two parts of one matrix, one after the other or in turn: read as they lie
    assert need(w_gate=rm(Z[0], (F, K), BF16), w_up=rm(Z[0] + 2 * F * K, (F, K), BF16)) == 0
    assert need(w_gate=rm(Z[0], (F, K), BF16, (2 * K, 1)), w_up=rm(Z[0] + 2 * K, (F, K), BF16, (2 * K, 1))) == 0
    # results that are two parts of one matrix
    assert need(gate=rm(Z[2], (M, F), BF16, (2 * F, 1)), up=rm(Z[2] + 2 * F, (M, F), BF16, (2 * F, 1))) == 0
    assert need(gate=rm(Z[2], (M, F), BF16, (2 * F, 2)), up=rm(Z[2] + 2, (M, F), BF16, (2 * F, 2))) == 0
    # an operand that doesn't lie in rows is copied, K to a multiple of 8: 256-byte pieces
    assert need(x=rm(X, (M, K), BF16, (1, M))) == M * K * 2
    assert need(x=rm(X + 2, (M, K), BF16)) == M * K * 2
    odd = dict(x=rm(X, (M, K - 1), BF16), w_gate=rm(Z[0], (F, K - 1), BF16), w_up=rm(Z[1], (F, K - 1), BF16))
    assert need(**odd) == (M + 2 * F) * K * 2
    # a broadcast weight once, a batch's own for every matrix
    three = dict(h=rm(D, (3, M, F), BF16), gate=None, up=None, x=rm(X, (3, M, K), BF16))
    assert need(**three, w_gate=rm(Z[0], (3, F, K), BF16, (0, 1, F))) == F * K * 2
    assert need(**three, w_gate=rm(Z[0], (F, K), BF16, (1, F))) == F * K * 2
    assert need(**three, w_gate=rm(Z[0], (3, F, K), BF16, (F * K, 1, F))) == 3 * F * K * 2
    # empty: nothing is read, nothing is wanted
    for m, f in ((0, F), (M, 0)):
        e = gated_args(api, x=rm(0, (m, K), BF16), w_gate=rm(0, (f, K), BF16), w_up=rm(0, (f, K), BF16), h=rm(0, (m, f), BF16))
        assert workspace(api, L.sl_gated_workspace_bytes, e) == 0
        api.sl_gated(e, 0)


# ------------------------------------------------------------ its backward pass

def backward_args(api, activation=SILU, ws=WS, ws_bytes=1 << 33, **t):  # noqa: F811
    a = filled(api, api.sl_gated_backward_args(), t)
    a.activation, a.workspace, a.workspace_bytes = activation, ws, ws_bytes
    return a


GOOD_B = dict(dh=rm(D, (M, F), F16), x=rm(X, (M, K), F16), w_gate=rm(Z[0], (F, K), F16), w_up=rm(Z[1], (F, K), F16),
              gate=rm(Z[2], (M, F), F16), up=rm(Z[3], (M, F), F16), dx=rm(Z[4], (M, K), F16), dw_gate=rm(Z[5], (F, K), F16),
              dw_up=rm(Z[6], (F, K), F16))


@pytest.mark.parametrize("change,what", [
    (dict(dh=rm(D, (M, F), F32)), "SL_ERR_DTYPE"),
    (dict(x=rm(X, (M, K), BF16)), "SL_ERR_DTYPE"),
    (dict(up=rm(Z[3], (M, F), F32)), "SL_ERR_DTYPE"),
    (dict(dw_up=rm(Z[6], (F, K), F32)), "SL_ERR_DTYPE"),
    (dict(dx=rm(Z[4], (M, K), F32)), "SL_ERR_DTYPE"),
    (dict(activation=0), "SL_ERR_ARG"),
    (dict(activation=RELU + 1), "SL_ERR_ARG"),
    (dict(dh=rm(D, (F,), F16)), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (M, K), F16, (-K, 1))), "SL_ERR_LAYOUT"),
    (dict(x=rm(X, (M + 1, K), F16)), "SL_ERR_SHAPE"),
    (dict(w_up=rm(Z[1], (F, K + 8), F16)), "SL_ERR_SHAPE"),
    (dict(gate=rm(Z[2], (F, M), F16)), "SL_ERR_SHAPE"),
    (dict(dx=rm(Z[4], (K, M), F16)), "SL_ERR_SHAPE"),
    (dict(dw_gate=rm(Z[5], (K, F), F16)), "SL_ERR_SHAPE"),
    (dict(dw_gate=rm(Z[5], (1, F, K), F16)), "SL_ERR_SHAPE"),              # the weight is a matrix
    (dict(x=rm(X, (1, M, K), F16)), "SL_ERR_SHAPE"),
    (dict(w_gate=rm(Z[0], (1, F, K), F16)), "SL_ERR_SHAPE"),
    (dict(dh=rm(0, (M, F), F16)), "SL_ERR_NULL"),
    (dict(x=rm(0, (M, K), F16)), "SL_ERR_NULL"),
    (dict(gate=rm(0, (M, F), F16)), "SL_ERR_NULL"),
    (dict(dw_up=rm(0, (F, K), F16)), "SL_ERR_NULL"),
    (dict(dw_gate=rm(0, (F, K), F16)), "SL_ERR_NULL"),
    (dict(dx=rm(Z[4] + 1, (M, K), F16)), "SL_ERR_ALIGN"),
    (dict(dx=rm(Z[4], (M, K), F16, (0, 1))), "SL_ERR_LAYOUT"),
    (dict(dw_up=rm(Z[6], (F, K), F16, (1, 1))), "SL_ERR_LAYOUT"),
    (dict(dx=rm(X, (M, K), F16)), "SL_ERR_ALIAS"),                         # not in place
    (dict(dx=rm(D, (M, K), F16)), "SL_ERR_ALIAS"),
    (dict(dw_gate=rm(Z[0], (F, K), F16)), "SL_ERR_ALIAS"),
    (dict(dw_up=rm(Z[5], (F, K), F16)), "SL_ERR_ALIAS"),
    (dict(dw_up=rm(Z[5] + 2 * K - 2, (F, K), F16, (2 * K, 1)), dw_gate=rm(Z[5], (F, K), F16, (2 * K, 1))), "SL_ERR_ALIAS"),
    (dict(ws=0), "SL_ERR_NULL"),
    (dict(ws_bytes=1024), "SL_ERR_SHAPE"),
    (dict(ws=WS + 4), "SL_ERR_ALIGN"),
    (dict(ws=Z[4]), "SL_ERR_ALIAS"),
    (dict(ws=Z[6] - 256), "SL_ERR_ALIAS"),
    (dict(ws=X), "SL_ERR_ALIAS"),
])
def test_gated_backward_refuses(api, change, what):  # noqa: F811
    refused(api, api.sl_gated_backward, backward_args(api, **{**GOOD_B, **change}), what)


def test_gated_backward_plans(api):  # noqa: F811
    L = api.lib()
    assert L.sl_gated_backward(None, None) == -1 and L.sl_gated_backward_workspace_bytes(None, None) == -1
    need = lambda **t: workspace(api, L.sl_gated_backward_workspace_bytes, backward_args(api, **{**GOOD_B, **t}))
    both, dx, dw = need(), need(dw_gate=None, dw_up=None), need(dx=None)
    assert 0 < dx < both and 0 < dw < both and both <= dx + dw
    assert need(dx=None, dw_gate=None, dw_up=None) == 0
    api.sl_gated_backward(backward_args(api, **{**GOOD_B, "dx": None, "dw_gate": None, "dw_up": None}, ws=0, ws_bytes=0), 0)
    # the two gradients as parts of one matrix
    need(dw_gate=rm(Z[5], (F, K), F16, (2 * K, 1)), dw_up=rm(Z[5] + 2 * K, (F, K), F16, (2 * K, 1)))
    need(dw_gate=rm(Z[5], (F, K), F16), dw_up=rm(Z[5] + 2 * F * K, (F, K), F16))
    # without tokens the weights' gradients are zeros: no copies
    none = {n: rm(0, (0, s), F16) for n, s in (("dh", F), ("x", K), ("gate", F), ("up", F), ("dx", K))}
    assert need(**none) == 0
    # nothing wanted is there
    api.sl_gated_backward(backward_args(api, **{**GOOD_B, **none, "w_gate": rm(0, (0, K), F16), "w_up": rm(0, (0, K), F16),
                                                "dh": rm(0, (0, 0), F16), "gate": rm(0, (0, 0), F16), "up": rm(0, (0, 0), F16),
                                                "dw_gate": rm(0, (0, K), F16), "dw_up": rm(0, (0, K), F16)}, ws=0, ws_bytes=0), 0)


def test_large_backward_reads_the_operands_as_they_lie(api):  # noqa: F811
    """Its workspace holds dg and du alone, both together a row of 2 x F to a
    multiple of 64; weights or activations off 16 bytes are copied again."""
    m, f, k = 4096, 4088, 4096
    big = dict(dh=rm(D, (m, f), BF16), x=rm(X, (m, k), BF16), w_gate=rm(Z[0], (f, k), BF16), w_up=rm(Z[1], (f, k), BF16),
               gate=rm(Z[2], (m, f), BF16), up=rm(Z[3], (m, f), BF16), dx=rm(Z[4], (m, k), BF16), dw_gate=rm(Z[5], (f, k), BF16),
               dw_up=rm(Z[6], (f, k), BF16))
    need = lambda **t: workspace(api, api.lib().sl_gated_backward_workspace_bytes, backward_args(api, **{**big, **t}))
    fp = -(-f // 64) * 64
    assert need() == need(dx=None) == need(dw_gate=None, dw_up=None) == m * 2 * fp * 2
    assert need(w_up=rm(Z[1] + 2, (f, k), BF16)) == m * 2 * fp * 2 + k * 2 * fp * 2
    assert need(w_up=rm(Z[1], (f, k), BF16, (k + 8, 1))) == m * 2 * fp * 2 + k * 2 * fp * 2      # one stride for both
    assert need(x=rm(X, (m, k), BF16, (1, m))) == m * 2 * fp * 2 + 2 * fp * m * 2 + k * m * 2


# --------------------------------------------------------------------- Python

def test_python_refuses(api):  # noqa: F811
    import torch
    h, w, q, s = torch.zeros(64, 128).half(), torch.zeros(32, 128).half(), torch.zeros(64, 128, dtype=torch.int8), torch.ones(64, 1)
    kept = torch.zeros(64, 32).half()
    # host tensors: a kernel that reads them faults the GPU
    for call in (lambda **kw: api.quantize_rows(h, **kw), lambda **kw: api.gemm(q, q, sfa=s, sfb=s, **kw),
                 lambda **kw: api.gated(h, w, w, **kw), lambda **kw: api.gated(h, w, w, keep=True, **kw),
                 lambda **kw: api.gated(q, q, q, sx=s, s_gate=s, s_up=s, **kw),
                 lambda **kw: api.gated_backward(kept, h, w, w, kept, kept, **kw)):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    with pytest.raises(ValueError, match="matrix"):
        api.quantize_rows(h[0])
    with pytest.raises(ValueError, match="2 are written"):
        api.quantize_rows(h, out=(q,))
    with pytest.raises(ValueError, match="activation"):
        api.gated(h, w, w, activation="swish")
    with pytest.raises(ValueError, match="activation"):
        api.gated_backward(kept, h, w, w, kept, kept, activation=None)
    with pytest.raises(ValueError, match="3 are written"):
        api.gated(h, w, w, keep=True, out=(kept, kept))
    with pytest.raises(ValueError, match="matri"):
        api.gated(h[0], w, w)
    with pytest.raises(ValueError, match="nothing to compute"):
        api.gated_backward(kept, h, w, w, kept, kept, need_dx=False, need_dw=False)
    for out in ((h, w), (None, w, w), (h, None, w), (h, w, None)):
        with pytest.raises(ValueError, match="out holds"):
            api.gated_backward(kept, h, w, w, kept, kept, out=out)
    with pytest.raises(TypeError):
        api.quantize_rows(torch.zeros(4, 128, dtype=torch.float64))


def test_operands_of_another_device_are_refused(api, monkeypatch):  # noqa: F811
    """The call runs on the current device's stream: an operand of another one's memory
    would fault the GPU."""
    import torch

    class Operand:
        is_cuda = True

        def __init__(self, index):
            self.index, self.device = index, f"cuda:{index}"

        def get_device(self):
            return self.index
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    assert api._one_device(Operand(1), None, Operand(1)) == 1
    for operands in ((Operand(0),), (Operand(1), Operand(0)), (None, Operand(2), Operand(1))):
        with pytest.raises(ValueError, match="the current device is cuda:1"):
            api._one_device(*operands)
    monkeypatch.delattr(torch._C, "_cuda_getDevice")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert api._one_device(Operand(3)) == 3
    # descriptors alone: nothing to check
    assert api._one_device(None, api.sl_tensor()) is None


def sized(m, f, k, batch=(), pitch=None, off=0, **wanted):
    """A backward call of that size (sequences ``pitch`` rows apart), ``off`` bytes
    behind a boundary of 16 where the weights and x start."""
    wide = lambda at, rows, cols: rm(at, (*batch, rows, cols), BF16, *([((pitch or rows) * cols, cols, 1)] if batch else []))
    apart = lambda i: i << 42  # 4 TiB
    t = dict(dh=wide(apart(1), m, f), x=wide(apart(2) + off, m, k), w_gate=rm(apart(3) + off, (f, k), BF16), w_up=rm(apart(4) + off, (f, k), BF16),
             gate=wide(apart(5), m, f), up=wide(apart(6), m, f), dx=wide(apart(7), m, k), dw_gate=rm(apart(8), (f, k), BF16),
             dw_up=rm(apart(9), (f, k), BF16))
    return {**t, **wanted}


NO_DX, NO_DW = dict(dx=None), dict(dw_gate=None, dw_up=None)


@pytest.mark.parametrize("call,accepted", [
    # many tokens: the transposes' 64 rows span 2^29 bytes
    (sized(1 << 22, 64, 64), True),
    (sized(1 << 22, 64, 64, off=2), True),
    (sized(1 << 24, 64, 64, off=2), False),
    (sized((1 << 24) - 64, 64, 64, off=2), True),
    # ... 256 of them 2^31; read as they lie nothing of the kind
    (sized((1 << 22) - 64, 256, 256), True),
    (sized((1 << 22) - 63, 256, 256), False),
    (sized(1 << 22, 256, 256), False),
    (sized(1 << 22, 256, 256, **NO_DW), True),
    (sized(1 << 22, 64, 256), False),   # (x itself spans 2^31)
    (sized(1 << 22, 64, 256, x=rm(2 << 42, (1 << 22, 256), BF16, (0, 1))), True),
    # a wide block: rows of dg and du
    (sized(64, 1 << 21, 64), True),
    (sized(255, 1 << 21, 64), True),
    (sized(256, (1 << 21) - 64, 64), True),
    (sized(256, (1 << 21) - 63, 64), False),
    (sized(256, 1 << 21, 64, **NO_DX), True),
    # ... and the weights' transposes
    (sized(1, 1 << 21, 256), True),
    (sized(1, 1 << 21, 256, off=2), False),
    (sized(1, (1 << 21) - 64, 256, off=2), True),
    (sized(1, 1 << 21, 255, off=2), True),
    (sized(1, 1 << 28, 8, **NO_DW), False),
    (sized(1, (1 << 29) - 1, 1), False),
    # sequences of two tokens that do not follow each other, 64 each; that do
    (sized(2, 64, 64, (1 << 16,), 3), True),
    (sized(2, 256, 64, (1 << 16,), 3), False),
    (sized(2, 256, 64, ((1 << 16) - 1,), 3), True),
    (sized(2, 256, 64, (1 << 16,)), True),
])
def test_gated_backward_sizes(api, call, accepted):  # noqa: F811
    """256 rows of what a product reads, or all of fewer, span less than 2^31 bytes."""
    L, args = api.lib(), backward_args(api, **call)
    if accepted:
        assert workspace(api, L.sl_gated_backward_workspace_bytes, args) > 0
    else:
        n = ctypes.c_int64(0)
        assert api.STATUS[L.sl_gated_backward_workspace_bytes(ctypes.byref(args), ctypes.byref(n))] == "SL_ERR_SHAPE"


@pytest.mark.parametrize("m,f,k,pitch,ws,dtype", [
    (300, 8, (1 << 22) - 8, None, 0, BF16),
    (300, 8, (1 << 22) - 7, None, None, BF16),                 # rows of 2^22 values, copied
    (300, 8, 1 << 22, None, None, BF16),
    (8, 256, 1 << 22, None, None, BF16),
    (255, 255, 1 << 22, None, 0, BF16),
    (1, 1, (1 << 30) - 8, None, 0, BF16),
    (1, 1, (1 << 30) - 1, None, None, BF16),
    (1, 1, 1 << 30, None, None, BF16),
    (300, 8, 64, 1 << 23, 300 * 64 * 2, BF16),                 # rows 2^24 bytes apart: copied
    (300, 8, 64, 1 << 23, 0, I8),                              # ... 2^23
    (300, 8, 64, 1 << 24, None, I8),                           # int8 codes are not
    (100, 8, 64, 1 << 24, 0, I8),
])
def test_gated_sizes(api, m, f, k, pitch, ws, dtype):  # noqa: F811
    """256 rows of what is read, or all of fewer, span less than 2^31 bytes."""
    apart = lambda i: i << 42
    t = dict(x=rm(apart(1), (m, k), dtype, (pitch or k, 1)), w_gate=rm(apart(2), (f, k), dtype), w_up=rm(apart(3), (f, k), dtype),
             h=rm(apart(4), (m, f), BF16))
    if dtype == I8:
        t.update(sx=rm(apart(5), (m, 1), F32), s_gate=rm(apart(6), (f, 1), F32), s_up=rm(apart(7), (f, 1), F32))
    args = gated_args(api, **t)
    if ws is None:
        n = ctypes.c_int64(0)
        assert api.STATUS[api.lib().sl_gated_workspace_bytes(ctypes.byref(args), ctypes.byref(n))] == "SL_ERR_SHAPE"
    else:
        assert workspace(api, api.lib().sl_gated_workspace_bytes, args) == ws


def test_packed_operands_are_refused_with_a_reason(api, monkeypatch):  # noqa: F811
    """Packed 6-bit data beside other operands: the library's
    refusal of its type, and host memory before that."""
    import torch

    class OnGpu(torch.Tensor):   # a host tensor that says it is on device 1
        is_cuda = True

        def get_device(self):
            return 1
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    gpu = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    q, s, d = gpu(64, 128, dtype=torch.int8), gpu(64, 1, dtype=torch.float32), gpu(64, 64, dtype=torch.bfloat16)
    h, w = gpu(64, 128, dtype=torch.float16), gpu(32, 128, dtype=torch.float16)
    packed = lambda make: api.PackedTensor(make(64 * 96, dtype=torch.uint8), api.SL_F6_E2M3, (64, 128), (128, 1))
    here, host = packed(gpu), packed(torch.zeros)
    with pytest.raises(ValueError, match="GPU tensors"):
        api._one_device(host)
    assert api._one_device(here, q) == 1
    for call in (lambda: api.gemm(q, here, out=d, sfa=s, sfb=s, stream=0), lambda: api.gemm(q, q, here, out=d, sfa=s, sfb=s, stream=0),
                 lambda: api.gemm(q, q, out=d, sfa=here, sfb=s, stream=0), lambda: api.gated(h, here, w, out=d, stream=0)):
        with pytest.raises(api.SLError) as e:
            call()
        assert e.value.name == "SL_ERR_DTYPE"


def test_a_workspace_is_one_buffer(api, monkeypatch):  # noqa: F811
    """A view with gaps holds other data between its bytes, an expanded tensor has
    fewer than its elements say: a call would write memory that is not its own."""
    import torch
    monkeypatch.setattr(api, "_one_device", lambda *operands: 0)
    monkeypatch.setattr(api, "_check_devices", lambda *operands: None)
    rows = lambda *shape: torch.zeros(*shape, dtype=torch.float16)
    kept, x, w, m = rows(64, 32), rows(64, 128), rows(32, 128), rows(64, 64)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12, 2, dtype=torch.float32)[:, 0],
               torch.zeros(64, 256, dtype=torch.uint8)[:, :128]):
        for call in (lambda **kw: api.gated(x[:, 1:8], w[:, 1:8], w[:, 1:8], stream=0, out=rows(64, 32), **kw),
                     lambda **kw: api.gated_backward(kept, x, w, w, kept, kept, stream=0, out=(rows(64, 128), rows(32, 128), rows(32, 128)), **kw),
                     lambda **kw: api.orthogonalize(m, out=rows(64, 64), stream=0, **kw),
                     lambda **kw: api.gemm(x, w, out=rows(64, 32), stream=0, **kw)):
            with pytest.raises(ValueError, match="contiguous"):
                call(workspace=ws)
    at = torch.zeros(8, 512, dtype=torch.uint8)[2:6]
    args = api.sl_gated_args()
    api.set_workspace(args, at)
    assert (args.workspace, args.workspace_bytes) == (at.data_ptr(), 2048)
    api.set_workspace(args, None)
    assert (args.workspace, args.workspace_bytes) == (None, 0)


@pytest.mark.parametrize("batch,m,n,k,tile", [
    # many matrices of few K-tiles: 128 x 128 on either side of 16 and of 64 rows
    (16, 16, 8192, 128, (128, 128)), (16, 17, 8192, 128, (128, 128)), (16, 32, 8192, 128, (128, 128)), (16, 64, 8192, 128, (128, 128)),
    (16, 65, 8192, 128, (128, 128)), (16, 16, 8192, 1024, (128, 128)), (16, 17, 8192, 1024, (128, 128)), (16, 64, 8192, 1024, (128, 128)),
    (64, 32, 8192, 512, (128, 128)), (1, 16, 131072, 1024, (128, 128)), (1, 17, 131072, 1024, (128, 128)),
    # one pass over B bounds the call
    (16, 16, 8192, 4096, (16, 32)), (16, 17, 8192, 4096, (32, 64)), (16, 64, 8192, 8192, (64, 64)), (1, 48, 8192, 4096, (64, 32)),
    (1, 1, 4096, 8192, (16, 16)),
    # one round of workgroups, or little more
    (1, 17, 1024, 2048, (32, 32)), (1, 24, 9440, 1664, (32, 32)), (2, 24, 7488, 2432, (32, 32)),
])
def test_few_rows_take_the_tile_that_is_less(api, batch, m, n, k, tile):  # noqa: F811
    r3 = lambda at, dt, *s: rm(at, (batch, *s) if batch > 1 else s, dt)
    p = api.sl_gemm_plan(gemm_args(api, a=r3(Z[0], I8, m, k), b=r3(Z[1], I8, n, k), d=r3(Z[2], BF16, m, n), sfa=r3(Z[3], F32, m, 1),
                                   sfb=r3(Z[4], F32, n, 1), block_k=0))
    assert (p["tile_m"], p["tile_n"]) == tile
