"""The compiled kernels of the int8 product and of the gated block and its
backward pass, under the checks that test_kernel_code.py makes of the GEMM's
ring kernels (MFMAs issued as inline assembly on accumulators in AGPRs,
barriers that the LDS reads before them have ended at) and test_ops_kernel_code.py
of kernels whose waves each wait for their own copies by counting."""

import pytest

import test_kernel_code as K
import test_ops_kernel_code as O
from test_kernel_code import code_objects  # noqa: F401

RING = "_ZN2sl12_GLOBAL__N_117dense_ring_kernelILi{ek}ELb{gated}ELi{fm}ELi{fn}ELi{ahead}ENS0_{epi}ENS_{params}EEEvT5_"
EPILOGUE = {"product": "9ScaledSum", "gated": "4GateILi{ek}EE", "backward": "8GradientILi{ek}EE"}
TYPES = {0: "fp16", 1: "bf16", 2: "int8"}

# symbol, MFMAs of one K-loop iteration, MFMAs after the loop
NAMES = {}
for what, eks, params in (("product", (2,), "11DenseParams"), ("gated", (0, 1, 2), "11DenseParams"),
                          ("backward", (0, 1), "11DenseParams"), ("backward", (0, 1), "9DensePair")):
    for ek in eks:
        for fm, fn, ahead, loop, after in ((8, 8, 0, 128, 32), (8, 6, 0, 96, 24), (8, 4, 0, 64, 16), (4, 4, 0, 32, 8), (4, 4, 2, 32, 8)):
            if fn == 6 and (what == "gated" or params == "9DensePair"):
                continue
            name = f"{what}{'_pair' if params == '9DensePair' else ''}_{TYPES[ek]}_{fm}{fn}{ahead}"
            NAMES[name] = (RING.format(ek=ek, gated=int(what == "gated"), fm=fm, fn=fn, ahead=ahead, epi=EPILOGUE[what].format(ek=ek),
                                       params=params), loop, after)
NAMES.update({f"across_{TYPES[ek]}_{a}": (f"_ZN2sl12_GLOBAL__N_116grad_ring_kernelILi{ek}ELb{a}EEEvNS_10GradParamsE", 128, 64)
              for ek in (0, 1) for a in (0, 1)})
NAMES.update({f"across_tile_{TYPES[ek]}_{a}": (f"_ZN2sl12_GLOBAL__N_116grad_tile_kernelILi{ek}ELb{a}EEEvNS_10GradParamsE", 32, 16)
              for ek in (0, 1) for a in (0, 1)})
K.KERNELS.update(NAMES)


@pytest.mark.parametrize("name", sorted(NAMES))
def test_accumulator_discipline(code_objects, name):  # noqa: F811
    K.test_ring_kernel_accumulator_discipline(code_objects, name)


@pytest.mark.parametrize("name", sorted(NAMES))
def test_barriers_follow_lds_waits(code_objects, name):  # noqa: F811
    K.test_ring_kernel_barriers_follow_lds_waits(code_objects, name)


# waves that stream K-tiles of their own: (symbol, stages, copies of a K-tile, K-tiles in flight at a wait)
STREAM = "_ZN2sl12_GLOBAL__N_119dense_stream_kernelILi{ek}ELb{gated}ELi{fm}ELi{fn}ELi{stages}ENS0_{epi}ENS_{params}EEEvT5_"
COUNTED = {}
for what, eks, params in (("product", (2,), "11DenseParams"), ("gated", (0, 1, 2), "11DenseParams"),
                          ("backward", (0, 1), "11DenseParams"), ("backward", (0, 1), "9DensePair")):
    for ek in eks:
        for fm, fn, stages in ((2, 2, 4), (2, 4, 3), (4, 2, 3), (4, 4, 2)):
            if params == "9DensePair" and (fm, fn) == (2, 4):
                continue
            COUNTED[f"{what}{'_pair' if params == '9DensePair' else ''}_stream_{TYPES[ek]}_{fm}{fn}"] = (
                STREAM.format(ek=ek, gated=int(what == "gated"), fm=fm, fn=fn, stages=stages,
                              epi=EPILOGUE[what].format(ek=ek), params=params), stages, 2 * (fm + fn), stages - 1)
O.COUNTED.update(COUNTED)


@pytest.mark.parametrize("name", sorted(COUNTED))
def test_counted_waits(code_objects, name):  # noqa: F811
    O.test_counted_waits(code_objects, name)


# both products in one launch: the two bodies of the kernels above in one
PAIRS = {f"across_pair_{TYPES[ek]}": (f"_ZN2sl12_GLOBAL__N_116grad_pair_kernelILi{ek}EEEvNS_8GradPairE", 64, 32) for ek in (0, 1)}
K.KERNELS.update(PAIRS)


@pytest.mark.parametrize("name", sorted(PAIRS))
def test_pair_of_products(code_objects, name):  # noqa: F811
    symbol, in_loops, after = PAIRS[name]
    L = K.disassemble(code_objects, symbol)
    ops = [l.replace(",", " ").split() for l in L]
    mf = [k for k, o in enumerate(ops) if o[0].startswith("v_mfma")]
    assert len(mf) == in_loops + after
    assert not [l for l in L if l.startswith("scratch_")], "scratch traffic"
    assert all(ops[k][1] == ops[k][4] for k in mf), "not accumulating in place"
    # runs of MFMAs (a loop's two statements, the products after it) hold no accumulator moves
    for a, b in zip(mf, mf[1:]):
        if b - a < 8:
            assert not [L[k] for k in range(a, b) if ops[k][0].startswith("v_accvgpr")], L[a]
    K.test_ring_kernel_barriers_follow_lds_waits(code_objects, name)


@pytest.mark.parametrize("ek", [0, 1])
@pytest.mark.parametrize("fm", [1, 2, 4])
def test_few_rows_kernel_stays_in_registers(code_objects, ek, fm):  # noqa: F811
    L = K.disassemble(code_objects, f"_ZN2sl12_GLOBAL__N_115grad_few_kernelILi{ek}ELi{fm}EEEvNS_10GradParamsE")
    assert not [l for l in L if l.startswith("scratch_")], "scratch traffic"
    assert [l for l in L if l.startswith("v_mfma")]
