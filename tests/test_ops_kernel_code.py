"""The orthogonalisation's kernels that issue their MFMAs as inline assembly on
accumulators in AGPRs (256 x 256 and 128 x 128 tiles), under the checks that
test_kernel_code.py makes of the GEMM's ring kernels."""

import pytest

import test_kernel_code as K
from test_kernel_code import code_objects  # noqa: F401

# symbol, MFMAs of one K-loop iteration, MFMAs after the loop
NAMES = {}
for mode, op, loop in ((0, 1, 128), (0, 2, 128), (1, 1, 192), (1, 2, 192), (2, 1, 128)):
    NAMES[f"ortho_ring_{mode}{op}"] = (f"_ZN2sl12_GLOBAL__N_117ortho_ring_kernelILi{mode}ELi{op}EEEvNS0_9OrthoGemmE", loop, 32)
    NAMES[f"ortho_128_{mode}{op}"] = (f"_ZN2sl12_GLOBAL__N_117ortho_gemm_kernelILi128ELi128ELi1ELi{mode}ELi{op}EEEvNS0_9OrthoGemmE",
                                      {0: 64, 1: 96, 2: 64}[mode], 0)
K.KERNELS.update(NAMES)


@pytest.mark.parametrize("name", sorted(NAMES))
def test_ortho_kernel_accumulator_discipline(code_objects, name):  # noqa: F811
    K.test_ring_kernel_accumulator_discipline(code_objects, name)


# ---------------------------------------------------------------------------
# The block-scaled product's kernels wait for a K-tile's copies into LDS by
# counting what was issued after them.
# ---------------------------------------------------------------------------

# name: (symbol, K-tiles of one pass of the loop, copies of a K-tile, K-tiles in flight at a wait)
COUNTED = {}
for ot in (0, 1, 2):
    for sb in (0, 1):
        for stages in (2, 4):
            COUNTED[f"tiles_{stages}_{sb}{ot}"] = (
                f"_ZN2sl12_GLOBAL__N_117gemm_block_kernelILi128ELi128ELi2ELi2ELi{stages}ELi{sb}ELi{ot}EEEvNS_15BlockGemmParamsE",
                stages, 8, stages - 2)
        for fm in (2, 4):
            for fn in (1, 2):
                stages = 3 if fm == 4 else 4
                COUNTED[f"stream_{fm}{fn}_{sb}{ot}"] = (
                    f"_ZN2sl12_GLOBAL__N_124gemm_block_stream_kernelILi{fm}ELi{fn}ELi{sb}ELi{ot}EEEvNS_15BlockGemmParamsE",
                    stages, 2 * (fm + fn), stages - 1)


@pytest.mark.parametrize("name", sorted(COUNTED))
def test_counted_waits(code_objects, name):  # noqa: F811
    """The K-loop as compiled, prologue and three passes in order: at the j-th
    wait of the loop every copy of K-tile j has landed, whatever order the
    compiler gave the copies' and the scales' loads; and the wait leaves no
    more operations in flight than the copies of the later K-tiles, so that
    it does not depend on that order."""
    import re
    symbol, stages, copies, ahead = COUNTED[name]
    text, succ = K.disassemble_cfg(code_objects, symbol)
    mfma = [k for k, l in enumerate(text) if l.startswith("v_mfma")]
    back = [(k, j) for k, ss in enumerate(succ) for j in ss if j < k and any(j <= m <= k for m in mfma)]
    head, end = min(j for _, j in back), max(k for k, _ in back)
    issued, copy_at, tile, counts, left = 0, [], 0, [], None
    for k in list(range(head)) + 3 * list(range(head, end + 1)):
        op = text[k].split()[0]
        if op.startswith(("buffer_load", "global_load")):
            if text[k].rstrip().endswith("lds"):
                copy_at.append(issued)
            issued, left = issued + 1, None
        wait = re.search(r"vmcnt\((\d+)\)", text[k]) if op == "s_waitcnt" else None
        if wait is not None:
            left = min(int(wait.group(1)), issued if left is None else left)
        # a K-tile is read after the barrier, or (no barrier) once its own wave has waited behind the request
        if k >= head and (op == "s_barrier" if name.startswith("tiles") else wait is not None and len(copy_at) >= (stages + tile) * copies):
            assert left is not None, f"K-tile {tile}: no wait"
            counts.append(left)
            assert len(copy_at) >= (tile + 1) * copies and copy_at[(tile + 1) * copies - 1] < issued - left, \
                f"K-tile {tile}: {left} in flight at its wait"
            tile += 1
    assert tile == 3 * stages and len(copy_at) == (stages - 1 + 3 * stages) * copies
    assert max(counts) <= ahead * copies, counts


# an X between two cycles, from x's one plane: the result a pair, both ways round
AGAIN = {
    "ortho_ring_22": ("_ZN2sl12_GLOBAL__N_117ortho_ring_kernelILi2ELi2EEEvNS0_9OrthoGemmE", 128, 32),
    "ortho_128_22": ("_ZN2sl12_GLOBAL__N_117ortho_gemm_kernelILi128ELi128ELi1ELi2ELi2EEEvNS0_9OrthoGemmE", 64, 0),
}
K.KERNELS.update(AGAIN)


@pytest.mark.parametrize("name", sorted(AGAIN))
def test_kept_iterate_accumulator_discipline(code_objects, name):  # noqa: F811
    K.test_ring_kernel_accumulator_discipline(code_objects, name)
