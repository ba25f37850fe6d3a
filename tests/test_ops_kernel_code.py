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
