"""Which kernels around a block keep values in scratch memory, and how much: the
kernels that should have none have none, and the others no more than when their
figures were taken (CPU only: compiles the sources to AMD assembly)."""
import re

import pytest

from test_codegen import _asm, pytestmark  # noqa: F401

# bytes a lane, by what the kernel's name holds; everything else: 0
MOST = {
    "norm.hip": [
        # the gradient of fp32 rows of 4097 to 8192: sixteen values a thread of each array
        (r"norm_bwd_kernelINS0_7NormCfgIfLi512ELi4E", 256),
        # of bf16 rows of 4097 to 8192 with more than one pick
        (r"norm_bwd_kernelINS0_7NormCfgItLi512ELi2ELb1EEELi2E", 16),
    ],
    "ortho.hip": [
        (r"ortho_small_kernelILi2ELi2E", 16),                      # 64 x 512: three registers
        (r"ortho_product_kernel.*ELi256ELi256E", 32),              # two to seven
    ],
    "grouped.hip": [
        (r"grouped_few_kernel", 32),                               # the zeros of what is out of range
    ],
    "group_rows.hip": [],
}


@pytest.mark.parametrize("src", list(MOST))
def test_scratch(src, tmp_path):
    sizes = dict(re.findall(r"\.amdhsa_kernel (\S+)\n(?:.*\n)*?\s*\.amdhsa_private_segment_fixed_size (\d+)",
                            _asm(src, tmp_path)))
    assert sizes
    for kernel, size in sizes.items():
        most = next((n for pattern, n in MOST[src] if re.search(pattern, kernel)), 0)
        assert int(size) <= most, (kernel, size)
