"""Which kernels around a block keep values in scratch memory, and how much: the
kernels that should have none have none, and the others no more than when their
figures were taken (CPU only: from the built library's kernel descriptions)."""
import re
import struct

import msgpack

from butterfly_rotated_ternary_amd import bmoe
from butterfly_rotated_ternary_amd import build as B

# bytes a lane, by what the kernel's name holds; everything else: 0
MOST = [
    # the gradient of fp32 rows of 4097 to 8192: sixteen values a thread of each array
    (r"norm_bwd_kernelINS0_7NormCfgIfLi512ELi4E", 256),
    # of bf16 rows of 4097 to 8192 with more than one pick
    (r"norm_bwd_kernelINS0_7NormCfgItLi512ELi2ELb1EEELi2E", 16),
    (r"ortho_small_kernelILi2ELi2E", 16),                      # 64 x 512: three registers
    (r"ortho_product_kernel.*ELi256ELi256E", 32),              # two to seven
    (r"grouped_few_kernel", 32),                               # the zeros of what is out of range
]
NAMES = r"norm_kernel|norm_bwd_kernel|norm_weights|ortho_|grouped_|group_count|group_scatter"


def kernels():
    """Name -> bytes of scratch memory a lane, from the AMDGPU metadata notes (type 32)
    of the code objects within the library."""
    with open(B.LIB, "rb") as f:
        data = f.read()
    out = {}
    for m in re.finditer(rb"AMDGPU\0\0", data):
        namesz, descsz, kind = struct.unpack("<III", data[m.start() - 12:m.start()])
        if namesz == 7 and kind == 32:
            meta = msgpack.unpackb(data[m.end():m.end() + descsz], strict_map_key=False)
            for k in meta["amdhsa.kernels"]:
                out[k[".name"]] = k[".private_segment_fixed_size"]
    return out


def test_scratch():
    bmoe.lib()  # (built if it is not)
    found = {k: v for k, v in kernels().items() if re.search(NAMES, k)}
    assert len(found) > 100
    for kernel, size in found.items():
        most = next((n for pattern, n in MOST if re.search(pattern, kernel)), 0)
        assert size <= most, (kernel, size)
