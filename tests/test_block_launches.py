"""Launches of the dense experts, the norms around a block and the orthogonalised
updates, recorded on the CPU (none is made): calls with the largest counts that
memory can hold have grids that HIP takes, and workspace sizes do not wrap."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from butterfly_rotated_ternary_amd import bmoe
from launches import ROOT, STUB, Launch

BF, F32 = bmoe.BMOE_BF16, bmoe.BMOE_F32
LOTS = 1 << 62
TOP = 2 ** 31 - 1

pytestmark = pytest.mark.skipif(not shutil.which("g++"), reason="g++ not available")

CHILD = r"""
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
stub.seen_count.restype = ctypes.c_size_t
stub.seen_data.restype = ctypes.POINTER(ctypes.c_ulonglong)
from butterfly_rotated_ternary_amd import bmoe
SPECS = {"norm": bmoe.NormSpec, "ortho": bmoe.OrthoSpec}
out = []
for name, args in json.load(sys.stdin):
    args = [ctypes.byref(SPECS[a]()) if isinstance(a, str) else
            ctypes.byref(bmoe.OrthoUpdate(*a)) if isinstance(a, list) else a for a in args]
    stub.seen_clear()
    status = getattr(bmoe.lib(), name)(*args)
    d = stub.seen_data()
    out.append([status, [[d[8 * i + j] for j in range(8)] for i in range(stub.seen_count())]])
print(json.dumps(out))
"""


def at(i):
    """Addresses 2^42 apart, beyond any array here."""
    return (i + 1) << 42


def record(calls, tmp_path):
    src, lib = os.path.join(tmp_path, "stub.cpp"), os.path.join(tmp_path, "stub.so")
    with open(src, "w") as f:
        f.write(STUB)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", src, "-o", lib], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), text=True,
                       capture_output=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return [(s, [Launch(v) for v in ls]) for s, ls in json.loads(r.stdout.splitlines()[-1])]


def group(T, N, k):
    return "bmoe_group_rows", [T, N, k, at(0), at(1), at(2), at(3), at(4), LOTS, None]


def product(dt, M, K, O, G, perm=True):
    return "bmoe_grouped_product", [dt, M, K, O, G, at(0), M, at(1) if perm else None, 1, at(2),
                                    at(3), at(4), None]


def product_bwd(dt, M, K, O, G):
    return "bmoe_grouped_product_backward", [dt, M, K, O, G, at(0), M, at(1), 1, at(2), at(3),
                                             at(4), at(5), at(6), at(7), LOTS, None]


def norm(dt, T, d, k):
    return "bmoe_residual_norm", [dt, T, d, k, "norm", at(0), min(T * k, TOP), at(1), at(2), at(3),
                                  at(4), at(5), at(6), at(7), None]


def norm_bwd(dt, T, d, k):
    return "bmoe_residual_norm_backward", [dt, T, d, k, "norm", *[at(0), min(T * k, TOP)],
                                           *[at(i) for i in range(1, 13)], at(13), LOTS, None]


def ortho(dt, B, rows, cols):
    return "bmoe_orthogonalize", [dt, B, rows, cols, "ortho", at(0), at(1), at(2), LOTS, None]


def step(B, rows, cols):
    return "bmoe_orthogonal_step", [F32, BF, B, rows, cols, "ortho", [0.1, 0.9, 1, 0.0, 1.0], at(0),
                                    at(1), at(2), at(3), LOTS, None]


# (call, workgroups that the first launches need at least)
CASES = [
    (group(TOP, 8, 1), [1, 1]),
    (group((1 << 28) - 1, 2000, 8), [256, 256]),
    (product(BF, TOP, 8, 8, 1), [TOP // 128]),
    (product(BF, 1 << 20, 64, 65536, 64), [(1 << 12) * 256]),
    (product(F32, TOP, 1, 1, 4096), [TOP // 128]),
    (product(BF, TOP, 3, 5, 7, False), [TOP // 128]),
    (product_bwd(BF, TOP, 8, 8, 1), [TOP // 128, 1]),
    (product_bwd(BF, 100000, 4096, 1024, 4096), [1, 4096 * 64]),
    (product_bwd(F32, 1 << 24, 1000, 1000, 100), [(1 << 17) * 8, 6400]),
    (norm(BF, TOP, 1, 1), [TOP // 16]),
    (norm(F32, TOP // 64, 7, 64), [TOP // 1024]),
    (norm(BF, 1 << 25, 2048, 1), [1 << 25]),
    (norm_bwd(BF, TOP, 1, 1), [512, 2]),
    (norm_bwd(F32, 1 << 23, 8192, 2), [512, 256]),
    (ortho(BF, 65535, 8, 8), [65535]),
    (ortho(BF, 65535, 100, 1000), [65535, 65535, 65535]),
    (ortho(F32, 4, 16384, 16384), [1024, 4096, 8000]),
    (step(65535, 40, 300), [65535]),
    (step(3, 16384, 1), [3, 192]),
    (ortho(BF, 65535, 40, 16384), [65535, 65535 * 64, 65535 * 64]),
]


def test_largest_calls_have_legal_grids(tmp_path):
    for (call, least), (status, launches) in zip(CASES, record([c for c, _ in CASES], str(tmp_path))):
        assert status == 0, (call, status)
        assert len(launches) >= len(least), (call, launches)
        for n, launch in zip(least, launches):
            assert launch.workgroups >= n, (call, launch)
        assert all(launch.legal() for launch in launches), (call, launches)


def test_workspace_sizes_of_the_largest_calls():
    assert bmoe.bmoe_group_rows_workspace_bytes(TOP, 4096, 1) < 16 << 20
    n = bmoe.bmoe_orthogonalize_workspace_bytes(65535, 16384, 16384)
    assert n > 65535 * 16384 * 16384 * 2 * 8          # two parts of X twice, of P and of Q
    assert bmoe.bmoe_residual_norm_backward_workspace_bytes(F32, TOP, 8192) < 128 << 20
    n = bmoe.bmoe_grouped_product_backward_workspace_bytes(BF, TOP, 65536, 65536, 4096)
    assert 0 < n < 1 << 20                            # tiles enough: no ranges
    assert bmoe.bmoe_grouped_product_backward_workspace_bytes(F32, TOP, 64, 64, 1) >= 64 * 64 * 64 * 4
