"""The launches that calls of the C entry points make, recorded on the CPU.

A small library in front of HIP's takes the launch functions: it notes grid,
workgroup and dynamic LDS and launches nothing. It has to be loaded before
libbmoe.so, so the calls run in a Python process of their own. Pointers are
made-up addresses that no host code reads."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
#include <cstddef>
#include <vector>
struct dim3 { unsigned x, y, z; };
static std::vector<unsigned long long> seen;
static int note(const void* f, dim3 g, dim3 b, size_t lds) {
  for (unsigned long long v : {(unsigned long long)g.x, (unsigned long long)g.y,
                               (unsigned long long)g.z, (unsigned long long)b.x,
                               (unsigned long long)b.y, (unsigned long long)b.z,
                               (unsigned long long)lds, (unsigned long long)f})
    seen.push_back(v);
  return 0;
}
extern "C" {
int hipExtLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t lds, void*, void*, void*, int) {
  return note(f, g, b, lds);
}
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t lds, void*) {
  return note(f, g, b, lds);
}
int hipGetLastError() { return 0; }
size_t seen_count() { return seen.size() / 8; }
const unsigned long long* seen_data() { return seen.data(); }
void seen_clear() { seen.clear(); }
}
"""

CHILD = r"""
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
stub.seen_count.restype = ctypes.c_size_t
stub.seen_data.restype = ctypes.POINTER(ctypes.c_ulonglong)
from butterfly_rotated_ternary_amd import bmoe
out = []
for name, args in json.load(sys.stdin):
    args = [ctypes.byref(bmoe.RouteSpec(**a)) if isinstance(a, dict) else
            (bmoe.BmoeTensor * len(a))(*map(tuple, a)) if isinstance(a, list) else a for a in args]
    stub.seen_clear()
    status = getattr(bmoe.lib(), name)(*args)
    d = stub.seen_data()
    out.append([status, [[d[8 * i + j] for j in range(8)] for i in range(stub.seen_count())]])
print(json.dumps(out))
"""


class Launch:
    def __init__(self, v):
        self.grid, self.block, self.lds = tuple(v[:3]), tuple(v[3:6]), v[6]
        self.kernel = v[7]  # equal for launches of one kernel within a recording

    @property
    def workgroups(self):
        return self.grid[0] * self.grid[1] * self.grid[2]

    def legal(self):
        """Within what HIP and the chip take: fewer than 2^32 threads per
        dimension, no empty dimension, at most 1024 threads and 160 KB."""
        return (all(g > 0 and b > 0 and g * b < 1 << 32 for g, b in zip(self.grid, self.block))
                and self.block[0] * self.block[1] * self.block[2] <= 1024 and self.lds <= 160 << 10)

    def __repr__(self):
        return f"Launch(grid={self.grid}, block={self.block}, lds={self.lds})"


def record(calls, tmp_path):
    """[(status, [Launch])] of calls [(entry point, [arguments])]; a dict among
    the arguments is a RouteSpec's, a list one of bmoe_tensor (address, entries,
    type)."""
    src, lib = os.path.join(tmp_path, "stub.cpp"), os.path.join(tmp_path, "stub.so")
    with open(src, "w") as f:
        f.write(STUB)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", src, "-o", lib], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, lib], input=json.dumps(calls), text=True,
                       capture_output=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    return [(s, [Launch(v) for v in ls]) for s, ls in json.loads(r.stdout.splitlines()[-1])]
