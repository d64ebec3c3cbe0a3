"""Gradient norm and clipping of lists above 64 MB, where a workgroup takes a
run of more than eight chunks of 4 KB, often over several tensors. Random data,
every entry compared in 64 bits (on the GPU), with the tolerances of the short
lists' tests: the norm is off by its one rounding (and 2^-40 for the sums), an
entry by the factor's two, the product's and its type's."""
import numpy as np
import pytest
import torch

from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
CHUNK = 4096

_RNG = np.random.default_rng(7)
LISTS = {  # alternately fp32 and bf16
    "few": [9000003, 20000005, 1, 7000013, 5000000],
    "many": [int(v) for v in _RNG.integers(100000, 2000000, 40)],
    # above 256 MB: the norm streams
    "large": [45000001, 80000003, 777],
    # more than one table of 112 tensors, each of runs
    "tables": [int(v) for v in _RNG.integers(100000, 400000, 250)],
}


def lay_out(sizes, offset, fill=None):
    """(tensors `offset` entries past an aligned start, their buffers, which end
    in 16 more guard entries)."""
    ts, bufs = [], []
    for i, n in enumerate(sizes):
        dt = torch.bfloat16 if i % 2 else torch.float32
        buf = torch.full((offset + n + 16,), -7.0, dtype=dt, device="cuda")
        ts.append(buf[offset:offset + n])
        if fill is not None:
            ts[-1].copy_(fill[i])
        bufs.append(buf)
    return ts, bufs


def slices(n, m=1 << 26):
    return [slice(a, min(n, a + m)) for a in range(0, n, m)]


def norm64(ts):
    return sum(float((t[r].double() ** 2).sum()) for t in ts for r in slices(t.numel())) ** 0.5


def check_scaled(got, before, f):
    for a, b in zip(got, before):
        for r in slices(a.numel()):
            want = b[r].double() * f
            tol = (3.1 * U + HALF[a.dtype]) * want.abs() + 2.0 ** -126
            assert ((a[r].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("offset,out_offset", [(0, 0), (0, 3), (3, 3), (5, 2)])
def test_clip_of_long_runs(name, offset, out_offset):
    sizes = LISTS[name]
    size = [n * (2 if i % 2 else 4) for i, n in enumerate(sizes)]
    total = sum(size)
    assert sum(size[:112]) > 2048 * 8 * CHUNK     # runs of more than eight chunks (a table's)
    assert (total > 256 << 20) == (name == "large")
    g = torch.Generator(device="cuda").manual_seed(len(sizes) + offset)
    data = [torch.randn(n, generator=g, device="cuda") for n in sizes]
    ts, bufs = lay_out(sizes, offset, data)
    before = [t.clone() for t in ts]
    out, obufs = lay_out(sizes, out_offset)
    del data
    ref = norm64(before)
    most = float(np.float32(0.3 * ref))
    print(f"[clip] {name}: {total / 1e6:.0f} MB, offsets {offset}, {out_offset}", flush=True)
    only = bmoe.grad_norm(ts)
    n1 = bmoe.clip_grads(ts, most, out=out)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    check_scaled(out, before, most / ref)
    # a factor of 1 copies
    kept, kbufs = lay_out(sizes, out_offset)
    bmoe.scale_grads(ts, only, 2 * most / 0.3, out=kept)
    assert all(torch.equal(a, b) for a, b in zip(kept, before))
    n2 = bmoe.clip_grads(ts, most)
    assert all(torch.equal(a, b) for a, b in zip(ts, out))
    assert torch.equal(only, n1) and torch.equal(only, n2)
    assert abs(float(only) - ref) <= (U + 2.0 ** -40) * ref
    for bs, o in ((bufs, offset), (obufs, out_offset), (kbufs, out_offset)):
        assert all((b[:o] == -7).all() and (b[-16:] == -7).all() for b in bs)


def test_clip_of_more_values_than_32_bits_count():
    """Random values on both sides of entry 2^31, all of them compared; in
    place, in one list with fp32 on either side."""
    g = torch.Generator(device="cuda").manual_seed(11)
    n = 2 ** 31 + 12345
    big = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ts = [torch.randn(1000003, generator=g, device="cuda"), big[3:],
          torch.randn(3000001, generator=g, device="cuda")]
    before = [t.clone() for t in ts]
    ref = norm64(before)
    most = float(np.float32(0.7 * ref))
    print(f"[clip] {n} entries", flush=True)
    norm = bmoe.clip_grads(ts, most)
    assert abs(float(norm) - ref) <= (U + 2.0 ** -40) * ref
    check_scaled(ts, before, most / ref)
