"""The ends of the stated ranges: the widest rows, the longest sides, the most experts
and picks; with 64-bit references on the GPU."""
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe
from test_orthogonalize_gpu import tol

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def half(dt):
    return 2.0 ** -8 if dt == BF else 2.0 ** -24


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,O_", [(65536, 8), (65536, 1), (8, 65536), (1, 65536), (65535, 3), (3, 65535)])
def test_widest_products(K, O_, dt):
    g = torch.Generator(device="cuda").manual_seed(K)
    M, off = 200, [0, 60, 61, 61, 190]
    a = torch.randn(M, K, generator=g, device="cuda").to(dt)
    w = torch.randn(4, O_, K, generator=g, device="cuda").to(dt)
    dc = torch.randn(M, O_, generator=g, device="cuda").to(dt)
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    c = bmoe.grouped_product(a, w, offs)
    b = bmoe.grouped_product_backward(a, w, offs, dc)
    assert not c[190:].any() and not b["da"][190:].any()
    for e in range(4):
        q = slice(off[e], off[e + 1])
        x, y, z = a[q].double(), w[e].double(), dc[q].double()
        # one rounding to the type; each matrix instruction adds two products (fp32) or
        # more to a sum and moves it by at most 2^-23 of what it holds then, in the
        # mean square no more than the sum's last value
        for got, ref, n, t in ((c[q], x @ y.t(), K, dt), (b["da"][q], z @ y, O_, dt),
                               (b["dw"][e], z.t() @ x, len(x), F32)):
            err = (got.double() - ref).norm()
            assert err <= (half(t) + 2.0 ** -23 * (n / 2 + 2)) * ref.norm()


@pytest.mark.parametrize("shape", [(16384, 1), (1, 16384), (65, 16384), (16384, 65), (64, 16384)])
def test_longest_sides(shape):
    u = torch.randn(shape, generator=torch.Generator().manual_seed(1))
    o = bmoe.orthogonalize(u.cuda()).double().cpu().numpy()
    ref = O.newton_schulz(u.double().numpy())
    assert ((o - ref) ** 2).sum() ** 0.5 <= tol(5, F32) * (ref ** 2).sum() ** 0.5


def test_most_experts_captured():
    """Cursors for 4096 experts take more LDS than a launch has by default."""
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-1, 4096, (3000, 2), generator=g, dtype=torch.int32).cuda()
    bmoe.group_rows(ids, 4096)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bmoe.group_rows(ids, 4096)
    for i in range(3):
        ids.copy_(torch.randint(-1, 4096, (3000, 2), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, bmoe.group_rows(ids, 4096)):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("dt", [BF, F32])
def test_most_picks_of_the_widest_rows(dt):
    T, k, d = 3, 64, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(T * k, d, generator=g, device="cuda").to(dt)
    dr = torch.randn(T, d, generator=g, device="cuda").to(dt)
    inv = torch.randperm(T * k, generator=g, device="cuda").int()
    gates = torch.rand(T, k, generator=g, device="cuda")
    r, _ = bmoe.residual_norm(u, None, k=k, inv=inv, gates=gates)
    rows = u.double()[inv.long()].view(T, k, d)
    ref = (gates.double()[:, :, None] * rows).sum(1)
    mag = (gates.double()[:, :, None] * rows.abs()).sum(1)
    assert ((r.double() - ref).abs() <= half(dt) * ref.abs() + 2.0 ** -24 * 65 * mag).all()
    t = bmoe.residual_norm_backward(u, r, k=k, inv=inv, gates=gates, dr_out=dr)
    want = gates.double()[:, :, None] * dr.double()[:, None]
    got = t["du"].double()[inv.long()].view(T, k, d)
    assert ((got - want).abs() <= (half(dt) + 2.0 ** -24) * want.abs()).all()
    terms = dr.double()[:, None] * rows
    err = (t["dgates"].double() - terms.sum(2)).abs()
    assert (err <= 2.0 ** -24 * 41 * terms.abs().sum(2)).all()
