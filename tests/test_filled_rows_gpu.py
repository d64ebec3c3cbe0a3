"""Rows that belong to no group and rows that no pick names: 0 in what the library's
wrappers allocate, as they were in what the caller gives."""
import pytest
import torch

from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def poisoned(*shapes, dt):
    """Leaves memory full of NaN to the next allocations of these sizes."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    keep = [torch.full(s, float("nan"), dtype=dt, device="cuda") for s in shapes]
    torch.cuda.synchronize()
    del keep


def ids_of(T, k, N, pad, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, N, generator=g).topk(k, dim=1).indices.int()
    if pad:
        ids[torch.rand(T, k, generator=g) < pad] = -1
    return ids.cuda()


# few rows a group (no tiles), tiles of each width, aligned rows and not, all rows
# padded, none
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,N,K,O_", [(1, 8, 256, 512, 264), (37, 3, 60, 100, 203),
                                        (700, 2, 16, 200, 1000), (2050, 2, 16, 201, 515),
                                        (4110, 2, 60, 520, 1032), (257, 2, 2, 3, 5)])
@pytest.mark.parametrize("pad", [0.0, 0.2, 1.0])
def test_products(T, k, N, K, O_, pad, dt):
    g = torch.Generator(device="cuda").manual_seed(T)
    a = torch.randn(T, K, generator=g, device="cuda").to(dt)
    w = torch.randn(N, O_, K, generator=g, device="cuda").to(dt)
    dc = torch.randn(T * k, O_, generator=g, device="cuda").to(dt)
    off, perm, inv = bmoe.group_rows(ids_of(T, k, N, pad, K), N)
    end = int(off[-1])
    c = torch.full((T * k, O_), 7.0, dtype=dt, device="cuda")
    da = torch.full((T * k, K), 7.0, dtype=dt, device="cuda")
    bmoe.grouped_product(a, w, off, perm=perm, k=k, out=c)
    b = bmoe.grouped_product_backward(a, w, off, dc, perm=perm, k=k, da=da)
    assert (c[end:] == 7.0).all() and (da[end:] == 7.0).all()
    poisoned((T * k, O_), dt=dt)
    got = bmoe.grouped_product(a, w, off, perm=perm, k=k)
    assert torch.equal(got[:end], c[:end]) and not got[end:].any()
    poisoned((T * k, K), dt=dt)
    got = bmoe.grouped_product_backward(a, w, off, dc, perm=perm, k=k)
    assert torch.equal(got["da"][:end], da[:end]) and not got["da"][end:].any()
    assert torch.equal(got["dw"], b["dw"])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,O_", [(96, 160), (97, 161)])
def test_rows_before_and_between(K, O_, dt):
    """Groups that begin behind row 0; no group at all; many rows at both ends."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M = 2000
    a = torch.randn(M, K, generator=g, device="cuda").to(dt)
    dc = torch.randn(M, O_, generator=g, device="cuda").to(dt)
    for offs in ([3, 3, 132, 133, 700], [1500, 1501, 1501, 1501, 1600], [0, 0, 0, 0, 0],
                 [M] * 5, [0, 1, 2, 3, M], [700, 700, 700, 700, 700]):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        w = torch.randn(4, O_, K, generator=g, device="cuda").to(dt)
        lo, hi = offs[0], offs[-1]
        c = bmoe.grouped_product(a, w, off, out=torch.empty(M, O_, dtype=dt, device="cuda"))
        r = bmoe.grouped_product_backward(a, w, off, dc, da=torch.empty(M, K, dtype=dt, device="cuda"))
        poisoned((M, O_), (M, K), dt=dt)
        got = bmoe.grouped_product(a, w, off)
        back = bmoe.grouped_product_backward(a, w, off, dc)
        for x, y in ((got, c), (back["da"], r["da"])):
            assert torch.equal(x[lo:hi], y[lo:hi]) and not x[:lo].any() and not x[hi:].any(), offs


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,d,extra", [(1, 8, 4096, 0), (40, 4, 256, 9), (300, 2, 61, 5000),
                                         (1700, 3, 1030, 1), (33, 64, 20, 0), (9000, 2, 8, 70000)])
@pytest.mark.parametrize("pad", [0.0, 0.2, 1.0])
def test_norm_gradient(T, k, d, extra, pad, dt):
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = T * k + extra
    u = torch.randn(rows, d, generator=g, device="cuda").to(dt)
    r = torch.randn(T, d, generator=g, device="cuda").to(dt)
    inv = torch.randperm(rows, generator=g, device="cuda")[:T * k].int()
    inv[torch.rand(T * k, generator=g, device="cuda") < pad] = -1
    gates = torch.rand(T, k, generator=g, device="cuda")
    w = torch.ones(d, device="cuda")
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[inv[inv >= 0].long()] = True
    for kw in (dict(gates=gates, w_post=w, w_pre=w, dr_out=r, dn=r), dict(dr_out=r)):
        du = torch.full_like(u, 7.0)
        want = bmoe.residual_norm_backward(u, r, k=k, inv=inv, du=du, **kw)
        assert (du[~named] == 7.0).all()
        poisoned((rows, d), dt=dt)
        got = bmoe.residual_norm_backward(u, r, k=k, inv=inv, **kw)
        assert torch.equal(got["du"][named], du[named]) and not got["du"][~named].any()
        for name in ("dr", "dgates", "dw_post", "dw_pre"):
            assert want[name] is None or torch.equal(want[name], got[name]), name


def test_marks_of_an_earlier_call_name_nothing():
    """What a workspace held before says nothing about the rows of this call."""
    T, k, d = 64, 2, 32
    g = torch.Generator(device="cuda").manual_seed(0)
    u, r = torch.randn(T * k, d, device="cuda"), torch.randn(T, d, device="cuda")
    full = torch.randperm(T * k, generator=g, device="cuda").int()
    some = full.clone()
    some[::3] = -1
    n = bmoe.bmoe_residual_norm_backward_filled_workspace_bytes(bmoe.BMOE_F32, T, d, T * k)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    spec = bmoe.NormSpec()
    for inv in (full, some, full.flip(0), some.flip(0)):
        du = torch.full_like(u, float("nan"))
        dr = torch.empty_like(r)
        assert bmoe.bmoe_residual_norm_backward_filled(
            bmoe.BMOE_F32, T, d, k, spec, u, T * k, inv, None, r, None, None, r, None, du, None, dr,
            None, None, ws) == 0
        named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
        named[inv[inv >= 0].long()] = True
        assert torch.isfinite(du).all() and not du[~named].any() and du[named].any(1).all()


def test_no_tokens_name_no_row():
    u, r = torch.randn(5, 16, device="cuda"), torch.empty(0, 16, device="cuda")
    poisoned((5, 16), dt=F32)
    got = bmoe.residual_norm_backward(u, r, inv=torch.empty(0, dtype=torch.int32, device="cuda"),
                                      dr_out=r)
    assert not got["du"].any()


def test_captured_and_replayed():
    T, k, N, K, O_ = 200, 2, 9, 72, 40
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn(T, K, generator=g, device="cuda")
    w = torch.randn(N, O_, K, generator=g, device="cuda")
    ids = ids_of(T, k, N, 0.3, 1)
    r = torch.randn(T, O_, generator=g, device="cuda")

    def step():
        off, perm, inv = bmoe.group_rows(ids, N)
        c = bmoe.grouped_product(a, w, off, perm=perm, k=k)
        t = bmoe.residual_norm_backward(c, r, k=k, inv=inv, dr_out=r)
        b = bmoe.grouped_product_backward(a, w, off, t["du"], perm=perm, k=k)
        return [c, t["du"], b["da"], b["dw"]]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        ids.copy_(ids_of(T, k, N, 0.1 * i, i))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, step()):
            assert torch.equal(x, y), i


def test_rows_behind_the_picks_without_inv():
    T, k, d, rows = 30, 2, 100, 67
    u, r = torch.randn(rows, d, device="cuda"), torch.randn(T, d, device="cuda")
    du, dr = torch.full_like(u, float("nan")), torch.empty_like(r)
    n = bmoe.bmoe_residual_norm_backward_filled_workspace_bytes(bmoe.BMOE_F32, T, d, rows)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert bmoe.bmoe_residual_norm_backward_filled(
        bmoe.BMOE_F32, T, d, k, bmoe.NormSpec(), u, rows, None, None, r, None, None, r, None, du,
        None, dr, None, None, ws) == 0
    assert torch.equal(du[:T * k], r.repeat_interleave(k, 0)) and not du[T * k:].any()
