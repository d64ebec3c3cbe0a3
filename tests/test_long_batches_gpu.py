"""GPU parity of routing, its gradient and the router's backward on batches of
more than 2^20 workgroups, whose grids have rows along a second dimension.
Every entry is compared with the definition in 64 bits (torch, on the GPU),
with the tolerances of the smaller batches' tests."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe
from test_route_gpu import U, eps_of

pytestmark = pytest.mark.gpu


def parts(T, n=1 << 22):
    return [slice(a, min(T, a + n)) for a in range(0, T, n)]


def eps(l):
    """eps_of() of finite logits, on the GPU: U (2 D + 96) a row."""
    hi, lo = l.amax(1, keepdim=True), l.amin(1, keepdim=True)
    return U * (2 * torch.maximum(hi - lo, torch.maximum(hi.abs(), lo.abs())) + 96)


def dlogits(l, ids, dg, score, renorm, scale):
    """(dl, the same with each term by its magnitude), fp64 [T][N]; distinct ids."""
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    s1 = torch.sigmoid(-l) if score == "sigmoid" else torch.ones_like(l)
    u = torch.zeros_like(l).scatter_(1, ids, scale * dg)
    if not renorm and score == "softmax":
        d = (u * s).sum(1, keepdim=True)
        return s * (u - d), s * (u.abs() + (u * s).abs().sum(1, keepdim=True))
    p = torch.zeros_like(l).scatter_(1, ids, s.gather(1, ids))
    if not renorm:
        return u * p * s1, u.abs() * p * s1
    p = p / p.sum(1, keepdim=True)
    return (p * s1 * (u - (u * p).sum(1, keepdim=True)),
            p * s1 * (u.abs() + (u * p).abs().sum(1, keepdim=True)))


@pytest.mark.parametrize("spec", [("sigmoid", True), ("softmax", False)], ids=str)
def test_route_and_its_gradient(spec):
    T, N, k = (1 << 24) + 37, 4, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(T, N, generator=g, device="cuda")
    dg = torch.randn(T, k, generator=g, device="cuda")
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1], scale=1.5)
    print(f"[route] T={T} N={N} k={k} {spec}", flush=True)
    ids, gates = bmoe.route_logits(l, k, sp)
    dl = torch.full((T, N), math.nan, device="cuda")
    bmoe.route_logits_backward(l, ids, dg, sp, dlogits=dl)
    for r in parts(T):
        l64 = l[r].double()
        want = torch.sort(l64, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(ids[r].long(), want)
        s = torch.sigmoid(l64) if spec[0] == "sigmoid" else torch.softmax(l64, 1)
        wg = s.gather(1, want)
        wg = 1.5 * (wg / wg.sum(1, keepdim=True) if spec[1] else wg)
        assert ((gates[r].double() - wg).abs() <= eps(l64) * wg).all()
        ref, mag = dlogits(l64, want, dg[r].double(), *spec, 1.5)
        assert ((dl[r].double() - ref).abs() <= 4 * eps(l64) * mag + 2.0 ** -126).all()


def check_products(x, w, l, ids, dg, spec, chain):
    """dx and dW of the whole batch; a sum of dW is a chain of at most `chain`
    additions, each off by U of what it adds up."""
    T, N = l.shape
    dx = torch.full_like(x, math.nan)
    out = bmoe.router_backward(x, w, l, ids, dg, bmoe.RouteSpec(spec[0], renorm=spec[1], scale=1.5),
                               dx=dx)
    w64 = w.double()
    dw, mw = torch.zeros_like(w64), torch.zeros_like(w64)
    for r in parts(T):
        l64 = l[r].double()
        ref, mag = dlogits(l64, ids[r].long(), dg[r].double(), *spec, 1.5)
        x64 = x[r].double()
        wx, mx = ref @ w64, ((4 * eps(l64) + (N + 2) * U) * mag) @ w64.abs()
        assert ((dx[r].double() - wx).abs() <= mx + U * (wx.abs() + mx) + 2.0 ** -126).all()
        dw += ref.t().contiguous() @ x64
        mw += ((4 * eps(l64) + (chain + 2) * U) * mag).t().contiguous() @ x64.abs()
    assert ((out["dw"].double() - dw).abs() <= mw + 2.0 ** -126).all()


def test_router_backward_of_many_picks():
    """17 of 17 experts: the pairs of a token take a wave."""
    T, d, N, k = (1 << 22) + 13, 16, 17, 17
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, d, generator=g, device="cuda")
    w = torch.randn(N, d, generator=g, device="cuda") / 4
    l = torch.randn(T, N, generator=g, device="cuda")
    dg = torch.randn(T, k, generator=g, device="cuda")
    ids = torch.argsort(torch.rand(T, N, generator=g, device="cuda"), dim=1).to(torch.int32)
    print(f"[router_backward] T={T} d={d} N={N} k={k}", flush=True)
    # ranges of 1024 tokens, four to a workgroup, the groups one after the other
    check_products(x, w, l, ids, dg, ("softmax", True), 1024 + 4 + T // 4096 + 1)


def test_dense_router_backward_in_fp32():
    """2^20 tiles of 64 tokens and some, in a grid whose second dimension is the
    columns'."""
    T, d, N, k = (1 << 26) + 70, 16, 2, 1
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, d, generator=g, device="cuda")
    w = torch.randn(N, d, generator=g, device="cuda") / 4
    l = torch.randn(T, N, generator=g, device="cuda")
    dg = torch.randn(T, k, generator=g, device="cuda")
    ids = torch.randint(0, N, (T, k), generator=g, device="cuda", dtype=torch.int32)
    print(f"[router_backward] T={T} d={d} N={N} k={k} dense", flush=True)
    # 2048 ranges of tokens, added one after the other
    check_products(x, w, l, ids, dg, ("softmax", False), T // 2048 + 16 + 2048)


def test_route_of_groups_that_no_lane_layout_holds():
    """Every token by a wave in 64 bits (33 groups of 66 experts)."""
    T, N, k = (1 << 22) + 5, 33 * 66, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    l = torch.empty(T, N, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    print(f"[route] T={T} N={N} k={k} in 33 groups", flush=True)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((T, k), -7.0, device="cuda")
    bmoe.route_logits(l, k, bmoe.RouteSpec("sigmoid", n_groups=33, topk_groups=5), ids=ids,
                      gates=gates)
    assert (ids >= 0).all() and (ids < N).all() and (gates > 0).all()
    rows = torch.cat([torch.arange(0, 40), torch.arange((1 << 22) - 40, T)]).cuda()
    l64 = l[rows].double().cpu().numpy()
    oid, og = O.route_logits(l64, k, score="sigmoid", n_groups=33, topk_groups=5)
    assert np.array_equal(ids[rows].cpu().numpy(), oid)
    assert (np.abs(gates[rows].double().cpu().numpy() - og) <= eps_of(l64) * og).all()


@pytest.mark.parametrize("dt,T", [(torch.float32, (1 << 26) + 70), (torch.bfloat16, (1 << 25) + 35)],
                         ids=["f32", "bf16"])
def test_plain_router(dt, T):
    """Logits of more than 2^20 tiles of tokens, and as many workgroups of the
    choice. A logit is a sum of 16 terms, its products in bf16 exact."""
    d, N, k = 16, 3, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=g, device="cuda").to(dt)
    w = torch.randn(N, d, generator=g, device="cuda").to(dt)
    print(f"[router] T={T} d={d} N={N} {dt}", flush=True)
    ids, gates, logits = bmoe.route(x, w, k, want_logits=True)
    assert torch.equal(bmoe.router_logits(x, w), logits)
    for r in parts(T):
        ref = x[r].double() @ w.double().t().contiguous()
        mag = x[r].double().abs() @ w.double().abs().t().contiguous()
        l64 = logits[r].double()
        assert ((l64 - ref).abs() <= 17 * U * mag).all()
        want = torch.sort(l64, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(ids[r].long(), want)
        wg = torch.softmax(l64.gather(1, want), 1)
        assert ((gates[r].double() - wg).abs() <= eps(l64) * wg).all()
