"""The operators around a block together, as a training step uses them; captured
and replayed, on two streams, and with arrays of more than 2^31 entries."""
import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LR, DECAY = 0.02, 0.1


def params(T, d, N, f, k, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = dict(x=torch.randn(T, d, generator=g), w_r=torch.randn(N, d, generator=g) / d ** 0.5,
             w1=torch.randn(N, f, d, generator=g) / d ** 0.5,
             w2=torch.randn(N, d, f, generator=g) / f ** 0.5)
    p = {key: v.to(dt) for key, v in p.items()}
    for key in ("g0", "g1", "g2"):
        p[key] = 1 + 0.1 * torch.randn(d, generator=g)
    p["dr"], p["dn"] = torch.randn(T, d, generator=g).to(dt), torch.randn(T, d, generator=g).to(dt)
    return p


SPEC = dict(score="sigmoid", scale=1.0)
NORM = dict(eps=1e-6, res_scale=0.9, out_scale=1.1)


def forward_backward(p, k):
    """A block of dense experts (squared ReLU between its products) between its
    norms, and every gradient."""
    N = p["w_r"].shape[0]
    spec, norm = bmoe.RouteSpec(**SPEC), bmoe.NormSpec(**NORM)
    first = bmoe.NormSpec(eps=NORM["eps"])
    _, n0 = bmoe.residual_norm(None, p["x"], first, w_pre=p["g0"])
    logits = bmoe.router_logits(n0, p["w_r"])
    ids, gates = bmoe.route_logits(logits, k, spec)
    offsets, perm, inv = bmoe.group_rows(ids, N)
    h = bmoe.grouped_product(n0, p["w1"], offsets, perm=perm, k=k)
    a = torch.relu(h).square()
    u = bmoe.grouped_product(a, p["w2"], offsets)
    r, n1 = bmoe.residual_norm(u, p["x"], norm, k=k, inv=inv, gates=gates, w_post=p["g1"], w_pre=p["g2"])
    t = bmoe.residual_norm_backward(u, r, norm, k=k, inv=inv, gates=gates, w_post=p["g1"],
                                    w_pre=p["g2"], dr_out=p["dr"], dn=p["dn"])
    b2 = bmoe.grouped_product_backward(a, p["w2"], offsets, t["du"])
    dh = b2["da"] * (2 * torch.relu(h))
    b1 = bmoe.grouped_product_backward(n0, p["w1"], offsets, dh, perm=perm, k=k)
    dn0, _ = bmoe.residual_norm(b1["da"], None, k=k, inv=inv)
    rb = bmoe.router_backward(n0, p["w_r"], logits, ids, t["dgates"], spec, dx_add=dn0)
    b0 = bmoe.residual_norm_backward(None, p["x"], first, w_pre=p["g0"], dr_out=t["dr"], dn=rb["dx"])
    out = dict(r=r, n=n1, x=b0["dr"], w1=b1["dw"], w2=b2["dw"], w_r=rb["dw"], g0=b0["dw_pre"],
               g1=t["dw_post"], g2=t["dw_pre"])
    return ids, out


def reference(p, ids, k):
    """The same in 64 bits by torch's differentiation, experts chosen as given."""
    q = {key: v.cpu().double().requires_grad_(key not in ("dr", "dn")) for key, v in p.items()}

    def rms(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + NORM["eps"]) * w
    n0 = rms(q["x"], q["g0"])
    s = torch.sigmoid(n0 @ q["w_r"].t())
    i = ids.cpu().long()
    g = s.gather(1, i)
    g = g / g.sum(1, keepdim=True)
    y = 0
    for j in range(k):
        h = torch.einsum("td,tfd->tf", n0, q["w1"][i[:, j]])
        y = y + g[:, j:j + 1] * torch.einsum("tf,tdf->td", torch.relu(h).square(), q["w2"][i[:, j]])
    r = NORM["res_scale"] * q["x"] + NORM["out_scale"] * rms(y, q["g1"])
    n = rms(r, q["g2"])
    keys = ["x", "w1", "w2", "w_r", "g0", "g1", "g2"]
    grads = torch.autograd.grad((r * q["dr"]).sum() + (n * q["dn"]).sum(), [q[key] for key in keys])
    return dict(r=r.detach(), n=n.detach(), **dict(zip(keys, grads)))


# fp32: a chain of at most 12 operators, each a sum of at most 300 terms: 12 *
# 316 * 2^-24 = 2.3e-4 relative to the terms, which exceed the results by less
# than 4 in the norm. bf16: about 12 roundings of 2^-8 on the way, as independent
# errors sqrt(12) * 2^-8 = 1.4e-2, again 4 for cancelling terms.
@pytest.mark.parametrize("dt,bound", [(F32, 1e-3), (BF, 5.6e-2)])
@pytest.mark.parametrize("T,d,N,f,k", [(150, 64, 7, 100, 3), (33, 256, 16, 40, 2), (1, 128, 5, 64, 1)])
def test_block_and_gradients(T, d, N, f, k, dt, bound):
    p = {key: v.cuda() for key, v in params(T, d, N, f, k, dt, seed=T).items()}
    ids, out = forward_backward(p, k)
    ref = reference(p, ids, k)
    for key, v in ref.items():
        got = out[key].cpu().double()
        assert float((got - v).norm()) <= bound * float(v.norm()) + 1e-30, key


@pytest.mark.parametrize("dt", [F32, BF])
def test_whole_step_of_the_weights(dt):
    """Clipped gradients through the orthogonalised step, each weight as its
    oracle says for the gradient that it was given."""
    k = 2
    p = {key: v.cuda() for key, v in params(200, 64, 6, 96, k, dt, seed=3).items()}
    _, out = forward_backward(p, k)
    grads = [out["w1"], out["w2"], out["w_r"]]
    norm = bmoe.clip_grads(grads, 1.0)
    assert torch.isfinite(norm)
    for key, g in zip(("w1", "w2", "w_r"), grads):
        w = p[key].clone()
        m = torch.zeros_like(g)
        bmoe.orthogonal_step(w, g, m, LR, weight_decay=DECAY)
        assert torch.equal(m, g)
        u = g.cpu().double().numpy() * (1 + float(np.float32(0.95)))
        o = np.stack([O.newton_schulz(x) for x in u.reshape(-1, *u.shape[-2:])]).reshape(u.shape)
        want = (1 - LR * DECAY) * p[key].cpu().double().numpy() - LR * o
        half = 2.0 ** -8 if dt == BF else 2.0 ** -24
        err = np.abs(w.cpu().double().numpy() - want) - half * np.abs(want) - 2.0 ** -22 * np.abs(want)
        # the iteration's own error (the bound of its tests) spread over a matrix
        assert np.linalg.norm(np.maximum(err, 0)) <= LR * np.linalg.norm(o) * 6.5e-4, key


def test_captured_and_replayed():
    k = 2
    p = {key: v.cuda() for key, v in params(300, 128, 9, 72, k, BF, seed=4).items()}
    w, m = torch.randn(3, 200, 96, device="cuda"), torch.zeros(3, 200, 96, device="cuda")
    v, mv = torch.randn(40, 64, device="cuda"), torch.zeros(40, 64, device="cuda")
    gw, gv = torch.randn_like(w), torch.randn_like(v)

    def step(w, m, v, mv):
        _, out = forward_backward(p, k)
        bmoe.orthogonal_step(w, gw, m, 0.1)
        bmoe.orthogonal_step(v, gv, mv, 0.1)
        return list(out.values()) + [w, m, v, mv]
    step(*[t.clone() for t in (w, m, v, mv)])
    torch.cuda.synchronize()
    state = [t.clone() for t in (w, m, v, mv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*state)
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(4):
        for t in (p["x"], p["dr"], p["dn"], gw, gv):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        ref = step(*before)
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, do not meet."""
    k = 2
    ps = [{key: v.cuda() for key, v in params(500 + 37 * i, 256, 8, 128, k, BF, seed=i).items()}
          for i in range(2)]
    us = [torch.randn(2, 300, 200, device="cuda") for _ in range(2)]
    want = [(forward_backward(p, k)[1], bmoe.orthogonalize(u)) for p, u in zip(ps, us)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = (forward_backward(ps[i], k)[1], bmoe.orthogonalize(us[i]))
    torch.cuda.synchronize()
    for (a, o), (b, q) in zip(want, got):
        assert torch.equal(o, q) and all(torch.equal(a[key], b[key]) for key in a)


def test_stream_argument():
    s = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.randint(0, 5, (400, 2), generator=g, device="cuda", dtype=torch.int32)
    x, w = torch.randn(400, 64, device="cuda"), torch.randn(5, 48, 64, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    off, perm, inv = bmoe.group_rows(ids, 5, stream=s)
    c = bmoe.grouped_product(x, w, off, perm=perm, k=2, stream=s)
    r, _ = bmoe.residual_norm(c, None, k=2, inv=inv, stream=s)
    o = bmoe.orthogonalize(w, stream=s)
    t = bmoe.residual_norm_backward(c, r, k=2, inv=inv, dr_out=r, stream=s)
    b = bmoe.grouped_product_backward(x, w, off, t["du"], perm=perm, k=2, stream=s)
    s.synchronize()
    off2, perm2, inv2 = bmoe.group_rows(ids, 5)
    c2 = bmoe.grouped_product(x, w, off2, perm=perm2, k=2)
    r2, _ = bmoe.residual_norm(c2, None, k=2, inv=inv2)
    t2 = bmoe.residual_norm_backward(c2, r2, k=2, inv=inv2, dr_out=r2)
    b2 = bmoe.grouped_product_backward(x, w, off2, t2["du"], perm=perm2, k=2)
    assert torch.equal(perm, perm2) and torch.equal(c, c2) and torch.equal(r, r2)
    assert torch.equal(o, bmoe.orthogonalize(w)) and torch.equal(b["dw"], b2["dw"])


# ---- arrays of more than 2^31 entries ------------------------------------------------

def test_rows_past_32_bits():
    """Expert rows and tokens that lie past entry 2^31 of their arrays."""
    R, d, T, k = 530000, 4096, 40, 3                     # 2.17e9 bf16 entries
    g = torch.Generator(device="cuda").manual_seed(7)
    big = torch.zeros(R, d, dtype=BF, device="cuda")
    rows = torch.randperm(2000, generator=g, device="cuda")[:T * k] + (R - 2000)
    big[rows] = torch.randn(T * k, d, generator=g, device="cuda").to(BF)
    small, r = big[rows].contiguous(), torch.randn(T, d, generator=g, device="cuda").to(BF)
    w = torch.ones(d, device="cuda")
    kw = dict(k=k, w_post=w, w_pre=w)
    far = bmoe.residual_norm(big, r, inv=rows.int(), **kw)
    near = bmoe.residual_norm(small, r, **kw)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    du = torch.zeros_like(big)
    a = bmoe.residual_norm_backward(big, r, inv=rows.int(), dr_out=r, dn=r, du=du, **kw)
    b = bmoe.residual_norm_backward(small, r, dr_out=r, dn=r, **kw)
    assert torch.equal(du[rows], b["du"]) and torch.equal(a["dw_post"], b["dw_post"])
    del du
    wt = torch.randn(2, 96, d, generator=g, device="cuda").to(BF) / 64
    off = torch.tensor([0, 50, T * k], dtype=torch.int32, device="cuda")
    c = bmoe.grouped_product(big, wt, off, perm=rows.int())
    assert torch.equal(c, bmoe.grouped_product(small, wt, off))
    dc = torch.randn(T * k, 96, generator=g, device="cuda").to(BF)
    a = bmoe.grouped_product_backward(big, wt, off, dc, perm=rows.int())
    b = bmoe.grouped_product_backward(small, wt, off, dc)
    assert torch.equal(a["dw"], b["dw"]) and torch.equal(a["da"], b["da"])


def test_experts_past_32_bits():
    """The last of 140 experts of 4096 x 4096: its weights, and its gradient."""
    G, d, M = 140, 4096, 130
    g = torch.Generator(device="cuda").manual_seed(8)
    w = torch.zeros(G, d, d, dtype=BF, device="cuda")
    w[-1] = torch.randn(d, d, generator=g, device="cuda").to(BF) / 64
    a = torch.randn(M, d, generator=g, device="cuda").to(BF)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[-1] = M
    last = w[-1:].contiguous()
    # (other tile widths than for one expert: sums in another order)
    ref = a.double() @ last[0].double().t()
    mag = a.double().abs() @ last[0].double().abs().t()
    err = (bmoe.grouped_product(a, w, off).double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -23 * (d + 1) * mag).all()
    got = bmoe.grouped_product_backward(a, w, off, a)
    assert not got["dw"][:-1].any()
    ref = a.double().t() @ a.double()
    mag = a.double().abs().t() @ a.double().abs()
    assert ((got["dw"][-1].double() - ref).abs() <= 2.0 ** -23 * (M + 1) * mag).all()
    ref = a.double() @ last[0].double()
    mag = a.double().abs() @ last[0].double().abs()
    err = (got["da"].double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -23 * (d + 1) * mag).all()


def test_matrices_past_32_bits():
    """A batch of 2100 matrices of 1024 x 1024 bf16: the last as if alone."""
    B, n = 2100, 1024
    g = torch.Generator(device="cuda").manual_seed(9)
    u = torch.empty(B, n, n, dtype=BF, device="cuda")
    for i in range(0, B, 100):
        u[i:i + 100] = torch.randn(100, n, n, generator=g, device="cuda")
    o = bmoe.orthogonalize(u)
    for i in (0, 1040, B - 1):
        alone = bmoe.orthogonalize(u[i])
        # (other tiles: sums in another order, then a rounding to bf16)
        diff = (o[i].double() - alone.double()).norm() / alone.double().norm()
        assert float(diff) <= 2.0 ** -8, i


def test_most_rows():
    """2^31 - 1 rows, the most there can be: their numbers' last sums do not wrap."""
    M = 2 ** 31 - 1
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    a = torch.zeros(M, 1, dtype=BF, device="cuda")
    dc = torch.zeros(M, 1, dtype=BF, device="cuda")
    w = torch.full((1, 1, 1), 3.0, dtype=BF, device="cuda")
    tail = torch.arange(1, 41, dtype=BF, device="cuda")[:, None]
    a[-40:], dc[-40:] = tail, 2 * tail
    a[5], dc[5] = 100.0, 1.0
    c = bmoe.grouped_product(a, w, off)
    assert torch.equal(c[-40:], 3 * tail) and float(c[5]) == 300.0
    assert int(torch.count_nonzero(c)) == 41
    del c
    g = bmoe.grouped_product_backward(a, w, off, dc)
    assert float(g["dw"]) == 100.0 + 2.0 * sum(i * i for i in range(1, 41))
    assert torch.equal(g["da"][-40:], 6 * tail) and int(torch.count_nonzero(g["da"])) == 41
    del a, dc, g
    ids = torch.ones(M, 1, dtype=torch.int32, device="cuda")
    ids[-3:] = 0
    ids[7] = 9                                           # a padded pick
    off, perm, inv = bmoe.group_rows(ids, 2)
    assert off.tolist() == [0, 3, M - 1]
    assert perm[:5].tolist() == [M - 3, M - 2, M - 1, 0, 1] and int(perm[-1]) == 7
    assert inv[-4:].tolist() == [M - 2, 0, 1, 2] and int(inv[7]) == -1
    assert torch.equal(perm[3 + 7:3 + 1000], torch.arange(8, 1001, dtype=torch.int32, device="cuda"))
