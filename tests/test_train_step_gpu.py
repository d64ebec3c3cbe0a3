"""GPU parity of the router's backward and of gradient clipping with the fp64
oracle, and of a whole training step of the layer: router, layer, backward of
both, loads, clipping."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe
from butterfly_rotated_ternary_amd import workloads as W
from devinputs import to_device
from test_route_gpu import SPECS, U, eps_of, grad_scale, rounded

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step of the type, relative


def check_router_backward(T, d, N, k, dt, spec, add, seed, ids=None, l=None, alias=False):
    rng = np.random.default_rng(seed)
    x_dev, x = rounded(rng.normal(0, 1, (T, d)), dt)
    w_dev, w = rounded(rng.normal(0, 1, (N, d)) / math.sqrt(d), dt)
    l_dev, l = rounded(rng.normal(0, 1, (T, N)) if l is None else l, "f32")
    if ids is None:
        ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    a_dev, a = rounded(rng.normal(0, 1, (T, d)), dt) if add else (None, None)
    score, renorm = spec
    # outputs inside larger buffers: nothing outside is written
    bx = torch.full((T * d + 256,), -7.0, device="cuda", dtype=x_dev.dtype)
    bw = torch.full((N * d + 256,), -7.0, device="cuda")
    dx, dw = bx[128:128 + T * d].view(T, d), bw[128:128 + N * d].view(N, d)
    if alias:
        dx.copy_(a_dev)
        a_dev = dx
    out = bmoe.router_backward(x_dev, w_dev, l_dev, torch.from_numpy(ids).cuda(),
                               torch.from_numpy(dg).cuda(),
                               bmoe.RouteSpec(score, renorm=renorm, scale=1.5), dx_add=a_dev,
                               dx=dx, dw=dw)
    torch.cuda.synchronize()
    for b, n in ((bx, T * d), (bw, N * d)):
        assert (b[:128] == -7).all() and (b[128 + n:] == -7).all()
    ref = O.router_backward(x, w, l, ids, dg, dx_add=a, score=score, renorm=renorm, scale=1.5)
    # dl is off by 4 EPS of its magnitude; a sum of n terms by n u of theirs
    A = grad_scale(l, ids, dg, score, renorm, 1.5)
    base = np.zeros((T, d)) if a is None else np.abs(a)
    sx = base * (N + 1) * U + ((4 * eps_of(l) + (N + 2) * U) * A) @ np.abs(w)
    sw = ((4 * eps_of(l) + (T + 2) * U) * A).T @ np.abs(x)
    got = out["dx"].double().cpu().numpy()
    err = np.abs(got - ref["dx"])
    tol = sx + HALF[dt] * (np.abs(ref["dx"]) + sx) + 2.0 ** -126
    assert (err <= tol).all(), float((err / tol).max())
    err = np.abs(out["dw"].double().cpu().numpy() - ref["dw"])
    tol = sw + 2.0 ** -126
    assert (err <= tol).all(), float((err / tol).max())
    return out


@pytest.mark.parametrize("T,d,N,k,dt,add", [
    (0, 64, 8, 2, "bf16", False), (1, 16, 1, 1, "f32", False), (1, 4096, 256, 4, "bf16", True),
    (3, 16, 5, 2, "bf16", True), (130, 64, 8, 2, "f32", True), (257, 512, 64, 2, "bf16", True),
    (100, 128, 65, 3, "f32", False), (65, 32, 33, 8, "bf16", False), (37, 8192, 20, 4, "bf16", True),
    (50, 256, 700, 6, "bf16", True), (21, 64, 4096, 64, "bf16", False),
    (19, 64, 1000, 5, "f32", True), (2000, 256, 40, 6, "bf16", False), (515, 1024, 130, 1, "bf16", True),
])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s[0]}-{'renorm' if s[1] else 'plain'}")
def test_router_backward_matches_oracle(T, d, N, k, dt, add, spec):
    print(f"[router_backward] T={T} d={d} N={N} k={k} {dt} add={add} {spec}", flush=True)
    check_router_backward(T, d, N, k, dt, spec, add, T + d + N)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_router_backward_odd_picks_and_aliased_dx(spec, dt):
    """Padded picks, ids listed twice, masked rows; dx_add is dx itself; one
    expert takes most rows."""
    rng = np.random.default_rng(9)
    T, N, k = 90, 24, 4
    ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    ids[0] = [5, -1, N, 9]
    ids[1] = [4, 4, 8, 4]
    ids[2] = [-1, -2, N + 5, 2 ** 31 - 1]
    ids[10:70, 0] = 3
    l = rng.normal(0, 1, (T, N))
    l[3] = -np.inf
    l[4, ::2] = -np.inf
    check_router_backward(T, 128, N, k, dt, spec, True, 5, ids=ids, l=l, alias=True)


def test_router_backward_same_bits_each_run():
    T, d, N, k = 3000, 512, 64, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, d, generator=g, device="cuda").bfloat16()
    l = torch.randn(T, N, generator=g, device="cuda")
    ids, _ = bmoe.route_logits(l, k)
    dg = torch.randn(T, k, generator=g, device="cuda")
    for spec in SPECS:
        sp = bmoe.RouteSpec(spec[0], renorm=spec[1])
        a = bmoe.router_backward(x, w, l, ids, dg, sp)
        b = bmoe.router_backward(x, w, l, ids, dg, sp)
        assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])


def test_router_backward_padded_rows_do_not_spread():
    """A padded token (ids -1) may hold anything, NaN and infinities included:
    it changes neither dW nor other rows, and its own dx is dx_add."""
    T, d, N, k = 300, 512, 16, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    w = torch.randn(N, d, generator=g, device="cuda").bfloat16()
    l = torch.randn(T, N, generator=g, device="cuda")
    ids, _ = bmoe.route_logits(l, k)
    dg = torch.randn(T, k, generator=g, device="cuda")
    add = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    pad = torch.arange(T, device="cuda") % 7 == 3
    for dt in (torch.bfloat16, torch.float32):
        xs, ws, adds = x.to(dt), w.to(dt), add.to(dt)
        ids2, xz, xn = ids.clone(), xs.clone(), xs.clone()
        ids2[pad] = -1
        xz[pad] = 0
        xn[pad] = float("nan")
        for spec in (("softmax", True), ("sigmoid", False), ("sigmoid", True)):
            sp = bmoe.RouteSpec(spec[0], renorm=spec[1])
            a = bmoe.router_backward(xz, ws, l, ids2, dg, sp, dx_add=adds)
            b = bmoe.router_backward(xn, ws, l, ids2, dg, sp, dx_add=adds)
            assert torch.equal(a["dw"], b["dw"]) and torch.equal(a["dx"], b["dx"])
            assert torch.equal(a["dx"][pad], adds[pad])


@pytest.mark.parametrize("spec", [("sigmoid", True), ("softmax", False)], ids=str)
def test_router_backward_captured_and_replayed(spec):
    T, d, N, k = 700, 256, 32, 2
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, d, device="cuda").bfloat16()
    w = torch.randn(N, d, generator=g, device="cuda").bfloat16()
    l = torch.randn(T, N, device="cuda")
    dg = torch.randn(T, k, device="cuda")
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1])

    def step():
        ids, _ = bmoe.route_logits(l, k, sp)
        return bmoe.router_backward(x, w, l, ids, dg, sp, dx_add=x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for t in (x, l, dg):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        assert torch.equal(out["dx"], ref["dx"]) and torch.equal(out["dw"], ref["dw"]), i


@pytest.mark.parametrize("spec", [("sigmoid", True), ("softmax", False)], ids=str)
def test_router_backward_more_values_than_32_bits_count(spec):
    """x with more than 2^31 values; only a few far rows have a gradient, so dW
    is theirs alone, and the other rows' dx is dx_add."""
    d, N, k = 2048, 8, 2
    T = 2 ** 31 // d + 3000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w_dev, w = rounded(np.random.default_rng(1).normal(0, 1, (N, d)) / math.sqrt(d), "bf16")
    l_dev, _ = rounded(np.zeros((1, N)), "f32")
    l_dev = torch.randn(T, N, generator=g, device="cuda")
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1])
    ids, _ = bmoe.route_logits(l_dev, k, sp)
    rows = torch.tensor([0, 5, 2 ** 31 // d - 1, 2 ** 31 // d, 2 ** 31 // d + 1, T - 1],
                        device="cuda")
    dg = torch.zeros(T, k, device="cuda")
    dg[rows] = torch.randn(len(rows), k, generator=g, device="cuda")
    print(f"[router_backward] T={T} d={d} {spec}", flush=True)
    out = bmoe.router_backward(x, w_dev, l_dev, ids, dg, sp, dx_add=x)
    l = l_dev[rows].double().cpu().numpy()
    xr, idn, dgn = x[rows].double().cpu().numpy(), ids[rows].cpu().numpy(), dg[rows].cpu().numpy()
    ref = O.router_backward(xr, w, l, idn, dgn, dx_add=xr, score=spec[0], renorm=spec[1])
    A = grad_scale(l, idn, dgn, *spec, 1.0)
    sx = np.abs(xr) * (N + 1) * U + ((4 * eps_of(l) + (N + 2) * U) * A) @ np.abs(w)
    err = np.abs(out["dx"][rows].double().cpu().numpy() - ref["dx"])
    assert (err <= sx + HALF["bf16"] * (np.abs(ref["dx"]) + sx)).all()
    sw = ((4 * eps_of(l) + (len(rows) + 2) * U) * A).T @ np.abs(xr)
    assert (np.abs(out["dw"].double().cpu().numpy() - ref["dw"]) <= sw + 2.0 ** -126).all()
    out["dx"][rows] = x[rows]
    assert torch.equal(out["dx"], x)


def test_norm_of_more_values_than_32_bits_count():
    n = 2 ** 31 + 12345
    t = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    t.fill_(0.5)
    t[-1] = 1024.0
    ref = math.sqrt(0.25 * (n - 1) + 1024.0 ** 2)
    assert abs(float(bmoe.grad_norm([t[3:], t[:3].clone()])) - ref) <= (U + 2.0 ** -40) * ref
    half = float(np.float32(ref / 2))
    bmoe.clip_grads([t], half)   # a factor of 1/2 to within three roundings of fp32
    assert t[0] == 0.25 and t[n // 2] == 0.25 and t[2 ** 31] == 0.25 and t[-1] == 512.0


# ---- gradient lists --------------------------------------------------------------

def make_list(sizes, rng, scale=1.0, offset=0):
    """Tensors (alternating fp32 and bf16) cut from buffers `offset` entries
    past an aligned start, with guard entries around; (tensors, buffers)."""
    ts, bufs = [], []
    for i, n in enumerate(sizes):
        dt = torch.bfloat16 if i % 2 else torch.float32
        buf = torch.full((n + offset + 16,), -7.0, dtype=dt, device="cuda")
        t = buf[offset:offset + n]
        t.copy_(torch.from_numpy((rng.normal(0, scale, n)).astype(np.float32)))
        ts.append(t)
        bufs.append(buf)
    return ts, bufs


def fp64(ts):
    return [t.double().cpu().numpy() for t in ts]


def guards_kept(ts, bufs, offset):
    return all((b[:offset] == -7).all() and (b[offset + t.numel():] == -7).all()
               for t, b in zip(ts, bufs))


SIZES = [[1], [3, 1, 2], [0, 5, 0, 17], [1000, 4097, 64], [70001, 1, 333, 8, 262147],
         [int(v) for v in np.random.default_rng(1).integers(0, 400, 260)]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("offset", [0, 1, 3, 6])
@pytest.mark.parametrize("factor", [0.3, 1.7])
def test_clip_in_place_and_apart(sizes, offset, factor):
    """factor: max_norm over the norm. The norm's squares are exact products
    summed in 64 bits, so it is off by its one rounding to fp32 (and 2^-40 for
    the sums); a scaled entry by the factor's two roundings (norm, quotient),
    the product's and the type's."""
    rng = np.random.default_rng(len(sizes) + offset)
    ts, bufs = make_list(sizes, rng, offset=offset)
    before = [t.clone() for t in ts]
    ref = O.grad_norm(fp64(ts))
    max_norm = float(np.float32(factor * ref))
    print(f"[clip] {len(sizes)} tensors, offset {offset}, factor {factor}", flush=True)
    only = bmoe.grad_norm(ts)
    apart, abufs = make_list(sizes, rng, offset=(offset + 2) % 7)
    n1 = bmoe.clip_grads(ts, max_norm, out=apart)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    n2 = bmoe.clip_grads(ts, max_norm)
    assert torch.equal(only, n1) and torch.equal(only, n2)
    assert abs(float(only) - ref) <= (U + 2.0 ** -40) * ref
    assert guards_kept(ts, bufs, offset) and guards_kept(apart, abufs, (offset + 2) % 7)
    want, _ = O.clip_grads(fp64(before), max_norm)
    for a, b, w in zip(ts, apart, want):
        assert torch.equal(a, b)
        half = HALF["bf16" if a.dtype == torch.bfloat16 else "f32"]
        assert (np.abs(a.double().cpu().numpy() - w) <= (3.1 * U + half) * np.abs(w) + 2.0 ** -126).all()
    if factor > 1:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    # scaling by a norm at hand is the same as clipping
    again = [t.clone() for t in before]
    bmoe.scale_grads(again, only, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(again, ts))


def test_norm_neither_overflows_nor_vanishes():
    big = torch.full((5000,), 1e30, device="cuda")
    assert float(bmoe.grad_norm([big])) == pytest.approx(1e30 * math.sqrt(5000), rel=1e-6)
    tiny = torch.full((5000,), 1e-30, device="cuda")
    assert float(bmoe.grad_norm([tiny])) == pytest.approx(1e-30 * math.sqrt(5000), rel=1e-6)
    mixed = [torch.full((100003,), 1e-3, device="cuda"), torch.tensor([1e4], device="cuda")]
    assert float(bmoe.grad_norm(mixed)) == pytest.approx(math.sqrt(1e8 + 0.100003), rel=1e-7)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_norm_that_is_not_finite_clips_nothing(bad):
    a = torch.randn(3000, device="cuda")
    b = torch.randn(500, device="cuda").bfloat16()
    b[77] = bad
    keep = [a.clone(), b.clone()]
    out = [torch.zeros_like(a), torch.zeros_like(b)]
    n = bmoe.clip_grads([a, b], 1.0, out=out)
    assert (math.isnan(float(n)) if math.isnan(bad) else float(n) == math.inf)
    bmoe.clip_grads([a, b], 1.0)
    for u, v, w in zip([a, b], keep, out):
        assert torch.equal(u.nan_to_num(3.0), v.nan_to_num(3.0))
        assert torch.equal(w.nan_to_num(3.0), v.nan_to_num(3.0))
    # finite entries whose norm passes fp32: also left as they are
    huge = torch.full((9,), 3e38, device="cuda")
    assert float(bmoe.clip_grads([huge], 1.0)) == math.inf and (huge == 3e38).all()


def test_clip_edges():
    z = torch.zeros(100, device="cuda")
    assert float(bmoe.clip_grads([z], 1.0)) == 0.0 and (z == 0).all()
    e = torch.empty(0, device="cuda")
    assert float(bmoe.grad_norm([e])) == 0.0
    a = torch.tensor([3.0, 4.0], device="cuda")
    assert float(bmoe.clip_grads([a], math.inf)) == 5.0 and a.tolist() == [3.0, 4.0]
    assert float(bmoe.clip_grads([a], 5.0)) == 5.0 and a.tolist() == [3.0, 4.0]
    bmoe.clip_grads([a.view(2, 1), e], 2.5)
    assert a.tolist() == [1.5, 2.0]
    with pytest.raises(bmoe.BmoeError):
        bmoe.clip_grads([a, a], 1.0)
    with pytest.raises(bmoe.BmoeError):
        bmoe.clip_grads([a], 0.0)
    with pytest.raises(ValueError):
        bmoe.clip_grads([a], 1.0, out=[])
    with pytest.raises(ValueError):
        bmoe.clip_grads([a, torch.zeros(2)], 1.0)


def test_clip_captured_and_replayed():
    g0 = torch.Generator(device="cuda").manual_seed(5)
    ts = [torch.zeros(n, device="cuda") for n in (70001, 5, 4096)]
    out = [torch.zeros_like(t) for t in ts]
    bmoe.clip_grads(ts, 1.0, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = bmoe.clip_grads(ts, 1.0, out=out)
    for i in range(4):
        for t in ts:
            t.copy_(torch.randn(t.shape, generator=g0, device="cuda") * (0.001 if i == 2 else 1.0))
        graph.replay()
        torch.cuda.synchronize()
        ref = [torch.zeros_like(t) for t in ts]
        n2 = bmoe.clip_grads(ts, 1.0, out=ref)
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, ref)), i


# ---- one training step -------------------------------------------------------------

@pytest.mark.parametrize("name,T", [("d512_e64_top2_bf16", 300), ("tiny_d64_e8_top2_f32", 200)])
def test_training_step_end_to_end(name, T):
    """logits -> ids, gates -> layer -> gradients of the layer -> gradients of
    the router on top -> loads and bias -> clipped gradients, each stage held
    to the oracle run on that stage's own inputs."""
    inp = W.make_inputs(name, T=T)
    rw = W.make_router_weights(inp)
    dev = to_device(inp)
    N, k, dt = inp.N, inp.k, inp.dtype
    wr = (torch.from_numpy(rw.w_bits.view(np.int16)).view(torch.bfloat16) if dt == "bf16"
          else torch.from_numpy(rw.w)).cuda()
    spec = bmoe.RouteSpec("sigmoid", n_groups=4, topk_groups=2, scale=1.5)
    kw = dict(score="sigmoid", renorm=True, scale=1.5)
    bias = torch.zeros(N, device="cuda")
    load = torch.empty(N, dtype=torch.int32, device="cuda")

    logits = bmoe.router_logits(dev["x"], wr)
    ids, gates = bmoe.route_logits(logits, k, spec, bias=bias)
    y, kept = bmoe.forward_keep(dev["x"], ids, gates, dev["theta"], dev["phi"], dev["w_packed"],
                                dev["alpha"])
    dy = torch.randn(y.shape, generator=torch.Generator("cuda").manual_seed(1),
                     device="cuda").to(y.dtype)
    g = bmoe.backward_kept(dev["x"], gates, N, dev["w_packed"], dev["alpha"], dy, kept)
    layer_dx = g["dx"].clone()
    r = bmoe.router_backward(dev["x"], wr, logits, ids, g["dgates"], spec, dx_add=g["dx"],
                             dx=g["dx"])
    bmoe.route_balance(ids, load, bias=bias, rate=1e-3)
    grads = [g["dtheta"], g["dphi"], g["dw"], r["dw"]]
    before = fp64(grads)
    norm = bmoe.clip_grads(grads, 0.5)
    torch.cuda.synchronize()

    l64 = logits.double().cpu().numpy()
    oid, og = O.route_logits(l64, k, n_groups=4, topk_groups=2, bias=np.zeros(N, np.float32), **kw)
    idn = ids.cpu().numpy()
    assert np.array_equal(idn, oid)
    assert np.allclose(gates.cpu().numpy(), og, rtol=float(eps_of(l64).max()), atol=0)
    ref = O.router_backward(inp.x, rw.w, l64, idn, g["dgates"].cpu().numpy(),
                            dx_add=layer_dx.double().cpu().numpy(), **kw)
    A = grad_scale(l64, idn, g["dgates"].cpu().numpy(), "sigmoid", True, 1.5)
    sx = (4 * eps_of(l64) + (N + 2) * U) * A @ np.abs(rw.w.astype(np.float64))
    sx = sx + (N + 1) * U * np.abs(layer_dx.double().cpu().numpy())
    err = np.abs(r["dx"].double().cpu().numpy() - ref["dx"])
    assert (err <= sx + HALF[dt] * (np.abs(ref["dx"]) + sx)).all()
    rl, rb = O.route_balance(idn, N, bias=np.zeros(N), rate=1e-3)
    assert np.array_equal(load.cpu().numpy(), rl)
    assert np.allclose(bias.cpu().numpy(), rb, rtol=U, atol=0)
    want, rn = O.clip_grads(before, 0.5)
    assert abs(float(norm) - rn) <= 1.01 * U * rn and rn > 0.5
    for a, w in zip(grads, want):
        assert (np.abs(a.double().cpu().numpy() - w) <= 4.2 * U * np.abs(w) + 2.0 ** -126).all()
    assert abs(O.grad_norm(fp64(grads)) - 0.5) <= 0.5 * 4.2 * U
