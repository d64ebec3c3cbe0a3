"""GPU parity of routing from logits, its gradient and the balance bias with
the fp64 oracle.

The ids have to be the oracle's, near ties included. Tolerances, with
u = 2^-24 and D the largest distance of a row's logits from the shift the
scores take (and from 0 for the sigmoid): an exponential of argument v carries
|v| u from the argument's rounding twice (the difference, its product with
log2 e) and two more units; a sum of n <= 4096 positive terms over lanes adds
at most 64 + 6 units; divisions, the scale and the last rounding a few. So a
score or a gate is off by at most EPS = u (2 D + 96), relative. A gradient is a
product of such factors p with a difference (u_j - sum u_i p_i): 4 EPS of the
same expression with every term taken by its magnitude."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SPECS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


def rounded(a, dt):
    """(device tensor, the exact values as fp64)."""
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(
        torch.bfloat16 if dt == "bf16" else torch.float32)
    return t.cuda(), t.double().numpy()


def eps_of(l):
    f = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(all="ignore"):
        hi, lo = np.nanmax(f, axis=1, initial=-np.inf), np.nanmin(f, axis=1, initial=np.inf)
    D = np.where(np.isfinite(hi), np.maximum(hi - lo, np.maximum(abs(hi), abs(lo))), 0.0)
    return U * (2 * D + 96)[:, None]


def check_route(l_dev, l, k, spec, bias=None, kw=None):
    kw = kw or {}
    score, renorm = spec
    scale = kw.pop("scale", 1.0)
    sp = bmoe.RouteSpec(score, renorm=renorm, scale=scale, **kw)
    b_dev = None if bias is None else torch.from_numpy(bias).cuda()
    T = l.shape[0]
    # outputs in the middle of larger buffers: nothing outside is written
    ids = torch.full((T * k + 64,), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((T * k + 64,), -7.0, device="cuda")
    bmoe.route_logits(l_dev, k, sp, bias=b_dev, ids=ids[32:32 + T * k].view(T, k),
                      gates=gates[32:32 + T * k].view(T, k))
    torch.cuda.synchronize()
    for buf in (ids, gates):
        assert (buf[:32] == -7).all() and (buf[32 + T * k:] == -7).all()
    oid, og = O.route_logits(l, k, score=score, renorm=renorm, scale=scale, bias=bias, **kw)
    got = ids[32:32 + T * k].view(T, k).cpu().numpy()
    wrong = np.flatnonzero((got != oid).any(axis=1))
    assert wrong.size == 0, (wrong[:5], got[wrong[:3]], oid[wrong[:3]])
    g = gates[32:32 + T * k].view(T, k).cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(g), np.isnan(og))
    fine = ~np.isnan(og)
    # below the smallest normal fp32 the spacing is absolute
    tol = eps_of(l) * np.abs(og) + 2.0 ** -126
    assert (np.abs(g - og)[fine] <= np.broadcast_to(tol, og.shape)[fine]).all()
    return got, g


CASES = [  # T, N, k, dtype, bias, groups
    (1, 1, 1, "f32", False, None), (1, 8, 2, "f32", True, None), (5, 7, 7, "bf16", True, None),
    (1, 256, 8, "f32", True, (8, 4, "top2")), (3, 256, 8, "bf16", False, (8, 4, "top2")),
    (257, 64, 2, "f32", False, None), (63, 60, 6, "bf16", True, (5, 2, "max")),
    (100, 65, 3, "f32", True, None), (129, 250, 15, "f32", True, (10, 3, "top2")),
    (40, 256, 16, "f32", True, None), (33, 256, 33, "bf16", True, None),
    (17, 300, 9, "f32", False, (60, 30, "top2")), (9, 1000, 64, "f32", True, (8, 3, "max")),
    (6, 4096, 64, "bf16", True, (64, 9, "top2")), (7, 4095, 5, "f32", True, (63, 4, "top2")),
    (1000, 8, 2, "bf16", True, (4, 2, "top2")), (31, 12, 3, "f32", True, (12, 4, "top2")),
    (20, 64, 64, "f32", True, None), (12, 48, 6, "f32", True, (8, 1, "max")),
    (5000, 128, 4, "f32", True, (4, 2, "top2")), (70, 512, 8, "bf16", True, (16, 4, "max")),
    # more than 1024 tokens: other lanes per token; groups that end inside a lane's
    # experts, and ones that no lane layout holds
    (1500, 216, 7, "bf16", True, (8, 3, "top2")), (1100, 500, 20, "f32", True, (4, 2, "max")),
    (1300, 300, 33, "f32", True, (3, 1, "top2")), (1025, 250, 16, "bf16", False, (10, 4, "top2")),
    (5, 4092, 7, "f32", True, (33, 4, "top2")), (3, 4092, 64, "bf16", False, (44, 2, "max")),
    (1031, 17, 16, "f32", True, (1, 1, "max")),
]


@pytest.mark.parametrize("T,N,k,dt,bias,groups", CASES)
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s[0]}-{'renorm' if s[1] else 'plain'}")
def test_route_matches_oracle(T, N, k, dt, bias, groups, spec):
    rng = np.random.default_rng(T * 31 + N)
    l_dev, l = rounded(rng.normal(0, 1.5, (T, N)) + rng.normal(0, 0.5, N), dt)
    b = (rng.integers(-100, 101, N) * np.float32(1e-3)).astype(np.float32) if bias else None
    kw = dict(scale=2.5)
    if groups:
        kw.update(n_groups=groups[0], topk_groups=groups[1], group_score=groups[2])
    print(f"[route] T={T} N={N} k={k} {dt} bias={bias} {groups} {spec}", flush=True)
    check_route(l_dev, l, k, spec, b, kw)


@pytest.mark.parametrize("spec", SPECS, ids=str)
@pytest.mark.parametrize("groups", [None, (4, 2, "max"), (4, 2, "top2")], ids=str)
@pytest.mark.parametrize("bias", [False, True])
def test_route_special_rows(spec, groups, bias):
    """Masked experts, rows with nothing left, ties, the type's lowest value,
    infinities, NaN, wide logits."""
    inf, nan, low = math.inf, math.nan, float(np.finfo(np.float32).min)
    N = 16
    rows = [np.full(N, -inf), np.zeros(N), np.full(N, low), np.arange(N) * 100.0 - 900.0,
            np.where(np.arange(N) == 11, 1.0, -inf), np.where(np.arange(N) % 4 == 1, 0.5, -inf),
            np.where(np.arange(N) == 3, nan, np.arange(N) / 8.0), np.full(N, nan),
            np.where(np.arange(N) == 9, inf, 0.25), np.repeat([1.0, 2.0, 2.0, 1.0], 4),
            np.tile([1.0, 2.0, 2.0, -1.0], 4), np.full(N, -200.0) + np.arange(N) % 3,
            np.where(np.arange(N) < 13, -inf, low), np.full(N, 1e30), -np.zeros(N)]
    l_dev, l = rounded(np.stack(rows), "f32")
    b = None
    if bias:
        b = np.zeros(N, dtype=np.float32)
        b[[2, 5, 6, 13]] = [0.25, -0.5, 0.25, 0.125]
    kw = {} if groups is None else dict(n_groups=groups[0], topk_groups=groups[1],
                                        group_score=groups[2])
    got, g = check_route(l_dev, l, 6, spec, b, dict(kw))
    assert (g[0] == 0).all() and np.isnan(g[6]).all()
    assert all(len(set(r)) == 6 and (r >= 0).all() and (r < N).all() for r in got)


def test_route_bias_infinite_or_nan():
    inf, nan = math.inf, math.nan
    l_dev, l = rounded(np.random.default_rng(2).normal(0, 1, (20, 12)), "f32")
    b = np.array([0, inf, 0, -inf, nan, 0, 0, 0, -inf, 0, 0, 0], dtype=np.float32)
    for spec in SPECS:
        got, _ = check_route(l_dev, l, 12, spec, b)
        assert (got[:, 0] == 1).all() and (got[:, -1] == 4).all()
        assert (got[:, 9:11] == [3, 8]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,k", [(64, 8), (256, 8), (300, 20), (4000, 64), (64, 64)])
def test_route_near_ties_are_decided_in_64_bits(score, N, k):
    """Choices that differ by less than fp32 holds: the bias is the fp32 value
    next to what brings each score to one of a few common levels, so within a
    level the order hangs on the scores' and biases' low bits."""
    rng = np.random.default_rng(N + k)
    l_dev, l = rounded(np.repeat(rng.normal(0, 1, (1, N)), 40, axis=0), "f32")
    s = O.scores(l[:1], score)[0]
    level = 0.9 - 0.1 * rng.integers(0, 4, N)
    b = (level - s).astype(np.float32)
    c = s + b.astype(np.float64)
    assert (np.abs(np.sort(c)[1:] - np.sort(c)[:-1]) < 1e-6).mean() > 0.5
    kw = dict(n_groups=4, topk_groups=4)
    check_route(l_dev, l, k, (score, True), b, kw)
    if k <= N // 2:
        check_route(l_dev, l, k, (score, False), b, dict(n_groups=4, topk_groups=2))
        check_route(l_dev, l, k, (score, True), b, dict(n_groups=4, topk_groups=2,
                                                        group_score="max"))


@pytest.mark.parametrize("T,N,k", [(40, 64, 8), (1100, 64, 16), (40, 256, 8), (1100, 256, 8),
                                   (1100, 255, 16), (1100, 500, 20), (1100, 510, 32),
                                   (30, 66, 64)])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s[0]}-{'renorm' if s[1] else 'plain'}")
def test_route_close_logits_in_any_order(T, N, k, spec):
    """Every logit has two others one and two steps of fp32 above it, at random
    places: the scores of the three agree to fp32's last bits, or in fp32."""
    rng = np.random.default_rng(T + N + k)
    v = rng.normal(0, 1, (T, (N + 2) // 3)).astype(np.float32)
    up = np.nextafter(v, np.float32(9))
    l = np.concatenate([v, up, np.nextafter(up, np.float32(9))], axis=1)
    l = rng.permuted(l, axis=1)[:, :N]
    l_dev, l = rounded(l, "f32")
    check_route(l_dev, l, k, spec)
    check_route(l_dev, l, k, spec, np.full(N, 0.25, np.float32))
    if N % 5 == 0 and k <= N // 5 * 2:
        check_route(l_dev, l, k, spec, np.full(N, -0.5, np.float32),
                    dict(n_groups=5, topk_groups=2))


@pytest.mark.parametrize("T,N,k", [(20, 256, 12), (1100, 256, 8), (1100, 256, 16), (1100, 500, 20),
                                   (20, 1000, 16), (20, 4000, 40)])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s[0]}-{'renorm' if s[1] else 'plain'}")
def test_route_picks_from_consecutive_experts(T, N, k, spec):
    """Most picks, or all, from a run of consecutive experts, anywhere."""
    rng = np.random.default_rng(T + N + k)
    l = rng.normal(0, 1, (T, N))
    for t in range(T):
        n = int(rng.integers(4, 20))
        at = int(rng.integers(0, N - n + 1))
        l[t, at:at + n] += 4.0
    l_dev, l = rounded(l, "f32")
    check_route(l_dev, l, k, spec)
    check_route(l_dev, l, k, spec, rng.uniform(0, 0.1, N).astype(np.float32))
    if N % 4 == 0:
        check_route(l_dev, l, k, spec, rng.uniform(0, 0.1, N).astype(np.float32),
                    dict(n_groups=4, topk_groups=1))


def test_route_exact_ties_of_equal_experts():
    """Equal logits with equal biases tie exactly: the lower id goes first."""
    rng = np.random.default_rng(4)
    l_dev, l = rounded(rng.integers(-2, 3, (300, 96)) / 4.0, "bf16")
    b = (rng.integers(-1, 2, 96) / 8.0).astype(np.float32)
    for spec in SPECS:
        check_route(l_dev, l, 12, spec, b)
        check_route(l_dev, l, 12, spec, b, dict(n_groups=6, topk_groups=3))
        check_route(l_dev, l, 12, spec, None, dict(n_groups=6, topk_groups=3))


def test_route_agrees_with_the_plain_router():
    """Without bias and groups, renormalised softmax gates are bmoe_router's:
    same ids, and gates within both calls' EPS."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.normal(0, 1, (500, 64)).astype(np.float32)).cuda().bfloat16()
    w = torch.from_numpy(rng.normal(0, 0.125, (100, 64)).astype(np.float32)).cuda().bfloat16()
    ids, gates, logits = bmoe.route(x, w, 5, want_logits=True)
    assert torch.equal(bmoe.router_logits(x, w), logits)
    ids2, gates2 = bmoe.route_logits(logits, 5)
    assert torch.equal(ids, ids2)
    eps = torch.from_numpy(eps_of(logits.double().cpu().numpy())).cuda()
    assert ((gates.double() - gates2.double()).abs() <= 2 * eps * gates2.double()).all()


def test_route_empty_and_other_stream():
    ids, gates = bmoe.route_logits(torch.empty(0, 16, device="cuda"), 3)
    assert ids.shape == (0, 3) and gates.shape == (0, 3)
    l_dev, l = rounded(np.random.default_rng(1).normal(0, 1, (200, 40)), "f32")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ids, _ = bmoe.route_logits(l_dev, 4, bmoe.RouteSpec("sigmoid"), stream=s)
    s.synchronize()
    assert np.array_equal(ids.cpu().numpy(), O.route_logits(l, 4, score="sigmoid")[0])


# ---- gradient ------------------------------------------------------------------

def grad_scale(l, ids, dg, score, renorm, scale):
    """The gradient's expression with each term by its magnitude, fp64 [T][N]."""
    s = O.scores(l, score)
    T, N = l.shape
    out = np.zeros((T, N))
    rows = np.arange(T)
    ok = (ids >= 0) & (ids < N)
    idc = np.where(ok, ids, 0).astype(np.int64)
    u = np.where(ok, np.abs(scale * dg.astype(np.float64)), 0.0)
    sj = np.where(ok, np.take_along_axis(s, idc, 1), 0.0)
    p = sj
    if renorm:
        tot = sj.sum(1, keepdims=True)
        p = sj / np.where(tot > 0, tot, 1.0)
    D = (u * p).sum(1, keepdims=True)
    for j in range(ids.shape[1]):
        v = p[:, j] * (u[:, j] + D[:, 0] if renorm else u[:, j])
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                v = v / (1.0 + np.exp(l[rows, idc[:, j]]))
        out[rows, idc[:, j]] += np.where(ok[:, j], np.where(np.isfinite(v), v, 0.0), 0.0)
    if score == "softmax" and not renorm:
        out += s * D
    return out


def check_backward(l_dev, l, ids, dg, spec, scale=1.5):
    score, renorm = spec
    T, N = l.shape
    buf = torch.full((T * N + 64,), -7.0, device="cuda")
    out = buf[32:32 + T * N].view(T, N)
    bmoe.route_logits_backward(l_dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dg).cuda(),
                               bmoe.RouteSpec(score, renorm=renorm, scale=scale), dlogits=out)
    torch.cuda.synchronize()
    assert (buf[:32] == -7).all() and (buf[32 + T * N:] == -7).all()
    got = out.cpu().numpy().astype(np.float64)
    ref = O.route_logits_backward(l, ids, dg, score=score, renorm=renorm, scale=scale)
    tol = 4 * eps_of(l) * grad_scale(l, ids, dg, score, renorm, scale) + 2.0 ** -126
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    return got


@pytest.mark.parametrize("T,N,k,dt", [
    (1, 1, 1, "f32"), (1, 256, 8, "f32"), (5, 7, 7, "bf16"), (257, 64, 2, "f32"),
    (100, 65, 3, "bf16"), (33, 250, 17, "f32"), (9, 1000, 64, "f32"), (5, 4096, 64, "bf16"),
    (7, 4095, 5, "f32"), (3000, 60, 6, "f32"), (64, 2050, 4, "f32"),
])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s[0]}-{'renorm' if s[1] else 'plain'}")
def test_route_backward_matches_oracle(T, N, k, dt, spec):
    rng = np.random.default_rng(T + 7 * N)
    l_dev, l = rounded(rng.normal(0, 1.5, (T, N)), dt)
    ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    print(f"[route_backward] T={T} N={N} k={k} {dt} {spec}", flush=True)
    check_backward(l_dev, l, ids, dg, spec)


@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_route_backward_odd_picks(spec):
    """Picks outside the experts, ids listed twice, masked picks, rows with
    nothing unmasked, logits far apart."""
    N = 70
    rng = np.random.default_rng(3)
    l = rng.normal(0, 2, (8, N))
    l[1] = -np.inf
    l[2, ::2] = -np.inf
    l[3] = np.linspace(-90, 90, N)
    l[4] -= 150.0
    l_dev, l = rounded(l, "f32")
    ids = np.argsort(rng.random((8, N)), axis=1)[:, :4].astype(np.int32)
    ids[0] = [5, -1, N, 9]
    ids[5] = [4, 4, 8, 4]
    ids[6] = [-1, -2, N + 5, 2 ** 31 - 1]
    ids[2] = [0, 1, 2, 3]
    dg = rng.normal(0, 1, (8, 4)).astype(np.float32)
    got = check_backward(l_dev, l, ids, dg, spec)
    assert (got[1] == 0).all() and (got[6] == 0).all()


@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_route_backward_against_differences(spec):
    """Central differences of the library's own gates (fp32, so steps of 2^-6
    and their h^2 error of at most |f'''| h^2 / 6 <= 2^-12 for these sizes)."""
    rng = np.random.default_rng(12)
    T, N, k, h = 40, 10, 3, 2.0 ** -6
    l = np.round(rng.normal(0, 1, (T, N)) * 64) / 64
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1])
    l_dev, _ = rounded(l, "f32")
    ids, _ = bmoe.route_logits(l_dev, k, sp)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    dl = bmoe.route_logits_backward(l_dev, ids, torch.from_numpy(dg).cuda(), sp).cpu().numpy()
    idn = ids.cpu().numpy()
    for e in range(N):
        vals = []
        for sgn in (1, -1):
            m = l.copy()
            m[:, e] += sgn * h
            i2, g2 = bmoe.route_logits(rounded(m, "f32")[0], k, sp)
            vals.append((i2.cpu().numpy(), g2.cpu().numpy().astype(np.float64)))
        same = [np.array([sorted(r) for r in v[0]]) == np.sort(idn, axis=1) for v in vals]
        rows = same[0].all(1) & same[1].all(1)     # the choice did not move
        assert rows.mean() > 0.5
        f = [np.array([sum(dg[t, list(idn[t]).index(i)] * g for i, g in zip(v[0][t], v[1][t]))
                       if rows[t] else 0.0 for t in range(T)]) for v in vals]
        num = (f[0] - f[1]) / (2 * h)
        tol = np.abs(dg).sum(1) * (2.0 ** -12 + 4 * 2.0 ** -24 / h)
        assert (np.abs(num - dl[:, e])[rows] <= tol[rows]).all()


# ---- balance -------------------------------------------------------------------

@pytest.mark.parametrize("T,N,k", [(0, 8, 2), (1, 1, 1), (1, 4096, 64), (256, 8, 2), (999, 60, 6),
                                   (4096, 64, 2), (32768, 256, 8), (70001, 4096, 5),
                                   (300000, 3, 3)])
def test_balance_matches_oracle(T, N, k):
    rng = np.random.default_rng(T + N)
    ids = rng.integers(0, N, (T, k)).astype(np.int32)
    if T > 10:
        ids[rng.integers(0, T, 5), rng.integers(0, k, 5)] = [-1, N, N + 7, -2 ** 31, 2 ** 31 - 1]
        ids[: T // 3] = np.minimum(ids[: T // 3], N // 2)
    b0 = (rng.integers(-5, 6, N) * 0.25).astype(np.float32)
    idd = torch.from_numpy(ids).cuda()
    load = torch.full((N,), 77, dtype=torch.int32, device="cuda")
    bias = torch.from_numpy(b0).cuda()
    print(f"[balance] T={T} N={N} k={k}", flush=True)
    out = bmoe.route_balance(idd, load, bias=bias, rate=0.125)
    assert out is load
    rl, rb = O.route_balance(ids, N, bias=b0, rate=0.125)
    assert np.array_equal(load.cpu().numpy(), rl)
    assert np.array_equal(bias.cpu().numpy().astype(np.float64), rb)   # exact in fp32
    # a second part: the loads add up, the bias follows the sum
    bmoe.route_balance(idd[: T // 2].contiguous(), load, bias=bias, rate=0.125, accumulate=True)
    rl2, rb2 = O.route_balance(ids[: T // 2], N, load=rl, bias=rb, rate=0.125)
    assert np.array_equal(load.cpu().numpy(), rl2)
    assert np.array_equal(bias.cpu().numpy().astype(np.float64), rb2)
    # counting only
    bmoe.route_balance(idd, load)
    assert np.array_equal(load.cpu().numpy(), rl)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_logits_than_32_bits_count(dt):
    """Rows on both sides of the 2^31st logit and the last ones, of a batch with
    more logits than 32 bits count; and their gradient's."""
    N, k = 256, 3
    T = 2 ** 31 // N + 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.empty(T, N, dtype=torch.bfloat16 if dt == "bf16" else torch.float32,
                         device="cuda")
    logits.normal_(generator=g)
    sp = bmoe.RouteSpec("sigmoid", scale=1.5)
    print(f"[route] T={T} N={N} {dt}", flush=True)
    ids, gates = bmoe.route_logits(logits, k, sp)
    dg = torch.randn(T, k, generator=g, device="cuda")
    dl = bmoe.route_logits_backward(logits, ids, dg, sp)
    rows = torch.cat([torch.arange(2 ** 31 // N - 40, 2 ** 31 // N + 40),
                      torch.arange(T - 40, T)]).cuda()
    l = logits[rows].double().cpu().numpy()
    oid, og = O.route_logits(l, k, score="sigmoid", scale=1.5)
    idn = ids[rows].cpu().numpy()
    assert np.array_equal(idn, oid)
    assert (np.abs(gates[rows].double().cpu().numpy() - og) <= eps_of(l) * og).all()
    dgn = dg[rows].cpu().numpy()
    ref = O.route_logits_backward(l, idn, dgn, score="sigmoid", scale=1.5)
    tol = 4 * eps_of(l) * grad_scale(l, idn, dgn, "sigmoid", True, 1.5) + 2.0 ** -126
    assert (np.abs(dl[rows].double().cpu().numpy() - ref) <= tol).all()


def test_two_streams_at_once():
    """Independent calls on two streams, in flight together, equal the same
    calls made alone."""
    g = torch.Generator(device="cuda").manual_seed(2)
    sp = bmoe.RouteSpec("sigmoid", n_groups=4, topk_groups=2)
    ls = [torch.randn(20000, 128, generator=g, device="cuda") for _ in range(2)]
    b = torch.randn(128, generator=g, device="cuda") * 0.1
    alone = [bmoe.route_logits(l, 4, sp, bias=b) for l in ls]
    loads = [bmoe.route_balance(a[0], torch.zeros(128, dtype=torch.int32, device="cuda"))
             for a in alone]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    both = [None, None]
    # each stream's own loads: one freed here would go to the other stream
    # while its kernel still runs
    ld = [torch.empty(128, dtype=torch.int32, device="cuda") for _ in range(2)]
    for _ in range(3):
        for i, s in enumerate(ss):
            r = bmoe.route_logits(ls[i], 4, sp, bias=b, stream=s)
            bmoe.route_balance(r[0], ld[i], stream=s)
            both[i] = (*r, ld[i])
    torch.cuda.synchronize()
    for a, l, r in zip(alone, loads, both):
        assert torch.equal(a[0], r[0]) and torch.equal(a[1], r[1]) and torch.equal(l, r[2])


# ---- graphs --------------------------------------------------------------------

def test_routing_captured_and_replayed():
    """Route, its gradient and the balance step in one graph: several replays
    on changing inputs, eager work between them, each equal to the eager call."""
    g0 = torch.Generator(device="cuda").manual_seed(3)
    T, N, k = 500, 96, 4
    sp = bmoe.RouteSpec("sigmoid", n_groups=6, topk_groups=3, scale=1.5)
    logits = torch.randn(T, N, generator=g0, device="cuda")
    dg = torch.randn(T, k, generator=g0, device="cuda")
    bias = torch.zeros(N, device="cuda")
    load = torch.zeros(N, dtype=torch.int32, device="cuda")

    def step(bias, load):
        ids, gates = bmoe.route_logits(logits, k, sp, bias=bias)
        dl = bmoe.route_logits_backward(logits, ids, dg, sp)
        bmoe.route_balance(ids, load, bias=bias, rate=0.01)
        return ids, gates, dl

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(bias.clone(), load.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(bias, load)
    eb, el = torch.zeros_like(bias), torch.zeros_like(load)
    for i in range(5):
        logits.copy_(torch.randn(T, N, generator=g0, device="cuda"))
        dg.copy_(torch.randn(T, k, generator=g0, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ref = step(eb, el)
        for a, b in zip(out + (bias, load), ref + (eb, el)):
            assert torch.equal(a, b), i
