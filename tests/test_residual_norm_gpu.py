"""Norms around a block on the GPU against the fp64 oracle.

Tolerances, per entry: one rounding of the result to its type (half a step) and
for values that go through fp32 sums of n terms, n + 16 roundings of 2^-24 of
the largest magnitude that enters the row (the chain of a row is two sums over
d, one over k, and a dozen single operations; each moves the row's values by
its relative error)."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle.bmoe_block import _picked
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def cuda(t):
    return None if t is None else t.cuda()


def half(dt):
    return 2.0 ** -8 if dt == BF else 2.0 ** -24


def close(got, ref, n, dt, scale=None, what=""):
    """scale: magnitude that fp32 roundings are relative to (default: a row's
    largest value)."""
    if scale is None:
        scale = np.abs(ref).max(axis=-1, keepdims=True)
    err = np.abs(f64(got) - ref)
    tol = half(dt) * np.abs(ref) + 2.0 ** -24 * (n + 16) * scale
    assert (err <= tol).all(), (what, float((err - tol).max()), float(err.max()))


def draw(T, d, k, dt, seed=0, routed=True, gates=True, post=True, pre=True, pad=0.0, extra=0):
    g = torch.Generator().manual_seed(seed)
    s = dict(u=torch.randn(T * k + extra, d, generator=g).to(dt), r=(2 * torch.randn(T, d, generator=g)).to(dt),
             inv=None, gates=None, w_post=None, w_pre=None, dr_out=torch.randn(T, d, generator=g).to(dt),
             dn=None, k=k)
    if routed:
        s["inv"] = torch.randperm(T * k + extra, generator=g)[:T * k].int()
        if pad:
            s["inv"][torch.rand(T * k, generator=g) < pad] = -1
    if gates:
        s["gates"] = torch.softmax(torch.randn(T, k, generator=g), 1)
    if post:
        s["w_post"] = 1 + 0.1 * torch.randn(d, generator=g)
    if pre:
        s["w_pre"] = 1 + 0.1 * torch.randn(d, generator=g)
        s["dn"] = torch.randn(T, d, generator=g).to(dt)
    return s


SCALES = dict(eps=1e-6, res_scale=0.75, out_scale=1.25)


def check(s, dt, forward=True, backward=True):
    k, T, d = s["k"], s["r"].shape[0], s["r"].shape[1]
    kw = dict(k=k, inv=f64(s["inv"]), gates=f64(s["gates"]), w_post=f64(s["w_post"]),
              w_pre=f64(s["w_pre"]), **SCALES)
    dk = dict(k=k, inv=cuda(s["inv"]), gates=cuda(s["gates"]), w_post=cuda(s["w_post"]),
              w_pre=cuda(s["w_pre"]))
    spec = bmoe.NormSpec(**SCALES)
    if forward:
        r_out, n = bmoe.residual_norm(s["u"].cuda(), s["r"].cuda(), spec, **dk)
        rr, rn = O.residual_norm(f64(s["u"]), f64(s["r"]), **kw)
        close(r_out, rr, 2 * d + k, dt, what="r")
        if n is None:
            assert rn is None
        else:
            close(n, rn, 4 * d + k, dt, what="n")
    if not backward:
        return
    du = torch.full(s["u"].shape, 7.0, dtype=dt, device="cuda")
    args = (s["u"].cuda(), s["r"].cuda(), spec)
    extra = dict(dr_out=cuda(s["dr_out"]), dn=cuda(s["dn"]), **dk)
    g = bmoe.residual_norm_backward(*args, du=du, **extra)
    ref = O.residual_norm_backward(f64(s["u"]), f64(s["r"]), dr_out=f64(s["dr_out"]),
                                   dn=f64(s["dn"]), **kw)
    scale_dr, scale_dy = scales(s, kw)
    close(g["dr"], ref["dr"], 4 * d, dt, scale=SCALES["res_scale"] * scale_dr, what="dr")
    rows, ok, at = _picked(f64(s["u"]), kw["inv"], T, k)
    gate = np.ones((T, k)) if s["gates"] is None else kw["gates"]
    for j in range(k):
        named = ok[:, j]
        close(g["du"][torch.from_numpy(at[named, j]).cuda()], ref["du"][at[named, j]], 8 * d + k, dt,
              scale=gate[named, j:j + 1] * scale_dy[named], what="du")
    unnamed = np.setdiff1d(np.arange(s["u"].shape[0]), at[ok])
    assert (g["du"].cpu()[torch.from_numpy(unnamed)] == 7.0).all()
    # sums over tokens (or over d) of products of an error-bearing row
    if s["gates"] is None:
        assert g["dgates"] is None
    else:
        mag = scale_dy * np.abs(rows).sum(2)
        close(g["dgates"], ref["dgates"], 8 * d + k, F32, scale=mag, what="dgates")
    for name, w in (("dw_pre", s["w_pre"]), ("dw_post", s["w_post"])):
        if w is None:
            assert g[name] is None
            continue
        top = np.abs(f64(s["dn"])).max(1) if name == "dw_pre" else SCALES["out_scale"] * scale_dr[:, 0]
        close(g[name], ref[name], 8 * d + T, F32, scale=top.sum() * HIGH, what=name)
    again = bmoe.residual_norm_backward(*args, **extra)
    for name in ("dr", "dgates", "dw_pre", "dw_post"):
        assert g[name] is None or torch.equal(g[name], again[name]), name


HIGH = 6.0  # no normalised value here is larger (normal draws; at most sqrt(d) in any row)


def scales(s, kw):
    """Magnitudes [T][1] of the terms that dr and dy are differences of:
    D(v, w, t) = q (w t - v q^2 mean(w t v)) may cancel, wholly so for d = 1, and
    its roundings are relative to q w t and to that times the normalised value."""
    def of(v, w, t):
        q = 1 / np.sqrt(np.mean(v ** 2, axis=1, keepdims=True) + SCALES["eps"])
        return q * np.abs(w).max() * t * (1 + HIGH)
    dr = np.abs(f64(s["dr_out"])).max(1, keepdims=True)
    if s["w_pre"] is not None:
        dr = dr + of(f64(s["r"]), kw["w_pre"], np.abs(f64(s["dn"])).max(1, keepdims=True))
    dy = SCALES["out_scale"] * dr
    if s["w_post"] is not None:
        y, _ = O.residual_norm(f64(s["u"]), None, k=s["k"], inv=kw["inv"], gates=kw["gates"],
                               T=s["r"].shape[0])
        dy = of(y, kw["w_post"], dy)
    return dr, dy


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d,k", [(1, 1, 1), (1, 4096, 8), (3, 7, 2), (5, 64, 1), (4, 500, 3),
                                   (9, 512, 2), (6, 513, 2), (130, 1000, 4), (33, 1024, 1),
                                   (17, 1025, 2), (20, 2048, 4), (7, 2055, 2), (5, 4095, 1),
                                   (6, 4096, 2), (4, 5000, 2), (3, 8191, 1), (5, 8192, 3),
                                   (2600, 48, 2), (1300, 520, 1)])
def test_widths(T, d, k, dt):
    check(draw(T, d, k, dt, seed=d + T, routed=k > 1, gates=k > 1, extra=3 if k > 1 else 0), dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("routed", [0, 1])
@pytest.mark.parametrize("gates,post,pre", [(0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 1), (0, 0, 0),
                                            (1, 0, 0)])
def test_parts_left_out(routed, gates, post, pre, dt):
    for d in (96, 2048):
        check(draw(21, d, 3, dt, seed=d, routed=routed, gates=gates, post=post, pre=pre), dt)


@pytest.mark.parametrize("dt", [BF, F32])
def test_padded_picks(dt):
    s = draw(40, 256, 4, dt, seed=3, pad=0.4, extra=9)
    s["inv"][:4] = -1                  # a token without any pick
    s["inv"][7] = 40 * 4 + 9           # behind u
    s["u"][~torch.isin(torch.arange(169), s["inv"])] = float("nan")   # rows of no pick
    s["u"] = s["u"].clone()
    check({**s, "u": torch.nan_to_num(s["u"])}, dt)
    # NaN in rows that nobody names goes nowhere
    spec = bmoe.NormSpec(**SCALES)
    kw = dict(k=4, inv=s["inv"].cuda(), gates=s["gates"].cuda(), w_post=s["w_post"].cuda(),
              w_pre=s["w_pre"].cuda())
    a, n = bmoe.residual_norm(s["u"].cuda(), s["r"].cuda(), spec, **kw)
    assert torch.isfinite(a).all() and torch.isfinite(n).all()
    g = bmoe.residual_norm_backward(s["u"].cuda(), s["r"].cuda(), spec, dr_out=s["dr_out"].cuda(),
                                    dn=s["dn"].cuda(), du=torch.zeros_like(s["u"]).cuda(), **kw)
    assert all(torch.isfinite(v).all() for v in g.values())
    assert (g["dgates"].view(-1)[s["inv"].cuda() < 0] == 0).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d", [40, 1000, 4096])
def test_without_a_block(dt, d):
    s = draw(11, d, 1, dt, seed=d, routed=0, gates=0, post=0)
    spec = bmoe.NormSpec(**SCALES)
    a, n = bmoe.residual_norm(None, s["r"].cuda(), spec, w_pre=s["w_pre"].cuda())
    ra, rn = O.residual_norm(None, f64(s["r"]), w_pre=f64(s["w_pre"]), **SCALES)
    close(a, ra, 1, dt)
    close(n, rn, 4 * d, dt)
    g = bmoe.residual_norm_backward(None, s["r"].cuda(), spec, w_pre=s["w_pre"].cuda(),
                                    dn=s["dn"].cuda())
    ref = O.residual_norm_backward(None, f64(s["r"]), w_pre=f64(s["w_pre"]), dn=f64(s["dn"]), **SCALES)
    close(g["dr"], ref["dr"], 4 * d, dt)
    assert g["du"] is None and g["dgates"] is None and g["dw_post"] is None


def test_no_residual_sums_a_tokens_rows():
    s = draw(50, 264, 3, BF, seed=4)
    a, n = bmoe.residual_norm(s["u"].cuda(), None, k=3, inv=s["inv"].cuda())
    ref, _ = O.residual_norm(f64(s["u"]), None, k=3, inv=f64(s["inv"]), T=50)
    assert n is None
    close(a, ref, 3, BF, scale=8.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_in_place_residual(dt):
    s = draw(30, 776, 2, dt, seed=5)
    kw = dict(k=2, inv=s["inv"].cuda(), gates=s["gates"].cuda(), w_post=s["w_post"].cuda(),
              w_pre=s["w_pre"].cuda())
    a, n = bmoe.residual_norm(s["u"].cuda(), s["r"].cuda(), **kw)
    r = s["r"].cuda()
    a2, n2 = bmoe.residual_norm(s["u"].cuda(), r, r_out=r, **kw)
    assert a2 is r and torch.equal(a, a2) and torch.equal(n, n2)
    dr = s["dr_out"].cuda()
    g = bmoe.residual_norm_backward(s["u"].cuda(), a, dr_out=s["dr_out"].cuda(), dn=s["dn"].cuda(), **kw)
    h = bmoe.residual_norm_backward(s["u"].cuda(), a, dr_out=dr, dr=dr, dn=s["dn"].cuda(), **kw)
    assert h["dr"] is dr and torch.equal(g["dr"], dr) and torch.equal(g["dw_pre"], h["dw_pre"])


def test_no_tokens():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    a, n = bmoe.residual_norm(e, e, w_post=w, w_pre=w)
    assert a.shape == n.shape == (0, 64)
    g = bmoe.residual_norm_backward(e, e, w_post=w, w_pre=w, dr_out=e, dn=e)
    assert not g["dw_post"].any() and not g["dw_pre"].any()


def test_zero_rows_and_infinities():
    """Zero rows norm to zero; an infinity or a NaN stays in its own token."""
    s = draw(6, 300, 1, F32, seed=6, routed=0, gates=0)
    s["u"][1] = 0
    s["r"][1] = 0
    s["r"][3, 7] = float("inf")
    s["u"][4, 0] = float("nan")
    kw = dict(w_post=s["w_post"].cuda(), w_pre=s["w_pre"].cuda())
    a, n = bmoe.residual_norm(s["u"].cuda(), s["r"].cuda(), **kw)
    assert not a[1].any() and not n[1].any() and a[4].isnan().all() and n[3, 7].isnan()
    good = [0, 1, 2, 5]
    assert torch.isfinite(a[good]).all() and torch.isfinite(n[good]).all()


# Rows of sixteen lanes, several to a wave (picks in up to four registers), and rows
# that end inside 16 bytes
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d", [2, 3, 5, 8, 9, 15, 20, 61, 64, 66, 100, 127, 128, 129])
@pytest.mark.parametrize("T,k", [(1, 1), (37, 2), (50, 17), (21, 64), (530, 3)])
def test_narrow_rows(T, k, d, dt):
    s = draw(T, d, k, dt, seed=d + k, routed=k > 1, gates=k > 1, pad=0.2 if k > 1 else 0.0,
             extra=5 if k > 1 else 0)
    check(s, dt)
