"""The routing gradient of rows with values that no gate depends on: they may
hold anything."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe
from test_route_gpu import SPECS, U, eps_of, grad_scale, rounded

pytestmark = pytest.mark.gpu


def gradient(l_dev, ids, dg, spec):
    """(dlogits by the gradient alone, the same through the router's backward):
    with W_r the unit matrix, dx is dl."""
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1], scale=1.5)
    i, d = torch.from_numpy(ids).cuda(), torch.from_numpy(dg).cuda()
    T, N = l_dev.shape
    dl = bmoe.route_logits_backward(l_dev, i, d, sp)
    eye = torch.eye(N, device="cuda")
    r = bmoe.router_backward(torch.ones(T, N, device="cuda"), eye, l_dev, i, d, sp)
    b = bmoe.router_backward(torch.ones(T, N, device="cuda").bfloat16(), eye.bfloat16(), l_dev, i,
                             d, sp)
    return dl.double().cpu().numpy(), r["dx"].double().cpu().numpy(), b["dx"].double().cpu().numpy()


def check(l, ids, dg, spec):
    """Against the oracle: dl to 4 EPS of its terms' magnitudes, dx in fp32 to N
    additions more, in bf16 to its half step more."""
    l_dev, l = rounded(l, "f32")
    with np.errstate(all="ignore"):
        ref = O.route_logits_backward(l, ids, dg, score=spec[0], renorm=spec[1], scale=1.5)
    fine = np.where(np.isfinite(dg), dg, 0).astype(np.float32)
    tol = 4 * eps_of(l) * grad_scale(l, ids, fine, *spec, 1.5)
    got = gradient(l_dev, ids, dg, spec)
    for g, more in zip(got, (0.0, l.shape[1] * U, l.shape[1] * U + 2.0 ** -8)):
        ok = ~np.isnan(ref)
        assert (np.isnan(g) != ok).all()
        bound = (1 + more) * tol + more * np.abs(ref) + 2.0 ** -126
        assert (np.abs(g - ref)[ok] <= bound[ok]).all()
    return ref


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_gradient_of_a_masked_pick_does_not_spread(spec, bad):
    """The gate of a masked expert is 0 whatever the logits, so what arrives as
    its gradient moves nothing."""
    rng = np.random.default_rng(1)
    T, N, k = 40, 16, 4
    l = rng.normal(0, 1, (T, N))
    ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    for t in range(T):       # 0 to 4 masked picks a row
        for j in range(t % 5):
            l[t, ids[t, j]] = -math.inf
            dg[t, j] = bad
    ref = check(l, ids, dg, spec)
    assert np.isfinite(ref).all() and (ref[4::5] == 0).all() and (ref[1::5] != 0).any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_gradient_through_a_pick_that_is_not_a_number(spec, bad):
    """A NaN among a token's picked logits (softmax: or an infinity) makes its
    gates NaN, and their gradient too, not 0: the picks' where they are
    renormalised, the row's for the full softmax, the pick's alone for plain
    sigmoids. Other rows keep theirs. A sigmoid of +inf is 1, its slope 0."""
    rng = np.random.default_rng(2)
    T, N, k = 30, 16, 3
    l = rng.normal(0, 1, (T, N))
    ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    l[np.arange(0, T, 3), ids[::3, 1]] = bad
    l_dev, _ = rounded(l, "f32")
    is_nan = np.zeros((T, N), dtype=bool)
    if spec[0] == "softmax" or math.isnan(bad):
        if not spec[1]:
            if spec[0] == "softmax":
                is_nan[::3] = True
            else:
                is_nan[np.arange(0, T, 3), ids[::3, 1]] = True
        else:
            np.put_along_axis(is_nan[::3], ids[::3].astype(np.int64), True, axis=1)
    got, *dx = gradient(l_dev, ids, dg, spec)
    assert (np.isnan(got) == is_nan).all()
    for v in dx:
        assert (np.isnan(v).all(axis=1) == is_nan.any(axis=1)).all()
    with np.errstate(all="ignore"):
        ref = O.route_logits_backward(l, ids, dg, score=spec[0], renorm=spec[1], scale=1.5)
    rows = np.arange(T) % 3 != 0
    tol = 4 * eps_of(l[rows]) * grad_scale(l[rows], ids[rows], dg[rows], *spec, 1.5) + 2.0 ** -126
    assert (np.abs(got - ref)[rows] <= tol).all()
    assert (np.isnan(ref) == is_nan).all()


@pytest.mark.parametrize("N", [16, 64, 512, 2048])
@pytest.mark.parametrize("spec", SPECS, ids=str)
def test_gradient_of_padded_rows_whatever_they_hold(spec, N):
    """Rows all of whose picks are padded (or masked) have no gradient, also
    where their logits and dgates are NaN or infinite, and change no other's."""
    rng = np.random.default_rng(N)
    T, k = 60, 4
    l = rng.normal(0, 1, (T, N))
    ids = np.argsort(rng.random((T, N)), axis=1)[:, :k].astype(np.int32)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    pad = np.arange(T) % 3 == 1
    ids[pad] = [-1, N, -7, 2 ** 31 - 1]
    clean = gradient(rounded(l, "f32")[0], ids, dg, spec)
    l[pad] = rng.choice([math.nan, math.inf, -math.inf, 0.0], (pad.sum(), N))
    dg[pad] = rng.choice([math.nan, math.inf, 1.0], (pad.sum(), k))
    l[4, :4] = -math.inf
    ids[4] = [0, 2, -1, 3]     # masked ones count as none
    got = gradient(rounded(l, "f32")[0], ids, dg, spec)
    for a, b in zip(got, clean):
        assert (a[pad] == 0).all() and (a[~pad] == b[~pad]).all()
