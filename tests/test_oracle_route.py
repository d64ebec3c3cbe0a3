"""Pins of the oracle of routing from logits, its gradient, the balance bias
and gradient clipping (CPU): worked values, brute force, differences, and
planted mistakes that must each fail a pin."""
import math
import os
import types

import numpy as np
import pytest

import oracle as O

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "oracle", "bmoe_route.py")
SPECS = [dict(score=s, renorm=r) for s in ("softmax", "sigmoid") for r in (True, False)]


def pin_worked(R):
    """Sigmoid scores 1/2, 3/4, 1/4, 9/10 (logits 0, ln 3, -ln 3, ln 9); a bias
    of 0.5 on expert 2 makes it the third choice's equal at 0.75 (lower id
    first), and the gates stay the scores."""
    l = np.array([[0.0, math.log(3), -math.log(3), math.log(9)]])
    ids, g = R.route_logits(l, 3, score="sigmoid", renorm=False, scale=2.0)
    assert ids.tolist() == [[3, 1, 0]] and np.allclose(g, [[1.8, 1.5, 1.0]], atol=1e-14)
    ids, g = R.route_logits(l, 2, score="sigmoid", bias=[0, 0, 1.0, 0])
    assert ids.tolist() == [[2, 3]]
    assert np.allclose(g, [[0.25 / 1.15, 0.9 / 1.15]], atol=1e-14)
    # two groups of two: largest 3/4 against 9/10; two largest 1.25 against 1.15
    ids, _ = R.route_logits(l, 2, score="sigmoid", n_groups=2, topk_groups=1, group_score="max")
    assert ids.tolist() == [[3, 2]]
    ids, _ = R.route_logits(l, 2, score="sigmoid", n_groups=2, topk_groups=1, group_score="top2")
    assert ids.tolist() == [[1, 0]]
    # softmax of (ln 1, ln 2, ln 5)
    l = np.log([[1.0, 2.0, 5.0]])
    ids, g = R.route_logits(l, 2, renorm=False)
    assert ids.tolist() == [[2, 1]] and np.allclose(g, [[5 / 8, 2 / 8]], atol=1e-14)
    ids, g = R.route_logits(l, 2, renorm=True)
    assert np.allclose(g, [[5 / 7, 2 / 7]], atol=1e-14)


def pin_ties_and_masks(R):
    inf = math.inf
    ids, g = R.route_logits([[1.0, 2.0, 2.0, 2.0]], 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(g, 0.5)
    ids, g = R.route_logits([[-inf, 1.0, -inf, -inf]], 3, bias=[9.0, 0, 0, 0])
    assert ids.tolist() == [[1, 0, 2]] and g.tolist() == [[1.0, 0.0, 0.0]]
    for spec in SPECS:
        ids, g = R.route_logits([[-inf, -inf, -inf]], 2, **spec)
        assert ids.tolist() == [[0, 1]] and g.tolist() == [[0.0, 0.0]]
        ids, g = R.route_logits([[0.0, math.nan, 3.0]], 2, **spec)
        assert ids.tolist() == [[2, 0]] and np.isnan(g).all()
    # a group with one unmasked expert counts by it alone; one with none is out
    ids, _ = R.route_logits([[2.0, -inf, 0.5, 0.5, -inf, -inf]], 1, score="sigmoid", n_groups=3,
                            topk_groups=2)
    assert ids.tolist() == [[0]]
    ids, _ = R.route_logits([[-inf, -inf, -3.0, -inf]], 2, score="sigmoid", n_groups=2,
                            topk_groups=1)
    assert ids.tolist() == [[2, 3]]
    # equal groups: the lower one
    ids, _ = R.route_logits([[1.0, 1.0, 1.0, 1.0]], 2, n_groups=2, topk_groups=1)
    assert ids.tolist() == [[0, 1]]


def pin_renormalised_gates_keep_tiny_scores(R):
    for score in ("softmax", "sigmoid"):
        _, g = R.route_logits([[-2000.0, -2000.0 - math.log(3)]], 2, score=score)
        assert np.allclose(g, [[0.75, 0.25]], atol=1e-12), score


def pin_gradient_by_differences(R):
    rng = np.random.default_rng(5)
    for spec in SPECS:
        for _ in range(4):
            l = rng.normal(0, 1.5, (3, 7))
            ids = np.stack([rng.permutation(7)[:3] for _ in range(3)]).astype(np.int32)
            dg = rng.normal(0, 1, (3, 3))

            def loss(v):
                s = R.scores(v, spec["score"])
                g = np.take_along_axis(s, ids.astype(np.int64), 1)
                if spec["renorm"]:
                    g = g / g.sum(1, keepdims=True)
                return float((1.7 * g * dg).sum())

            got = R.route_logits_backward(l, ids, dg, scale=1.7, **spec)
            h = 1e-5
            for t in range(3):
                for e in range(7):
                    a, b = l.copy(), l.copy()
                    a[t, e] += h
                    b[t, e] -= h
                    assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8, spec


def pin_gradient_edges(R):
    l = np.array([[0.3, -1.0, 0.8]])
    for spec in SPECS:
        # a pick outside the experts counts for nothing
        a = R.route_logits_backward(l, np.array([[2, -1, 7]]), np.array([[1.0, 5.0, 9.0]]), **spec)
        b = R.route_logits_backward(l, np.array([[2]]), np.array([[1.0]]), **spec)
        assert np.allclose(a, b, atol=0)
        # a row with nothing unmasked moves nothing
        z = R.route_logits_backward(np.full((1, 3), -np.inf), np.array([[0, 1]]),
                                    np.array([[1.0, 2.0]]), **spec)
        assert (z == 0).all()
    # without renorm an id listed twice adds up
    two = R.route_logits_backward(l, np.array([[1, 1]]), np.array([[1.0, 2.0]]), renorm=False)
    one = R.route_logits_backward(l, np.array([[1]]), np.array([[3.0]]), renorm=False)
    assert np.allclose(two, one, atol=1e-15)


def pin_balance(R):
    ids = np.array([[0, 1], [0, 2], [0, 1], [-1, 9]])
    load, bias = R.route_balance(ids, 4, bias=[0.0, 0.5, 0.0, 0.0], rate=0.25)
    # loads 3 2 1 0, mean 1.5
    assert load.tolist() == [3, 2, 1, 0] and bias.tolist() == [-0.25, 0.25, 0.25, 0.25]
    load, bias = R.route_balance(ids, 4, load=[0, 0, 0, 6], bias=np.zeros(4), rate=1.0)
    assert load.tolist() == [3, 2, 1, 6] and bias.tolist() == [0, 1, 1, -1]   # mean 3


def pin_router_backward_and_clip(R):
    rng = np.random.default_rng(8)
    x, w = rng.normal(size=(5, 4)), rng.normal(size=(6, 4))
    ids = np.stack([rng.permutation(6)[:2] for _ in range(5)]).astype(np.int32)
    dg, add = rng.normal(size=(5, 2)), rng.normal(size=(5, 4))

    def loss(x, w):
        s = R.scores(x @ w.T, "sigmoid")
        return float((np.take_along_axis(s, ids.astype(np.int64), 1) * dg).sum())

    got = R.router_backward(x, w, x @ w.T, ids, dg, score="sigmoid", renorm=False, dx_add=add)
    h = 1e-6
    for m, key, ref in ((x, "dx", got["dx"] - add), (w, "dw", got["dw"])):
        for i in np.ndindex(m.shape):
            v = m[i]
            m[i] = v + h
            a = loss(x, w)
            m[i] = v - h
            b = loss(x, w)
            m[i] = v
            assert abs((a - b) / (2 * h) - ref[i]) < 1e-8, key
    out, norm = R.clip_grads([np.array([3.0, 0.0]), np.array([[-4.0]])], 2.5)
    assert norm == 5.0 and out[0].tolist() == [1.5, 0.0] and out[1].tolist() == [[-2.0]]
    out, _ = R.clip_grads([np.array([3.0])], 7.0)
    assert out[0].tolist() == [3.0]
    out, norm = R.clip_grads([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and out[0][1] == 1.0


PINS = [pin_worked, pin_ties_and_masks, pin_renormalised_gates_keep_tiny_scores,
        pin_gradient_by_differences, pin_gradient_edges, pin_balance,
        pin_router_backward_and_clip]

MUTANTS = {
    "bias_in_gates": [("sj = np.take_along_axis(s,", "sj = np.take_along_axis(c,"),
                      ("g = np.where(lj == -np.inf, 0.0, sj)", "g = sj"),
                      ("ls = -np.logaddexp(0.0, -lj)",
                       "ls = np.log(np.take_along_axis(c, ids.astype(np.int64), axis=1))")],
    "tie_high": [("np.lexsort((np.arange(N),", "np.lexsort((-np.arange(N),")],
    "group_sum_of_one": [('kind == "max" or c.shape[2] == 1', "True")],
    "group_always_top2": [('if kind == "max" or c.shape[2] == 1:', "if c.shape[2] == 1:")],
    "group_tie_high": [('np.argsort(-gs, axis=1, kind="stable")[:, :topk_groups]',
                        "np.argsort(gs[:, ::-1] * -1, axis=1, kind='stable')[:, :topk_groups]")],
    "mask_forgotten": [("c = np.where(l == -np.inf, -np.inf, c)", "c = c + 0")],
    "no_scale": [("return ids, g * scale", "return ids, g")],
    "renorm_dropped": [("g = np.where(tot > 0, u / np.where(tot > 0, tot, 1.0), 0.0)", "g = u")],
    "no_projection": [("ds = (u - (u * sj).sum() / tot) / tot", "ds = u / tot")],
    "softmax_diag_only": [("s[t] * (dS - (dS * s[t]).sum())", "s[t] * dS * (1 - s[t])")],
    "duplicate_last_wins": [("dS[i] += x", "dS[i] = x")],
    "balance_sign": [("np.sign(cnt.sum() - N * cnt)", "np.sign(N * cnt - cnt.sum())")],
    "load_not_added": [("cnt = cnt + np.asarray(load, dtype=np.int64)", "pass")],
    "dx_add_dropped": [("dx = dx + np.asarray(dx_add, dtype=np.float64)", "pass")],
    "clip_up": [("if np.isfinite(norm) and norm > max_norm else 1.0", "")],
}


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_pin(pin):
    pin(O)


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_mistake_fails_a_pin(name):
    src = open(SRC).read()
    for old, new in MUTANTS[name]:
        assert old in src, old
        src = src.replace(old, new)
    m = types.ModuleType("mutant")
    exec(compile(src.replace("from __future__ import annotations", ""), name, "exec"), m.__dict__)
    failed = 0
    for pin in PINS:
        try:
            pin(m)
        except Exception:
            failed += 1
    assert failed, name


def test_choice_matches_a_loop():
    rng = np.random.default_rng(1)
    for _ in range(30):
        G = int(rng.integers(1, 5))
        N = G * int(rng.integers(2, 6))
        keep = int(rng.integers(1, G + 1))
        k = int(rng.integers(1, keep * (N // G) + 1))
        l = rng.integers(-3, 4, (4, N)) / 2.0
        b = rng.integers(-2, 3, N) / 4.0
        score = ("softmax", "sigmoid")[int(rng.integers(2))]
        kind = ("max", "top2")[int(rng.integers(2))]
        ids, _ = O.route_logits(l, k, score=score, bias=b, n_groups=G, topk_groups=keep,
                                group_score=kind)
        c = O.scores(l, score) + b
        for t in range(4):
            groups = [sorted(c[t, g * (N // G):(g + 1) * (N // G)], reverse=True)
                      for g in range(G)]
            val = [g[0] if kind == "max" else g[0] + g[1] for g in groups]
            kept = sorted(range(G), key=lambda g: (-val[g], g))[:keep]
            cand = [e for e in range(N) if e // (N // G) in kept]
            assert ids[t].tolist() == sorted(cand, key=lambda e: (-c[t, e], e))[:k]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_gradient_at_a_masked_pick_counts_nothing(score, renorm, bad):
    l = np.array([[0.5, -np.inf, 1.0, -1.0], [-np.inf, -np.inf, 2.0, 0.0]])
    ids = np.array([[0, 1, 2], [0, 2, 1]], dtype=np.int32)
    dg = np.array([[1.0, 0.0, -2.0], [0.0, 3.0, 0.0]])
    want = O.route_logits_backward(l, ids, dg, score=score, renorm=renorm)
    dg[0, 1] = dg[1, 0] = dg[1, 2] = bad
    assert np.array_equal(O.route_logits_backward(l, ids, dg, score=score, renorm=renorm), want)
    assert np.isfinite(want).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_through_a_nan_pick_is_nan(score):
    """Renormalised gates of a token with a NaN among its picks are NaN, and so
    is their gradient."""
    l = np.array([[0.5, np.nan, 1.0, -1.0], [0.5, 0.0, 1.0, -1.0]])
    ids = np.array([[0, 1], [0, 1]], dtype=np.int32)
    g = O.route_logits_backward(l, ids, np.ones((2, 2)), score=score, renorm=True)
    assert np.isnan(g[0, :2]).all() and np.isfinite(g[1]).all()


def test_gradient_of_a_row_without_picks_is_zero_whatever_its_logits():
    l = np.array([[np.nan, 1.0, 2.0], [np.inf, 0.0, 1.0], [np.nan, -np.inf, 0.0], [0.0, 1.0, 2.0]])
    ids = np.array([[-1, 3], [-1, -1], [1, -1], [0, 1]], dtype=np.int32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            g = O.route_logits_backward(l, ids, np.ones((4, 2)), score=score, renorm=renorm)
            assert (g[:3] == 0).all() and np.isfinite(g[3]).all()
