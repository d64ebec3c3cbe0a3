"""Plain fp64 CPU oracle of routing from logits, its gradient, the balance
bias, the router product's gradient and gradient clipping.

TEST INFRASTRUCTURE ONLY: used by ``tests/``. The HIP library never calls it,
and it shares no code with the HIP path.

Readings (the pages describe a top-k mixture of experts without a router):

* scores: softmax over the experts, or the sigmoid of each logit; a logit of
  ``-inf`` masks its expert (score 0, choice ``-inf``);
* choice: score + bias; without a bias the order is that of the logits;
* a group's score: its largest choice, or the sum of the two largest unmasked
  ones; ties go to the lower group, then to the lower expert;
* gates: scale * score, or scale * score / sum of the chosen scores (0 where
  all chosen are masked); a NaN logit, or +inf for the softmax, makes the
  token's gates NaN;
* a pick outside the experts, or a masked one, has no gradient.
"""
from __future__ import annotations

import numpy as np

__all__ = ["scores", "route_logits", "route_logits_backward", "route_balance",
           "router_backward", "grad_norm", "clip_grads"]


def scores(logits, score):
    """fp64 scores [T][N]; masked experts 0."""
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(l))
            return np.where(l >= 0, 1.0, e) / (1.0 + e)
        m = l.max(axis=1, keepdims=True)
        ex = np.where(l == -np.inf, 0.0, np.exp(l - m))
        s = ex / ex.sum(axis=1, keepdims=True)
        return np.where(l == -np.inf, np.where(np.isnan(m), np.nan, 0.0), s)


def _group_score(c, kind):
    """c [T][G][size] -> [T][G]."""
    srt = -np.sort(-np.where(np.isnan(c), -np.inf, c), axis=2)
    if kind == "max" or c.shape[2] == 1:
        return srt[:, :, 0]
    a, b = srt[:, :, 0], srt[:, :, 1]
    return np.where(b == -np.inf, a, a + np.where(b == -np.inf, 0.0, b))


def route_logits(logits, k, *, score="softmax", bias=None, renorm=True, scale=1.0, n_groups=1,
                 topk_groups=1, group_score="top2"):
    """(ids int32 [T][k], gates fp64 [T][k])."""
    l = np.asarray(logits, dtype=np.float64)
    T, N = l.shape
    s = scores(l, score)
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)[None, :]
    c = np.where(l == -np.inf, -np.inf, c)
    order_by = l if bias is None else c
    kept = np.ones((T, N), dtype=bool)
    if n_groups > 1:
        size = N // n_groups
        by = l if bias is None and group_score == "max" else c
        gs = _group_score(by.reshape(T, n_groups, size), group_score)
        best = np.argsort(-gs, axis=1, kind="stable")[:, :topk_groups]
        kg = np.zeros((T, n_groups), dtype=bool)
        np.put_along_axis(kg, best, True, axis=1)
        kept = np.repeat(kg, size, axis=1)
    # three classes: ordinary (and -inf) values, then NaN, then not kept
    cls = np.where(kept, np.where(np.isnan(order_by), 1, 0), 2)
    val = np.where(np.isnan(order_by), 0.0, -order_by)
    ids = np.empty((T, k), dtype=np.int32)
    for t in range(T):
        ids[t] = np.lexsort((np.arange(N), val[t], cls[t]))[:k]
    lj = np.take_along_axis(l, ids.astype(np.int64), axis=1)
    sj = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    with np.errstate(all="ignore"):
        if renorm:
            # ratios of the chosen scores, shifted so that none vanishes
            if score == "softmax":
                u = np.exp(lj - lj.max(axis=1, keepdims=True))
            else:
                # log sigmoid(l) = l - log(1 + e^l)
                ls = -np.logaddexp(0.0, -lj)
                u = np.exp(ls - ls.max(axis=1, keepdims=True))
            u = np.where(lj == -np.inf, 0.0, u)
            tot = u.sum(axis=1, keepdims=True)
            g = np.where(tot > 0, u / np.where(tot > 0, tot, 1.0), 0.0)
        else:
            g = np.where(lj == -np.inf, 0.0, sj)
    bad = np.isnan(l).any(axis=1)
    if score == "softmax":
        bad |= (l == np.inf).any(axis=1)
    g[bad] = np.nan
    return ids, g * scale


def route_logits_backward(logits, ids, dgates, *, score="softmax", renorm=True, scale=1.0):
    """fp64 dlogits [T][N] through the Jacobian of the gates, pick by pick."""
    l = np.asarray(logits, dtype=np.float64)
    T, N = l.shape
    k = ids.shape[1]
    s = scores(l, score)
    out = np.zeros((T, N))
    for t in range(T):
        # (a masked pick's gate is constant)
        js = [j for j in range(k) if 0 <= ids[t, j] < N and l[t, ids[t, j]] != -np.inf]
        if not js:
            continue
        e = [int(ids[t, j]) for j in js]
        u = scale * np.asarray([dgates[t, j] for j in js], dtype=np.float64)
        sj = s[t, e]
        if renorm:
            tot = sj.sum()
            if tot == 0:
                continue
            # d g_j / d s_i = (delta_ij - p_j) / tot
            ds = (u - (u * sj).sum() / tot) / tot
        else:
            ds = u
        if renorm and score == "softmax":
            # sum_i dS_i s_i = (sum u s - sum u s) / tot is 0: only the chosen move
            for i, x in zip(e, sj * ds):
                out[t, i] += x
            continue
        dS = np.zeros(N)
        for i, x in zip(e, ds):
            dS[i] += x
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = dS * s[t] / (1.0 + np.exp(l[t]))  # s (1 - s)
        else:
            out[t] = s[t] * (dS - (dS * s[t]).sum())
    return out


def route_balance(ids, N, *, bias=None, rate=0.0, load=None):
    """(load int64 [N], bias fp64 or None)."""
    flat = np.asarray(ids).reshape(-1)
    flat = flat[(flat >= 0) & (flat < N)]
    cnt = np.bincount(flat, minlength=N).astype(np.int64)
    if load is not None:
        cnt = cnt + np.asarray(load, dtype=np.int64)
    if bias is None:
        return cnt, None
    return cnt, np.asarray(bias, dtype=np.float64) + rate * np.sign(cnt.sum() - N * cnt)


def router_backward(x, w, logits, ids, dgates, *, dx_add=None, **spec):
    dl = route_logits_backward(logits, ids, dgates, **spec)
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    dx = dl @ w
    if dx_add is not None:
        dx = dx + np.asarray(dx_add, dtype=np.float64)
    return {"dx": dx, "dw": dl.T @ x, "dl": dl}


def grad_norm(grads):
    return float(np.sqrt(sum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads)))


def clip_grads(grads, max_norm):
    norm = grad_norm(grads)
    f = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return [np.asarray(g, dtype=np.float64) * f for g in grads], norm
