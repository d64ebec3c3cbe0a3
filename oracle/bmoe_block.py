"""Plain fp64 CPU oracle of what stands around an expert layer's block: rows
grouped by expert and their products, the norms around the block, the
Newton-Schulz iteration.

TEST INFRASTRUCTURE ONLY: used by ``tests/``. The HIP library never calls it,
and it shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def group_rows(ids: np.ndarray, n_experts: int):
    """(offsets, perm, inv) of the flat ids: a stable sort by expert, ids outside
    [0, n_experts) last and without a slot."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < n_experts), flat, n_experts)
    perm = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[perm], np.arange(n_experts + 1), side="left")
    inv = np.full(flat.size, -1, dtype=np.int64)
    inside = perm[:offsets[n_experts]]
    inv[inside] = np.arange(inside.size)
    return offsets.astype(np.int32), perm.astype(np.int32), inv.astype(np.int32)


def grouped_product(a, w, offsets, rows):
    """c[q] = w[e] a[rows[q]]; rows of no group are NaN."""
    c = np.full((len(rows), w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        q = slice(offsets[e], offsets[e + 1])
        c[q] = a[rows[q]] @ w[e].T
    return c


def grouped_product_backward(a, w, offsets, rows, dc):
    da = np.full((len(rows), w.shape[2]), np.nan)
    dw = np.zeros(w.shape)
    for e in range(w.shape[0]):
        q = slice(offsets[e], offsets[e + 1])
        da[q] = dc[q] @ w[e]
        dw[e] = dc[q].T @ a[rows[q]]
    return da, dw


def _picked(u, inv, T, k):
    """u's rows by token [T][k][d] (zeros for a row outside u) and which exist."""
    at = np.arange(T * k) if inv is None else np.asarray(inv).astype(np.int64)
    ok = (at >= 0) & (at < len(u))
    rows = np.where(ok[:, None], u[np.where(ok, at, 0)], 0.0)
    return rows.reshape(T, k, -1), ok.reshape(T, k), at.reshape(T, k)


def residual_norm(u, r, *, k=1, inv=None, gates=None, w_post=None, w_pre=None, eps=1e-6,
                  res_scale=1.0, out_scale=1.0, T=None):
    """(r', n) in fp64, neither rounded."""
    T = len(r) if r is not None else T
    total = 0.0 if r is None else res_scale * r
    if u is not None:
        rows, _, _ = _picked(u, inv, T, k)
        g = np.ones((T, k)) if gates is None else gates
        y = np.zeros((T, u.shape[1]))
        for j in range(k):
            y = y + g[:, j:j + 1] * rows[:, j]
        if w_post is not None:
            y = y / np.sqrt(np.mean(y ** 2, axis=1, keepdims=True) + eps) * w_post
        total = total + out_scale * y
    n = None
    if w_pre is not None:
        n = total / np.sqrt(np.mean(total ** 2, axis=1, keepdims=True) + eps) * w_pre
    return total, n


def _rms_backward(v, w, dout, eps):
    """Gradients of v / sqrt(mean v^2 + eps) * w with respect to v and w."""
    s = np.sqrt(np.mean(v ** 2, axis=1, keepdims=True) + eps)
    t = dout * w
    dv = t / s - v * np.mean(t * v, axis=1, keepdims=True) / s ** 3
    return dv, np.sum(dout * v / s, axis=0)


def residual_norm_backward(u, r_out, *, k=1, inv=None, gates=None, w_post=None, w_pre=None,
                           dr_out=None, dn=None, eps=1e-6, res_scale=1.0, out_scale=1.0):
    """Gradients from dr' and dn, at r' = r_out. du: NaN where no pick names a row."""
    T, d = r_out.shape
    out = {}
    dr = np.zeros((T, d)) if dr_out is None else dr_out.copy()
    if w_pre is not None:
        dv, out["dw_pre"] = _rms_backward(r_out, w_pre, dn, eps)
        dr = dr + dv
    out["dr"] = res_scale * dr
    if u is None:
        return out
    rows, ok, at = _picked(u, inv, T, k)
    g = np.ones((T, k)) if gates is None else gates
    y = np.zeros((T, d))
    for j in range(k):
        y = y + np.where(ok[:, j:j + 1], g[:, j:j + 1] * rows[:, j], 0.0)
    dy = out_scale * dr
    if w_post is not None:
        dy, out["dw_post"] = _rms_backward(y, w_post, dy, eps)
    du = np.full(u.shape, np.nan)
    for j in range(k):
        du[at[ok[:, j], j]] = (g[:, j:j + 1] * dy)[ok[:, j]]
    out["du"] = du
    if gates is not None:
        out["dgates"] = np.where(ok, np.einsum("td,tkd->tk", dy, rows), 0.0)
    return out


def newton_schulz(u, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """The iterate of one matrix: singular values through an odd polynomial."""
    a, b, c = coeffs
    x = u / (np.sqrt(np.sum(u * u)) + eps)
    if x.shape[0] > x.shape[1]:
        return newton_schulz_wide(x.T, steps, a, b, c).T
    return newton_schulz_wide(x, steps, a, b, c)


def newton_schulz_wide(x, steps, a, b, c):
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x
