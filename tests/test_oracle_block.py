"""The block oracle against hand values, differences and identities (CPU)."""
import numpy as np
import pytest

import oracle as O


def test_group_rows_by_hand():
    off, perm, inv = O.group_rows(np.array([[2, 0], [7, 2], [0, -1]]), 3)
    assert off.tolist() == [0, 2, 2, 4]
    assert perm.tolist() == [1, 4, 0, 3, 2, 5]
    assert inv.tolist() == [2, 0, -1, 3, 1, -1]


def test_grouped_product_is_each_row_by_its_expert():
    rng = np.random.default_rng(0)
    ids = rng.integers(0, 4, (5, 2))
    a, w = rng.standard_normal((5, 3)), rng.standard_normal((4, 6, 3))
    off, perm, inv = O.group_rows(ids, 4)
    c = O.grouped_product(a, w, off, perm // 2)
    for r in range(10):
        assert np.allclose(c[inv[r]], w[ids.reshape(-1)[r]] @ a[r // 2])


def _difference(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def test_grouped_gradients_by_differences():
    rng = np.random.default_rng(1)
    a, w, dc = rng.standard_normal((7, 3)), rng.standard_normal((3, 4, 3)), rng.standard_normal((7, 4))
    off, rows = np.array([0, 4, 4, 7]), np.arange(7)
    da, dw = O.grouped_product_backward(a, w, off, rows, dc)

    def f():
        return float(np.sum(O.grouped_product(a, w, off, rows) * dc))
    assert np.allclose(da, _difference(f, a), atol=1e-7)
    assert np.allclose(dw, _difference(f, w), atol=1e-7)
    assert not dw[1].any()


@pytest.mark.parametrize("gated,post,pre", [(1, 1, 1), (0, 1, 0), (1, 0, 1), (0, 0, 1), (1, 0, 0)])
def test_norm_gradients_by_differences(gated, post, pre):
    rng = np.random.default_rng(2)
    T, d, k = 3, 5, 2
    u, r = rng.standard_normal((7, d)), rng.standard_normal((T, d))
    inv = np.array([4, 0, -1, 6, 2, 3])
    gates = rng.standard_normal((T, k)) if gated else None
    w_post = rng.standard_normal(d) if post else None
    w_pre = rng.standard_normal(d) if pre else None
    dr, dn = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    kw = dict(k=k, inv=inv, gates=gates, w_post=w_post, w_pre=w_pre, eps=0.01, res_scale=0.7,
              out_scale=1.3)

    def f():
        a, n = O.residual_norm(u, r, **kw)
        return float(np.sum(a * dr) + (np.sum(n * dn) if pre else 0.0))
    g = O.residual_norm_backward(u, O.residual_norm(u, r, **kw)[0], dr_out=dr,
                                 dn=dn if pre else None, **kw)
    named = inv[inv >= 0]
    assert np.allclose(g["du"][named], _difference(f, u)[named], atol=1e-6)
    assert np.isnan(np.delete(g["du"], named, axis=0)).all()
    assert np.allclose(g["dr"], _difference(f, r), atol=1e-6)
    for name, x in (("dgates", gates), ("dw_post", w_post), ("dw_pre", w_pre)):
        if x is not None:
            assert np.allclose(g[name], _difference(f, x), atol=1e-6), name


def test_norm_without_a_block_and_of_an_empty_token():
    r, w = np.array([[3.0, 4.0]]), np.array([1.0, 2.0])
    a, n = O.residual_norm(None, r, w_pre=w, eps=0.0)
    assert np.allclose(n, np.array([[3.0, 8.0]]) / np.sqrt(12.5)) and np.array_equal(a, r)
    a, _ = O.residual_norm(np.ones((2, 2)), r, inv=np.array([-1]), w_post=w)
    assert np.array_equal(a, r)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (5, 1)])
def test_newton_schulz_moves_singular_values_alone(shape):
    u = np.random.default_rng(3).standard_normal(shape)
    a, b, c = 3.4445, -4.7750, 2.0315
    left, s, right = np.linalg.svd(u, full_matrices=False)
    start = s = s / np.sqrt(np.sum(s * s))
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(O.newton_schulz(u, eps=0.0), (left * s) @ right, atol=1e-10)
    # what starts above 0.02 is past 0.02 * 3.3 ** 4 > 1 of linear growth within five steps
    assert (s[start > 0.02] > 0.6).all() and (s < 1.25).all()
