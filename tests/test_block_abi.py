"""Host-side refusals of the dense experts, the norms around a block and the
orthogonalised updates: every one returns before any HIP call, so they run
without a GPU. Pointers are made-up addresses that nothing reads."""
import ctypes

import pytest
import torch

from butterfly_rotated_ternary_amd import bmoe

BF, F32 = bmoe.BMOE_BF16, bmoe.BMOE_F32
OK, NULL, SHAPE, DTYPE, WS, ALIGN, VALUE = 0, 1, 2, 3, 6, 8, 9


def at(i):
    """Aligned addresses far from each other."""
    return 0x1000000000 * (i + 1)


def test_group_rows_refuses():
    n = bmoe.bmoe_group_rows_workspace_bytes
    assert n(4, 0, 2) == 0 and n(4, 4097, 2) == 0 and n(-1, 8, 2) == 0 and n(4, 8, 0) == 0
    assert n(1 << 30, 8, 2) == 0 and n(0, 8, 2) > 0 and n(4, 8, 2) > 0
    big = n(4, 8, 2)

    def call(T=4, N=8, k=2, ids=at(0), off=at(1), perm=at(2), inv=at(3), ws=at(4), wb=big):
        return bmoe.lib().bmoe_group_rows(T, N, k, ids, off, perm, inv, ws, wb, None)
    assert call(N=0) == SHAPE and call(T=-1) == SHAPE and call(k=0) == SHAPE
    for name in ("ids", "off", "perm", "inv"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: at(5) + 4}) == ALIGN, name
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(perm=at(0)) == VALUE and call(inv=at(2) + 16) == VALUE


def product(dt=BF, M=8, K=16, O=24, G=4, a=at(0), rows=5, perm=at(1), k=2, w=at(2), off=at(3),
            c=at(4)):
    return bmoe.lib().bmoe_grouped_product(dt, M, K, O, G, a, rows, perm, k, w, off, c, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(M=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(K=65537)),
    (SHAPE, dict(O=0)), (SHAPE, dict(O=65537)), (SHAPE, dict(G=0)), (SHAPE, dict(G=4097)),
    (SHAPE, dict(k=0)), (SHAPE, dict(rows=0)), (OK, dict(M=0, a=None)), (NULL, dict(a=None)),
    (NULL, dict(w=None)), (NULL, dict(off=None)), (NULL, dict(c=None)), (ALIGN, dict(a=at(0) + 8)),
    (ALIGN, dict(perm=at(1) + 4)), (ALIGN, dict(off=at(3) + 4)), (VALUE, dict(c=at(0) + 144)),
    (VALUE, dict(c=at(2) + 16)), (VALUE, dict(c=at(3)))])
def test_grouped_product_refuses(want, kw):
    assert product(**kw) == want


def test_grouped_product_backward_refuses():
    n = bmoe.bmoe_grouped_product_backward_workspace_bytes
    assert n(7, 8, 16, 24, 4) == 0 and n(BF, 8, 0, 24, 4) == 0 and n(BF, 8, 16, 24, 4097) == 0
    big = n(BF, 8, 16, 24, 4)
    assert big > 0

    def call(dt=BF, M=8, K=16, O=24, G=4, a=at(0), rows=5, perm=at(1), k=2, w=at(2), off=at(3),
             dc=at(4), da=at(5), dw=at(6), ws=at(7), wb=big):
        return bmoe.lib().bmoe_grouped_product_backward(dt, M, K, O, G, a, rows, perm, k, w, off,
                                                        dc, da, dw, ws, wb, None)
    assert call(dt=9) == DTYPE and call(K=0) == SHAPE and call(k=0) == SHAPE
    for name in ("a", "w", "off", "dc"):
        assert call(**{name: None}) == NULL, name
    for name in ("a", "perm", "w", "off", "dc", "da", "dw", "ws"):
        assert call(**{name: at(8) + 8}) == ALIGN, name
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(da=at(4)) == VALUE and call(dw=at(5)) == VALUE and call(ws=at(2)) == VALUE


def spec(**kw):
    return ctypes.byref(bmoe.NormSpec(**kw))


def norm(dt=BF, T=4, d=16, k=2, sp=None, u=at(0), rows=8, inv=at(1), g=at(2), r=at(3), post=at(4),
         pre=at(5), out=at(6), n=at(7)):
    return bmoe.lib().bmoe_residual_norm(dt, T, d, k, sp or spec(), u, rows, inv, g, r, post, pre,
                                         out, n, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(T=-1)), (SHAPE, dict(d=0)), (SHAPE, dict(d=8193)),
    (SHAPE, dict(k=0)), (SHAPE, dict(k=65)), (SHAPE, dict(T=1 << 30)), (SHAPE, dict(rows=-1)),
    (SHAPE, dict(inv=None, rows=7)), (VALUE, dict(sp=spec(eps=-1.0))),
    (VALUE, dict(sp=spec(eps=float("nan")))), (VALUE, dict(sp=spec(res_scale=float("inf")))),
    (VALUE, dict(sp=spec(out_scale=float("nan")))), (OK, dict(T=0, u=None, r=None)),
    (NULL, dict(u=None, r=None)), (NULL, dict(u=None)), (NULL, dict(n=None)), (NULL, dict(out=None)),
    (NULL, dict(pre=None, out=None)), (ALIGN, dict(u=at(0) + 2)), (ALIGN, dict(g=at(2) + 4)),
    (ALIGN, dict(pre=at(5) + 4)), (VALUE, dict(out=at(0))), (VALUE, dict(out=at(3) + 16)),
    (VALUE, dict(n=at(3))), (VALUE, dict(out=at(3), n=at(3))), (VALUE, dict(n=at(6) + 112))])
def test_residual_norm_refuses(want, kw):
    assert norm(**kw) == want


def test_residual_norm_needs_a_spec():
    assert bmoe.lib().bmoe_residual_norm(BF, 4, 16, 2, None, at(0), 8, at(1), at(2), at(3), at(4),
                                         at(5), at(6), at(7), None) == NULL


def test_residual_norm_backward_refuses():
    n = bmoe.bmoe_residual_norm_backward_workspace_bytes
    assert n(5, 4, 16) == 0 and n(BF, -1, 16) == 0 and n(BF, 4, 8193) == 0 and n(BF, 0, 16) > 0
    big = n(BF, 4, 16)
    names = ("u", "inv", "g", "x", "post", "pre", "dro", "dn", "du", "dg", "dr", "dpost", "dpre")

    def call(dt=BF, T=4, d=16, k=2, sp=None, rows=8, wb=big, ws=at(20), **kw):
        p = {name: at(i) for i, name in enumerate(names)}
        p.update(kw)
        return bmoe.lib().bmoe_residual_norm_backward(
            dt, T, d, k, sp or spec(), p["u"], rows, p["inv"], p["g"], p["x"], p["post"], p["pre"],
            p["dro"], p["dn"], p["du"], p["dg"], p["dr"], p["dpost"], p["dpre"], ws, wb, None)
    assert call(dt=4) == DTYPE and call(d=8193) == SHAPE and call(k=0) == SHAPE
    assert call(sp=spec(eps=-1.0)) == VALUE
    for name in ("x", "dn", "u", "g", "post", "pre"):
        assert call(**{name: None}) == NULL, name
    assert call(pre=None, dpre=None) == NULL                      # dn without its norm
    assert call(pre=None, dpre=None, dn=None, dro=None) == NULL   # nothing to differentiate
    for name in names:
        assert call(**{name: at(21) + 8}) == ALIGN, name
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(du=at(0)) == VALUE and call(dr=at(3)) == VALUE and call(dpost=at(5)) == VALUE
    assert call(dr=at(6) + 16) == VALUE and call(dg=at(8)) == VALUE


def ortho(**kw):
    return ctypes.byref(bmoe.OrthoSpec(**kw))


def test_orthogonalize_refuses():
    n = bmoe.bmoe_orthogonalize_workspace_bytes
    assert n(-1, 4, 4) == 0 and n(65536, 4, 4) == 0 and n(1, 0, 4) == 0 and n(1, 16385, 4) == 0
    assert n(1, 4, 16385) == 0 and n(0, 4, 4) > 0
    big = n(2, 8, 16)

    def call(dt=F32, B=2, rows=8, cols=16, sp=None, u=at(0), o=at(1), ws=at(2), wb=big):
        return bmoe.lib().bmoe_orthogonalize(dt, B, rows, cols, sp or ortho(), u, o, ws, wb, None)
    assert call(dt=2) == DTYPE and call(rows=0) == SHAPE and call(B=0, u=None) == OK
    assert call(u=None) == NULL and call(o=None) == NULL
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(u=at(0) + 4) == ALIGN and call(o=at(1) + 8) == ALIGN
    assert call(o=at(0) + 16) == VALUE and call(o=at(2)) == VALUE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=nan),
                dict(coeffs=(nan, 0, 0)), dict(coeffs=(1.5, inf, 0)),
                dict(coeffs=(16.0, 0, 0)),                 # |a| alone
                dict(steps=2, coeffs=(3.9, 0, 0)),         # sigma^2 past the range in the 2nd step
                dict(steps=8, coeffs=(1.0, 1.0, 0.0))):    # grows step by step
        assert call(sp=ortho(**bad)) == VALUE, bad
    assert bmoe.lib().bmoe_orthogonalize(F32, 2, 8, 16, None, at(0), at(1), at(2), big, None) == NULL


def test_orthogonal_step_refuses():
    big = bmoe.bmoe_orthogonalize_workspace_bytes(2, 8, 16)

    def call(wd=F32, gd=BF, rows=8, sp=None, up=None, g=at(0), m=at(1), w=at(2), ws=at(3), wb=big):
        u = bmoe.OrthoUpdate(0.1, 0.9, 1, 0.0, 1.0)
        for key, v in (up or {}).items():
            setattr(u, key, v)
        return bmoe.lib().bmoe_orthogonal_step(wd, gd, 2, rows, 16, sp or ortho(), ctypes.byref(u),
                                               g, m, w, ws, wb, None)
    assert call(wd=3) == DTYPE and call(gd=3) == DTYPE and call(rows=0) == SHAPE
    assert call(sp=ortho(steps=0)) == VALUE
    for bad in (dict(beta=1.0), dict(beta=-0.1), dict(beta=float("nan")), dict(lr=float("inf")),
                dict(weight_decay=float("nan")), dict(scale=float("inf"))):
        assert call(up=bad) == VALUE, bad
    for name in ("g", "m", "w"):
        assert call(**{name: None}) == NULL and call(**{name: at(5) + 4}) == ALIGN, name
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(m=at(0)) == VALUE and call(w=at(0) + 16) == VALUE and call(w=at(1)) == VALUE
    assert bmoe.lib().bmoe_orthogonal_step(F32, F32, 2, 8, 16, ortho(), None, at(0), at(1), at(2),
                                           at(3), big, None) == NULL


def test_wrappers_refuse_before_the_library():
    x, off = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int32)
    w, ids = torch.zeros(2, 5, 8), torch.zeros(4, 2, dtype=torch.int32)
    for bad in (lambda: bmoe.group_rows(ids, 2), lambda: bmoe.grouped_product(x, w, off),
                lambda: bmoe.residual_norm(x, x), lambda: bmoe.orthogonalize(x),
                lambda: bmoe.group_rows(ids.long(), 2),
                lambda: bmoe.grouped_product(x, w[0], off),
                lambda: bmoe.grouped_product(x, w[:, :, :4], off),
                lambda: bmoe.grouped_product(x, w, off[:2]),
                lambda: bmoe.grouped_product(x.t(), w, off),
                lambda: bmoe.residual_norm(None, None),
                lambda: bmoe.residual_norm(None, x, gates=torch.zeros(4, 1)),
                lambda: bmoe.residual_norm(x, x, k=2),
                lambda: bmoe.residual_norm_backward(x, x),
                lambda: bmoe.residual_norm_backward(x, x, dr_out=x, dn=x),
                lambda: bmoe.orthogonalize(x[0]), lambda: bmoe.orthogonalize(x.t()),
                lambda: bmoe.orthogonal_step(x, x[:2], x, 0.1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bmoe.orthogonalize(x.half())


def test_counts_past_an_int_are_refused():
    """Not wrapped to small ones (tensors without storage: nothing runs)."""
    lots = 2 ** 32 + 8

    def meta(*shape, dt=torch.bfloat16):
        return torch.empty(*shape, dtype=dt, device="meta")
    i32, w = torch.int32, torch.float32
    off = meta(3, dt=i32)
    for call in [lambda: bmoe.group_rows(meta(lots, 1, dt=i32), 4),
                 lambda: bmoe.group_rows(meta(2 ** 30, 4, dt=i32), 4),
                 lambda: bmoe.group_rows(meta(4, 1, dt=i32), lots),
                 lambda: bmoe.grouped_product(meta(lots, 8), meta(2, 8, 8), off),
                 lambda: bmoe.grouped_product(meta(8, 8), meta(2, 8, 8), off, perm=meta(lots, dt=i32)),
                 lambda: bmoe.grouped_product(meta(8, lots), meta(2, 8, lots), off),
                 lambda: bmoe.grouped_product(meta(8, 8), meta(2, 8, 8), off, perm=meta(8, dt=i32),
                                              k=lots),
                 lambda: bmoe.grouped_product_backward(meta(lots, 8), meta(2, 8, 8), off,
                                                       meta(lots, 8)),
                 lambda: bmoe.residual_norm(None, meta(lots, 1), w_pre=meta(1, dt=w)),
                 lambda: bmoe.residual_norm(meta(lots, 1), meta(4, 1), inv=meta(4, dt=i32)),
                 lambda: bmoe.residual_norm_backward(None, meta(lots, 1), dr_out=meta(lots, 1)),
                 lambda: bmoe.orthogonalize(meta(8, lots)),
                 lambda: bmoe.orthogonalize(meta(lots, 8, 8)),
                 lambda: bmoe.orthogonal_step(meta(8, lots), meta(8, lots), meta(8, lots, dt=w), 0.1)]:
        with pytest.raises(ValueError, match="at most 2"):
            call()
