"""The bounds that the norm's gradient is held to are the oracle's values, and no
gradient with a mistake in it lies within them (CPU)."""
import numpy as np
import pytest

import norm_bounds as B
import oracle as O

WIDTHS = [(1, 4096, 8), (20, 2048, 4), (6, 4096, 2), (4, 5000, 2), (5, 8192, 3), (7, 2055, 2),
          (40, 320, 8), (50, 128, 3), (9, 61, 5)]


def oracle(s):
    kw = dict(k=s["k"], inv=B.f64(s["inv"]), gates=B.f64(s["gates"]), w_post=B.f64(s["w_post"]),
              w_pre=B.f64(s["w_pre"]), **B.SCALES)
    r, n = O.residual_norm(B.f64(s["u"]), B.f64(s["r"]), **kw)
    g = O.residual_norm_backward(B.f64(s["u"]), B.f64(s["r"]), dr_out=B.f64(s["dr_out"]),
                                 dn=B.f64(s["dn"]), **kw)
    return dict(r=r, n=n), g


@pytest.mark.parametrize("dt", [B.BF, B.F32])
@pytest.mark.parametrize("T,d,k", WIDTHS)
def test_the_oracles_values_rounded_lie_within(T, d, k, dt):
    s = B.draw(T, d, k, dt, seed=d + k, pad=0.2)
    fwd, back = oracle(s)
    want, named = B.backward(s)
    assert not B.outside({name: B.rounded(v, name, dt) for name, v in fwd.items()}, B.forward(s))
    back["du"] = np.where(named[:, None], back["du"], 0.0)
    for name, (ref, _) in want.items():
        assert np.allclose(ref, back[name], rtol=1e-9, atol=1e-9 * np.abs(ref).max()), name
    assert not B.outside({name: B.rounded(back[name], name, dt) for name in want}, want)


@pytest.mark.parametrize("dt", [B.BF, B.F32])
@pytest.mark.parametrize("T,d,k,wrong", [
    (*w, wrong) for w in WIDTHS for wrong in B.WRONG
    if w[2] > 2 or wrong != "dgates of the first two picks only"])
def test_wrong_gradients_lie_outside(T, d, k, wrong, dt):
    s = B.draw(T, d, k, dt, seed=d + k)
    want, _ = B.backward(s)
    got, _ = B.backward(s, wrong)
    assert B.outside({name: B.rounded(v, name, dt) for name, (v, _) in got.items()}, want)


@pytest.mark.parametrize("dt", [B.BF, B.F32])
def test_wrong_sums_of_a_tokens_rows_lie_outside(dt):
    s = B.draw(20, 2048, 4, dt, seed=1)
    want = B.forward(s)
    short = dict(s, gates=s["gates"].clone())
    short["gates"][:, 3] = 0
    got = {name: B.rounded(v, name, dt) for name, (v, _) in B.forward(short).items()}
    assert set(B.outside(got, want)) == {"r", "n"}
