"""The norms around a block and their gradient on the GPU within bounds that follow
each operation's rounding (a gradient with any of the mistakes that the CPU tests
make lies outside of them)."""
import numpy as np
import pytest
import torch

import norm_bounds as B
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = B.BF, B.F32


def cuda(t):
    return None if t is None else t.cuda()


def check(s):
    kw = dict(k=s["k"], inv=cuda(s["inv"]), gates=cuda(s["gates"]), w_post=cuda(s["w_post"]),
              w_pre=cuda(s["w_pre"]))
    spec = bmoe.NormSpec(**B.SCALES)
    u, r = s["u"].cuda(), s["r"].cuda()
    got = dict(zip(("r", "n"), bmoe.residual_norm(u, r, spec, **kw)))
    want = B.forward(s)
    assert not B.outside({name: B.f64(got[name]) for name in want}, want)
    got = bmoe.residual_norm_backward(u, r, spec, dr_out=cuda(s["dr_out"]), dn=cuda(s["dn"]),
                                      du=torch.zeros_like(u), **kw)
    want, _ = B.backward(s)
    assert not B.outside({name: B.f64(got[name]) for name in want}, want)


# every width's kernel, one token to several a workgroup, one pick to many
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,d,k", [(1, 4096, 8), (20, 2048, 4), (6, 4096, 2), (4, 5000, 2),
                                   (5, 8192, 3), (7, 2055, 2), (5, 4095, 1), (3, 8191, 1),
                                   (900, 2048, 2), (1700, 1030, 3), (33, 1024, 1), (130, 1000, 4),
                                   (40, 320, 8), (21, 500, 17), (3100, 256, 2), (2600, 48, 2),
                                   (50, 128, 3), (9, 61, 64), (6, 3, 2)])
def test_widths(T, d, k, dt):
    check(B.draw(T, d, k, dt, seed=T + d, pad=0.1 if k > 1 else 0.0))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("gates,post,pre", [(0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 1), (0, 0, 0)])
def test_parts_left_out(gates, post, pre, dt):
    for d, k in ((96, 3), (1111, 2), (4096, 4)):
        check(B.draw(21, d, k, dt, seed=d, gates=gates, post=post, pre=pre))
