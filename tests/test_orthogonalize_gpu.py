"""Newton-Schulz orthogonalisation and the weight step on the GPU against fp64.

Tolerance, relative in the Frobenius norm. An iterate is an odd matrix
polynomial, whose derivative in that norm is at most the largest |p'| on the
iterates' range: p' = a + 3 b s^2 + 5 c s^4 is below 3.9 for |s| <= 1.21. A
step's own error is that of three products with operands of 22 bits (2^-22 rms
of each product's terms, with coefficients of up to 4.8) and fp32 sums, below
2^-19 in all. So after n steps: 2^-19 (1 + 3.9 + ... + 3.9^(n-1)) + 3.9^n 2^-23
(the last for the rounded start), and half a step for a bf16 result (2^-8)."""
import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def tol(steps, dt):
    return (2.0 ** -19 * sum(3.9 ** i for i in range(steps)) + 3.9 ** steps * 2.0 ** -23 +
            (2.0 ** -8 if dt == BF else 2.0 ** -24))


def rel(got, ref):
    return float(np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref))


def randn(shape, dt, seed=0, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dt)


SHAPES = [(1, 1), (1, 9), (9, 1), (8, 8), (7, 300), (300, 7), (64, 512), (130, 120), (127, 128),
          (129, 257), (257, 129), (128, 128), (100, 1000), (1000, 100), (520, 300), (264, 1032)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_matrix(rows, cols, dt):
    u = randn((rows, cols), dt, rows + cols, 0.02)
    for steps in (1, 5):
        o = bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(steps))
        assert o.dtype == dt and o.shape == u.shape
        assert rel(o, O.newton_schulz(f64(u), steps)) <= tol(steps, dt), steps


@pytest.mark.parametrize("shape", [(3, 40, 72), (5, 72, 40), (2, 200, 136), (70, 24, 16)])
def test_batches_are_each_matrix_by_itself(shape):
    u = randn(shape, F32, 1)
    u *= torch.logspace(-3, 3, shape[0]).view(-1, 1, 1)
    o = bmoe.orthogonalize(u.cuda())
    for i in range(shape[0]):
        assert rel(o[i], O.newton_schulz(f64(u[i]))) <= tol(5, F32)
        assert torch.equal(o[i], bmoe.orthogonalize(u[i].cuda()))


@pytest.mark.parametrize("shape", [(96, 160), (160, 96)])
def test_extremes(shape):
    for scale in (1e-30, 1e30):                       # squares neither vanish nor overflow
        u = randn(shape, F32, 2, scale)
        o = bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(eps=0.0))
        assert rel(o, O.newton_schulz(f64(u), eps=0.0)) <= tol(5, F32)
    z = torch.zeros(shape, device="cuda")
    assert not bmoe.orthogonalize(z).any()
    for bad in (float("nan"), float("inf")):
        u = randn((2, *shape), F32, 3)
        u[0, 5, 9] = bad
        o = bmoe.orthogonalize(u.cuda())
        assert o[0].isnan().all() and torch.isfinite(o[1]).all()
    # a row of very different size, and rank one
    u = randn(shape, F32, 4)
    u[3] *= 1e4
    assert rel(bmoe.orthogonalize(u.cuda()), O.newton_schulz(f64(u))) <= tol(5, F32)
    u = randn((shape[0], 1), F32, 5) @ randn((1, shape[1]), F32, 6)
    assert rel(bmoe.orthogonalize(u.cuda()), O.newton_schulz(f64(u))) <= tol(5, F32)


def test_other_coefficients_and_in_place():
    u = randn((88, 200), F32, 7)
    spec = bmoe.OrthoSpec(12, (1.5, -0.5, 0.0), eps=0.0)   # the cubic iteration
    ref = O.newton_schulz(f64(u), 12, (1.5, -0.5, 0.0), 0.0)
    dev = u.cuda()
    o = bmoe.orthogonalize(dev, spec, out=dev)
    # its derivative is at most 1.5
    assert o is dev and rel(o, ref) <= 2.0 ** -19 * sum(1.5 ** i for i in range(12)) + 1.5 ** 12 * 2.0 ** -23


@pytest.mark.parametrize("w_dt", [F32, BF])
@pytest.mark.parametrize("g_dt", [F32, BF])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(48, 100), (3, 130, 64), (33, 17)])
def test_step(shape, nesterov, g_dt, w_dt):
    w, g = randn(shape, w_dt, 8, 0.1), randn(shape, g_dt, 9, 0.01)
    m = randn(shape, F32, 10, 0.05)
    dw, dm = w.cuda(), m.cuda()
    lr, beta, decay, scale = 0.02, 0.95, 0.1, 1.5
    out = bmoe.orthogonal_step(dw, g.cuda(), dm, lr, beta=beta, nesterov=nesterov,
                               weight_decay=decay, scale=scale)
    assert out is dw
    b32 = float(np.float32(beta))
    rm = b32 * f64(m) + f64(g)
    assert (np.abs(f64(dm) - rm) <= 2.0 ** -24 * np.abs(rm)).all()   # one fused operation
    u = (f64(g) + b32 * rm if nesterov else rm).reshape(-1, *shape[-2:])
    o = np.stack([O.newton_schulz(x) for x in u]).reshape(shape)
    step = f64(dw) - (1 - lr * decay) * f64(w)
    half = 2.0 ** -8 if w_dt == BF else 2.0 ** -24
    # w's rounding, the fp32 scalars', and the iteration's error spread over a matrix
    bound = half * np.abs(f64(dw)) + 2.0 ** -22 * np.abs(f64(w))
    err = np.maximum(np.abs(step + lr * scale * o) - bound, 0.0)
    for e, x in zip(err.reshape(-1, *shape[-2:]), o.reshape(-1, *shape[-2:])):
        assert np.linalg.norm(e) <= lr * scale * np.linalg.norm(x) * tol(5, F32)


def test_same_bits_each_run():
    u = randn((300, 260), F32, 11).cuda()
    first = bmoe.orthogonalize(u)
    for _ in range(3):
        assert torch.equal(first, bmoe.orthogonalize(u))


# Batches and sizes whose launches take each of the tiles (64, 128 eight waves deep,
# 128, 192 and 256), wide and tall, whole chunks and not
@pytest.mark.parametrize("shape", [(1, 1500, 1510), (1, 2050, 2100), (42, 550, 561), (64, 500, 510),
                                   (80, 500, 512)])
@pytest.mark.parametrize("tall", [False, True])
def test_every_tile(shape, tall):
    B, m, n = shape
    u = randn((B, n, m) if tall else shape, F32, B, 0.01)
    steps = 1 if B == 1 else 5
    o = bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(steps))
    for i in {0, B // 2, B - 1}:
        assert rel(o[i], O.newton_schulz(f64(u[i]), steps)) <= tol(steps, F32), i


# Small sides: one workgroup, slabs of columns (up to 64 of them), batches, each
# type, and the momentum's step; a slab of one column
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("shape", [(1, 64, 513), (1, 33, 1000), (3, 64, 2048), (1, 32, 1025),
                                   (2, 17, 3001), (1, 1, 1300), (1, 50, 16384), (5, 8, 1281)])
@pytest.mark.parametrize("tall", [False, True])
def test_slabs(shape, tall, dt):
    B, m, n = shape
    shape = (B, n, m) if tall else shape
    u = randn(shape, dt, n, 0.01)
    for steps in (1, 2, 5):
        o = bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(steps))
        for i in {0, B - 1}:
            assert rel(o[i], O.newton_schulz(f64(u[i]), steps)) <= tol(steps, dt), (i, steps)
    w, mo = randn(shape, dt, 1, 0.1), randn(shape, F32, 2, 0.01)
    dw, dm = w.cuda(), mo.cuda()
    bmoe.orthogonal_step(dw, u.cuda(), dm, 0.02, beta=0.5)
    rm = 0.5 * f64(mo) + f64(u)
    assert (np.abs(f64(dm) - rm) <= 2.0 ** -24 * np.abs(rm)).all()
    half = 2.0 ** -8 if dt == BF else 2.0 ** -24
    for i in {0, B - 1}:
        o = O.newton_schulz(f64(u[i]) + 0.5 * rm[i])
        err = np.abs(f64(dw[i]) - (f64(w[i]) - 0.02 * o)) - half * np.abs(f64(dw[i])) - \
            2.0 ** -22 * np.abs(f64(w[i]))
        assert np.linalg.norm(np.maximum(err, 0)) <= 0.02 * np.linalg.norm(o) * tol(5, F32)
    bad = u.cuda()
    bad[0, -1, -1] = float("nan")
    assert bmoe.orthogonalize(bad)[0].isnan().all()
