"""Newton-Schulz steps of matrices whose rows or columns differ in size, each row
and column judged by itself.

Tolerance. X's entries are pairs of fp16 of 2^15 times the value (for the default
coefficients): below 2^-18 what is lost is uniform within half of the last
subnormal place, 2^-40, so 2^-40 / sqrt(3) in the mean square. One step takes a row
that is small to about a = 3.4445 times itself, and with it that error: for n
entries 3.4445 sqrt(n) 2^-40 / sqrt(3) = 2 sqrt(n) 2^-40 in the 2-norm. P's and Q's
own entries add a term of a few 2^-40 without sqrt(n). Two and a half times the mean
square's is allowed (a sum over hundreds of independent roundings is within a few
hundredths of it), and 2^-19 of the row's own norm for the 22 bits and the fp32 sums."""
import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


# one workgroup, slabs, tiles of 64 and of 128
@pytest.mark.parametrize("m,n", [(32, 900), (64, 512), (24, 3000), (130, 520), (600, 1500)])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("side", ["short", "long"])
def test_small_rows_and_columns(m, n, tall, side):
    u = randn((m, n), m + n)
    if side == "short":
        u *= torch.logspace(0, -6, m)[:, None]
    else:
        u *= torch.logspace(0, -6, n)[None]
    if tall:
        u = u.t().contiguous()
    o = f64(bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(1)))
    ref = O.newton_schulz(f64(u), 1)
    if (side == "short") == tall:
        o, ref = o.T, ref.T
    err, size = np.linalg.norm(o - ref, axis=1), np.linalg.norm(ref, axis=1)
    tol = 5 * np.sqrt(ref.shape[1]) * 2.0 ** -40 + 2.0 ** -19 * size
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("m,n", [(64, 512), (24, 3000), (200, 520)])
def test_one_row_far_above_the_others(m, n):
    u = randn((m, n), 3)
    u[5] *= 1e5
    o = f64(bmoe.orthogonalize(u.cuda(), bmoe.OrthoSpec(1)))
    ref = O.newton_schulz(f64(u), 1)
    err, size = np.linalg.norm(o - ref, axis=1), np.linalg.norm(ref, axis=1)
    assert (err <= 5 * np.sqrt(n) * 2.0 ** -40 + 2.0 ** -19 * size).all()


# Coefficients up to the range's ends: whatever scales they leave, no operand passes
# fp16. A polynomial of these entries is at most 15 in Q and 3.87 in X: the errors are
# those of the scales 2^12 and up, relative to the whole matrix.
@pytest.mark.parametrize("steps,coeffs", [(1, (14.9, 0.0, 0.0)), (2, (3.8, 0.0, 0.0)),
                                          (1, (0.0, 0.0, 14.9)), (3, (1.9, 0.0, -0.4)),
                                          (2, (0.02, 0.01, 0.0)), (1, (-14.0, 28.0, -14.0))])
@pytest.mark.parametrize("shape", [(40, 72), (16, 1500), (130, 200), (200, 130)])
def test_coefficients_at_the_range(shape, steps, coeffs):
    # one singular value is nearly all of the matrix: as near to 1 as it can be
    u = randn((shape[0], 1), 4) @ randn((1, shape[1]), 5) + 1e-2 * randn(shape, 6)
    spec = bmoe.OrthoSpec(steps, coeffs)
    o = f64(bmoe.orthogonalize(u.cuda(), spec))
    ref = O.newton_schulz(f64(u), steps, coeffs)
    assert np.isfinite(o).all()
    # each step: operands of 2^-22 with terms of up to |a| + |b| + |c| times the iterate
    grow = np.prod([max(1.0, sum(abs(c) for c in coeffs))] * steps)
    assert np.linalg.norm(o - ref) <= 2.0 ** -19 * steps * grow * max(1.0, np.linalg.norm(ref))


def amplified(u, steps, a=3.4445, b=-4.7750, c=2.0315):
    """How much of one step's relative error the whole iteration can make: an odd
    polynomial of a matrix moves a small change by its divided differences between the
    singular values and their negatives."""
    s = np.linalg.svd(u, compute_uv=False)
    s = s / np.sqrt(np.sum(s * s))
    total = 0.0
    for _ in range(steps):
        p = a * s + b * s ** 3 + c * s ** 5
        x, y = np.concatenate([s, -s]), np.concatenate([p, -p])
        dx, dy = x[:, None] - x[None], y[:, None] - y[None]
        slope = a + 3 * b * x ** 2 + 5 * c * x ** 4
        near = np.abs(dx) < 1e-9
        grow = np.abs(np.where(near, slope[:, None], dy / np.where(near, 1.0, dx))).max()
        total = (total * grow * np.linalg.norm(s) + np.linalg.norm(p)) / np.linalg.norm(p)
        s = p
    return total


# A step's own error is below 2^-19 of the result (three products of 22-bit operands,
# coefficients of up to 4.8, fp32 sums); later steps amplify it as far as these
# singular values let them, 30 to 100 times in all.
@pytest.mark.parametrize("shape", [(64, 512), (512, 64), (32, 900), (24, 3000), (130, 520),
                                   (520, 130), (300, 260)])
def test_five_steps_in_the_norm(shape):
    u = randn(shape, sum(shape))
    o, ref = f64(bmoe.orthogonalize(u.cuda())), O.newton_schulz(f64(u))
    assert np.linalg.norm(o - ref) <= 2.0 ** -19 * amplified(f64(u), 5) * np.linalg.norm(ref)
