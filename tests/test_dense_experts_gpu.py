"""Rows grouped by expert and their products on the GPU against the fp64 oracle.

Tolerances, per entry: one rounding of the result to its type (half a step,
bf16 2^-8 relative), and for the fp32 sum of n products at most n + 1 roundings
of 2^-24 each, doubled for matrix instructions that may truncate:
2^-23 (n + 1) times the sum of the products' magnitudes."""
import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half(dt):
    return 2.0 ** -8 if dt == BF else 2.0 ** -24


def close(got, ref, mag, n, dt, rows=slice(None)):
    err = np.abs(f64(got)[rows] - ref[rows])
    tol = half(dt) * np.abs(ref[rows]) + 2.0 ** -23 * (n + 1) * mag[rows]
    worst = float((err - tol).max(initial=-1.0))
    assert worst <= 0, (worst, float(err.max()))


def draw(T, K, O_, N, k, dt, seed=0, skew=0.0, pad=0.0):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(T, N, generator=g).clamp_(1e-6, 1 - 1e-6)
    ids = torch.topk(-torch.log(-torch.log(u)) - skew * torch.log1p(torch.arange(N).float()), k,
                     dim=1).indices.int()
    if pad:
        ids[torch.rand(T, k, generator=g) < pad] = -1 if N % 2 else N
    a = torch.randn(T, K, generator=g).to(dt)
    w = (torch.randn(N, O_, K, generator=g) / K ** 0.5).to(dt)
    dc = torch.randn(T * k, O_, generator=g).to(dt)
    return ids, a, w, dc


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 256), (5, 2, 3), (683, 3, 7), (1024, 2, 64),
                                   (1025, 2, 64), (4099, 6, 60), (32768, 8, 256), (300, 7, 4096)])
@pytest.mark.parametrize("pad", [0.0, 0.3])
def test_group_rows(T, k, N, pad):
    ids = draw(T, 1, 1, N, k, F32, seed=T, skew=0.5, pad=pad)[0]
    got = bmoe.group_rows(ids.cuda(), N)
    for name, x, y in zip(("offsets", "perm", "inv"), got, O.group_rows(ids.numpy(), N)):
        assert np.array_equal(x.cpu().numpy(), y), name


def test_group_rows_of_nothing_and_of_one_expert():
    off, perm, inv = bmoe.group_rows(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert not off.any() and off.numel() == 6 and perm.numel() == inv.numel() == 0
    ids = torch.full((3000, 1), 4, dtype=torch.int32, device="cuda")
    off, perm, inv = bmoe.group_rows(ids, 5)
    assert off.tolist() == [0, 0, 0, 0, 0, 3000]
    assert torch.equal(perm, torch.arange(3000, dtype=torch.int32, device="cuda"))
    assert torch.equal(perm, inv)
    off, _, inv = bmoe.group_rows(ids + 1, 5)
    assert not off.any() and (inv == -1).all()


SHAPES = [  # T, K, O, N, k, skew: ragged, odd and empty groups, one row to many tiles
    (1, 64, 32, 4, 1, 0.0), (1, 2048, 264, 32, 8, 0.0), (3, 8, 8, 8, 2, 0.0), (7, 1, 1, 3, 2, 0.0),
    (16, 100, 203, 5, 3, 0.0), (33, 33, 31, 2, 2, 1.1), (130, 136, 120, 3, 2, 0.5),
    (257, 512, 640, 6, 2, 1.1), (1003, 100, 203, 60, 3, 1.1), (700, 72, 1000, 2, 1, 0.0),
    (2100, 264, 128, 1, 1, 0.0), (90, 1024, 96, 70, 5, 0.0), (515, 250, 130, 4, 4, 0.4),
]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,K,O_,N,k,skew", SHAPES)
def test_product_and_gradients(T, K, O_, N, k, skew, dt):
    ids, a, w, dc = draw(T, K, O_, N, k, dt, seed=T + K, skew=skew, pad=0.2 if T > 20 else 0.0)
    off, perm, inv = O.group_rows(ids.numpy(), N)
    dev = [torch.from_numpy(x).cuda() for x in (off, perm)]
    A, W, D = f64(a), f64(w), f64(dc)
    rows, end = perm // k, off[-1]
    out = torch.full((T * k, O_), 7.0, dtype=dt, device="cuda")
    c = bmoe.grouped_product(a.cuda(), w.cuda(), dev[0], perm=dev[1], k=k, out=out)
    ref = O.grouped_product(A, W, off, rows)
    mag = O.grouped_product(np.abs(A), np.abs(W), off, rows)
    close(c, ref, mag, K, dt, slice(0, end))
    assert (out[end:] == 7.0).all()          # padded picks belong to no group
    da = torch.full((T * k, K), 7.0, dtype=dt, device="cuda")
    g = bmoe.grouped_product_backward(a.cuda(), w.cuda(), dev[0], dc.cuda(), perm=dev[1], k=k, da=da)
    rda, rdw = O.grouped_product_backward(A, W, off, rows, D)
    mda, mdw = O.grouped_product_backward(np.abs(A), np.abs(W), off, rows, np.abs(D))
    close(g["da"], rda, mda, O_, dt, slice(0, end))
    assert (da[end:] == 7.0).all()
    most = int(np.diff(off).max())
    close(g["dw"], rdw, mdw, most, F32)
    for e in np.flatnonzero(np.diff(off) == 0):
        assert not g["dw"][e].any()
    again = bmoe.grouped_product_backward(a.cuda(), w.cuda(), dev[0], dc.cuda(), perm=dev[1], k=k)
    assert torch.equal(again["dw"], g["dw"])


@pytest.mark.parametrize("dt", [BF, F32])
def test_groups_of_given_rows(dt):
    """Without perm: groups that begin behind row 0, end before the last row, and
    tiles that end inside a group; NaN in rows of no group goes nowhere."""
    g = torch.Generator().manual_seed(5)
    M, K, O_ = 900, 96, 160
    off = torch.tensor([3, 3, 132, 133, 133, 700, 861], dtype=torch.int32)
    a, w = torch.randn(M, K, generator=g).to(dt), (torch.randn(6, O_, K, generator=g) / 10).to(dt)
    dc = torch.randn(M, O_, generator=g).to(dt)
    for t in (a, dc):
        t[:3] = float("nan")
        t[861:] = float("inf")
    rows, o = np.arange(M), off.numpy()
    inside = slice(3, 861)
    c = bmoe.grouped_product(a.cuda(), w.cuda(), off.cuda(),
                             out=torch.full((M, O_), 7.0, dtype=dt, device="cuda"))
    A, W, D = f64(a), f64(w), f64(dc)
    close(c, O.grouped_product(A, W, o, rows), O.grouped_product(abs(A), abs(W), o, rows), K, dt, inside)
    assert (c[:3] == 7.0).all() and (c[861:] == 7.0).all()
    r = bmoe.grouped_product_backward(a.cuda(), w.cuda(), off.cuda(), dc.cuda())
    rda, rdw = O.grouped_product_backward(A, W, o, rows, D)
    mda, mdw = O.grouped_product_backward(abs(A), abs(W), o, rows, abs(D))
    close(r["da"], rda, mda, O_, dt, inside)
    close(r["dw"], rdw, mdw, 600, F32)


def test_bad_offsets_and_rows_stay_in_bounds():
    """Offsets outside [0, M] and rows outside a are clamped: nothing is read or
    written outside, and groups with good rows are right."""
    off = torch.tensor([-5, 40, 30, 1000, 2000], dtype=torch.int32)
    perm = torch.arange(200, dtype=torch.int32)
    perm[150:] = 1 << 30
    perm[160:] = -7
    g = torch.Generator().manual_seed(6)
    a, w = torch.randn(100, 64, generator=g).to(BF), torch.randn(4, 48, 64, generator=g).to(BF)
    c = bmoe.grouped_product(a.cuda(), w.cuda(), off.cuda(), perm=perm.cuda(), k=2)
    ref = f64(a)[perm[:30] // 2] @ f64(w)[0].T
    mag = abs(f64(a)[perm[:30] // 2]) @ abs(f64(w)[0].T)
    close(c[:30], ref, mag, 64, BF)
    r = bmoe.grouped_product_backward(a.cuda(), w.cuda(), off.cuda(),
                                      torch.zeros(200, 48, dtype=BF, device="cuda"),
                                      perm=perm.cuda(), k=2)
    assert not r["dw"].any()


def test_no_rows():
    w = torch.randn(3, 8, 16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = torch.empty(0, 16, device="cuda")
    assert bmoe.grouped_product(a, w, off).shape == (0, 8)
    r = bmoe.grouped_product_backward(a, w, off, torch.empty(0, 8, device="cuda"))
    assert r["da"].shape == (0, 16) and not r["dw"].any()
    r = bmoe.grouped_product_backward(torch.ones(5, 16, device="cuda"), w, off,
                                      torch.ones(5, 8, device="cuda"))
    assert not r["dw"].any()


@pytest.mark.parametrize("dt", [BF, F32])
def test_large_tiles_many_rows(dt):
    """Groups of several tiles with a reduction of many K-steps."""
    ids, a, w, dc = draw(1500, 1024, 520, 4, 2, dt, seed=9, skew=0.6)
    off, perm, inv = bmoe.group_rows(ids.cuda(), 4)
    c = bmoe.grouped_product(a.cuda(), w.cuda(), off, perm=perm, k=2)
    r = bmoe.grouped_product_backward(a.cuda(), w.cuda(), off, dc.cuda(), perm=perm, k=2)
    o, rows = off.cpu().numpy(), perm.cpu().numpy() // 2
    A, W, D = f64(a), f64(w), f64(dc)
    close(c, O.grouped_product(A, W, o, rows), O.grouped_product(abs(A), abs(W), o, rows), 1024, dt)
    rda, rdw = O.grouped_product_backward(A, W, o, rows, D)
    mda, mdw = O.grouped_product_backward(abs(A), abs(W), o, rows, abs(D))
    close(r["da"], rda, mda, 520, dt)
    close(r["dw"], rdw, mdw, int(np.diff(o).max()), F32)


# Tiles 256 columns wide at every height (64 to 256 rows, and groups of several),
# of 128 columns, aligned and not; gradients of 256 x 256 and 128 x 128 entries
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,K,O_,N,k,skew", [(4110, 520, 1032, 60, 2, 0.3), (2050, 200, 1000, 16, 2, 0.2),
                                             (2050, 201, 1000, 16, 2, 0.2),
                                             (4110, 264, 259, 40, 2, 0.3)])
def test_every_tile(T, K, O_, N, k, skew, dt):
    ids, a, w, dc = draw(T, K, O_, N, k, dt, seed=K, skew=skew)
    off, perm, inv = bmoe.group_rows(ids.cuda(), N)
    c = bmoe.grouped_product(a.cuda(), w.cuda(), off, perm=perm, k=k)
    r = bmoe.grouped_product_backward(a.cuda(), w.cuda(), off, dc.cuda(), perm=perm, k=k)
    o, rows = off.cpu().numpy(), perm.cpu().numpy() // k
    A, W, D = f64(a), f64(w), f64(dc)
    close(c, O.grouped_product(A, W, o, rows), O.grouped_product(abs(A), abs(W), o, rows), K, dt)
    rda, rdw = O.grouped_product_backward(A, W, o, rows, D)
    mda, mdw = O.grouped_product_backward(abs(A), abs(W), o, rows, abs(D))
    close(r["da"], rda, mda, O_, dt)
    close(r["dw"], rdw, mdw, int(np.diff(o).max()), F32)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 65, 133])
@pytest.mark.parametrize("O_", [1, 3, 5, 7, 9, 66, 131])
def test_short_and_odd_rows(K, O_, dt):
    """Rows shorter than 16 bytes and rows that end inside 16 bytes, each in an
    array that ends with its last row, among NaN that no product may touch."""
    N, M = 3, 150
    ids, a, w, dc = draw(M, K, O_, N, 1, dt, seed=K * O_)
    off, perm, inv = bmoe.group_rows(ids.cuda(), N)
    o, rows = off.cpu().numpy(), perm.cpu().numpy()
    A, W, D = f64(a), f64(w), f64(dc)

    def between(t):  # the same rows between NaN, at 16 bytes
        flat = torch.full((t.numel() + 128,), float("nan"), dtype=dt, device="cuda")
        v = flat[64:64 + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    x, y, z = between(a), between(w), between(dc)
    c = bmoe.grouped_product(x, y, off, perm=perm)
    close(c, O.grouped_product(A, W, o, rows), O.grouped_product(abs(A), abs(W), o, rows), K, dt)
    r = bmoe.grouped_product_backward(x, y, off, z, perm=perm)
    rda, rdw = O.grouped_product_backward(A, W, o, rows, D)
    mda, mdw = O.grouped_product_backward(abs(A), abs(W), o, rows, abs(D))
    close(r["da"], rda, mda, O_, dt)
    close(r["dw"], rdw, mdw, int(np.diff(o).max()), F32)


@pytest.mark.parametrize("N", [959, 960, 961, 962, 963, 3273, 3274, 3275, 3276])
@pytest.mark.parametrize("M", [2049, 8192, 8193, 20000])
def test_group_rows_of_many_experts(M, N):
    """Around the counts of experts and ids where the launches change."""
    g = torch.Generator().manual_seed(N)
    ids = torch.randint(-1, N + 1, (M, 1), generator=g, dtype=torch.int32)
    got = bmoe.group_rows(ids.cuda(), N)
    for name, x, y in zip(("offsets", "perm", "inv"), got, O.group_rows(ids.numpy(), N)):
        assert np.array_equal(x.cpu().numpy(), y), name
