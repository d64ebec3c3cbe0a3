"""The picks-only router gradient over long ranges of tokens: pairs in a launch
of their own, lists by sixteen waves or four, cursors carried over many blocks
of 64 picks, ranges that end early, and several groups of ranges. Experts are
picked with a strong skew, so that most blocks hold one many times."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from butterfly_rotated_ternary_amd import bmoe
from range_cases import CASES
from test_route_gpu import U, eps_of, grad_scale, rounded

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def skewed_ids(rng, T, N, k):
    """k experts a token, the low ids far more often, expert 3 by two tokens in
    three; some padded, some listed twice, a run of padded tokens."""
    ids = np.minimum(rng.geometric(8.0 / N, (T, k)) - 1, N - 1).astype(np.int32)
    spread = rng.random((T, k)) < 0.3
    ids[spread] = rng.integers(0, N, spread.sum())
    ids[rng.random(T) < 0.66, 0] = 3
    ids[rng.random((T, k)) < 0.02] = -1
    ids[rng.random((T, k)) < 0.01] = N + 3
    ids[T // 3:T // 3 + 100] = -1
    return ids


@pytest.mark.parametrize("T,d,N,k,threads,ranges,pairs", CASES)
@pytest.mark.parametrize("dt,spec", [("bf16", ("sigmoid", True)), ("bf16", ("softmax", True)),
                                     ("f32", ("sigmoid", False))], ids=str)
def test_long_ranges_match_oracle(T, d, N, k, threads, ranges, pairs, dt, spec):
    rng = np.random.default_rng(T + k)
    x_dev, x = rounded(rng.normal(0, 1, (T, d)), dt)
    w_dev, w = rounded(rng.normal(0, 1, (N, d)) / math.sqrt(d), dt)
    l_dev, l = rounded(rng.normal(0, 1, (T, N)), "f32")
    a_dev, a = rounded(rng.normal(0, 1, (T, d)), dt)
    ids = skewed_ids(rng, T, N, k)
    dg = rng.normal(0, 1, (T, k)).astype(np.float32)
    dg[rng.random((T, k)) < 0.05] = 0.0
    i_dev, g_dev = torch.from_numpy(ids).cuda(), torch.from_numpy(dg).cuda()
    sp = bmoe.RouteSpec(spec[0], renorm=spec[1], scale=1.5)
    print(f"[router_backward] T={T} d={d} N={N} k={k} {dt} {spec}", flush=True)
    out = bmoe.router_backward(x_dev, w_dev, l_dev, i_dev, g_dev, sp, dx_add=a_dev)
    again = bmoe.router_backward(x_dev, w_dev, l_dev, i_dev, g_dev, sp, dx_add=a_dev)
    assert torch.equal(out["dx"], again["dx"]) and torch.equal(out["dw"], again["dw"])
    # (in fp64 on the GPU: the products of these sizes)
    dl = O.route_logits_backward(l, ids, dg, score=spec[0], renorm=spec[1], scale=1.5)
    A = grad_scale(l, ids, dg, *spec, 1.5)
    E = 4 * eps_of(l)
    dl, A, E = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (dl, A, E))
    x64, w64, a64 = x_dev.double(), w_dev.double(), a_dev.double()
    # dx: k products and dx_add, in order
    want = dl @ w64 + a64
    tol = ((E + (k + 2) * U) * A) @ w64.abs() + (k + 2) * U * a64.abs()
    assert ((out["dx"].double() - want).abs() <= tol + HALF[dt] * (want.abs() + tol) + 2.0 ** -126).all()
    # dW: a wave adds its range's entries of an expert (narrow rows: up to eight
    # shares of them), these and the four waves' sums and then the groups' are
    # added in order
    tokens = 1 << (-(-T // ranges) - 1).bit_length()
    ok = (ids >= 0) & (ids < N)
    where = np.repeat(np.arange(T) // tokens, k).reshape(T, k)[ok] * N + ids[ok]
    chain = int(np.bincount(where).max()) + 4 * 8 + (ranges + 3) // 4
    want = dl.t().contiguous() @ x64
    tol = ((E + (chain + 2) * U) * A).t().contiguous() @ x64.abs()
    err = (out["dw"].double() - want).abs()
    assert (err <= tol + 2.0 ** -126).all(), float((err / (tol + 2.0 ** -126)).max())
