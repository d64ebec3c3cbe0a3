"""Calls with the largest token counts that the header takes are launched with
grids that HIP takes (CPU only: launches are recorded, none is made). HIP
refuses a grid dimension of 2^32 or more threads, and a call that fails there
may have enqueued its first kernels already."""
import shutil

import pytest

from butterfly_rotated_ternary_amd import bmoe
from launches import record
from range_cases import CASES as RANGES

BF, F32 = bmoe.BMOE_BF16, bmoe.BMOE_F32
A, LOTS = 1 << 40, 1 << 62  # an aligned address; more workspace than any call asks for
TOP = 2 ** 31 - 1
DENSE, SPARSE = dict(score="softmax", renorm=False), dict(score="sigmoid", renorm=True)

pytestmark = pytest.mark.skipif(not shutil.which("g++"), reason="g++ not available")


def logits(dt, T, d, N):
    return "bmoe_router_logits", [dt, T, d, N, A, A, A, None]


def router(dt, T, d, N, k):
    return "bmoe_router", [dt, T, d, N, k, A, A, A, A, A, A, LOTS, None]


def route(dt, T, N, k, spec):
    return "bmoe_route", [dt, T, N, k, spec, A, None, A, A, None]


def route_bwd(dt, T, N, k, spec):
    return "bmoe_route_backward", [dt, T, N, k, spec, A, A, A, A, None]


def router_bwd(dt, T, d, N, k, spec):
    return "bmoe_router_backward", [dt, T, d, N, k, spec, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A,
                                    7 * A, 8 * A, 9 * A, LOTS, None]


def groups(n, keep):
    return dict(score="sigmoid", n_groups=n, topk_groups=keep)


# (call, workgroups that the first launches need at least); tokens per
# workgroup of the kernels: 16 where 16 lanes take one, 4 where a wave does
CASES = [
    (route(F32, TOP, 1, 1, SPARSE), [TOP // 16]),
    (route(BF, (1 << 27) - 1, 17, 16, SPARSE), [1 << 23]),
    (route(BF, (1 << 26) + 3, 33 * 66, 4, groups(33, 4)), [1 << 24]),
    (route_bwd(F32, (1 << 28) - 1, 4, 1, SPARSE), [1 << 24]),
    (route_bwd(F32, 1 << 28, 4, 1, SPARSE), [1 << 24]),
    (route_bwd(F32, TOP, 1, 1, DENSE), [TOP // 16]),
    (route_bwd(BF, 1 << 26, 17, 17, SPARSE), [1 << 24]),
    (route_bwd(F32, TOP // 64, 300, 64, DENSE), [TOP // 256]),
    # picks only: pairs, lists, then the products of both roles (16 bytes a thread), join
    (router_bwd(F32, (1 << 26) + 1, 16, 17, 17, SPARSE), [1 << 24, 1 << 16, 1 << 20]),
    (router_bwd(BF, 1 << 24, 2048, 8, 1, SPARSE), [1 << 14, 1 << 24]),
    (router_bwd(BF, (1 << 24) - 5, 4096, 256, 2, SPARSE), [1 << 14, 1 << 25]),
    (router_bwd(F32, 1 << 23, 2048, 8, 4, SPARSE), [1 << 17, 1 << 13, 1 << 24]),
    # dense: dl, then dx in 64-token tiles
    (router_bwd(F32, 1 << 30, 16, 1, 1, DENSE), [1 << 26, 1 << 24]),
    (router_bwd(F32, TOP, 16, 1, 1, DENSE), [TOP // 16, TOP // 64]),
    (router_bwd(BF, 1 << 28, 16, 4, 1, DENSE), [1 << 24, 1 << 22]),
    (logits(F32, 1 << 30, 16, 1), [1 << 24]),
    (logits(F32, TOP, 16, 70), [2 * (TOP // 64)]),
    (logits(BF, TOP, 16, 1), [TOP // 32]),
    (logits(BF, TOP, 64, 65), [TOP // 128]),
    (router(F32, 1 << 26, 16, 8, 2), [1 << 20, 1 << 24]),
    (router(BF, TOP // 2, 64, 16, 2), [TOP // 256, TOP // 8]),
]


@pytest.fixture(scope="module")
def recorded(tmp_path_factory):
    return record([c for c, _ in CASES], tmp_path_factory.mktemp("launches"))


@pytest.mark.parametrize("i", range(len(CASES)), ids=lambda i: f"{CASES[i][0][0]}-{i}")
def test_largest_calls_have_legal_grids(i, recorded):
    (name, args), need = CASES[i]
    status, ls = recorded[i]
    assert status == 0 and len(ls) >= len(need)
    for l in ls:
        assert l.legal(), (name, args[:5], l)
    for l, n in zip(ls, need):
        # all of them there, and no more than the rows' last one left over
        assert n <= l.workgroups, (name, args[:5], l, n)


def spans(T, d, N, k, e, ws):
    """Bytes of the router backward's tensors, in the order of its pointers."""
    return dict(x=T * d * e, w=N * d * e, logits=4 * T * N, ids=4 * T * k, dgates=4 * T * k,
                dx_add=T * d * e, dx=T * d * e, dw=4 * N * d, ws=ws)


@pytest.mark.parametrize("dt", [BF, F32])
def test_router_backward_refuses_shared_memory(dt, tmp_path):
    """What is written (dx, dw, the workspace) shares no byte with another
    tensor; the exception is dx_add, which dx may be. Nothing is launched."""
    T, d, N, k = 40, 64, 8, 2
    size = spans(T, d, N, k, 2 if dt == BF else 4,
                 bmoe.bmoe_router_backward_workspace_bytes(dt, T, d, N, k))
    names = list(size)
    far = {n: A + (i << 30) for i, n in enumerate(names)}
    calls, want = [], []

    def add(status, **moved):
        p = {**far, **moved}
        calls.append(("bmoe_router_backward", [dt, T, d, N, k, SPARSE, *(p[n] for n in names),
                                               size["ws"], None]))
        want.append(status)

    add(0)
    add(0, dx_add=far["dx"])
    add(0, dx_add=None)
    add(0, w=far["x"])                                   # both only read
    for a in ("dx", "dw", "ws"):
        for b in names:
            if a == b:
                continue
            first = far[b] + size[b] // 16 * 16 - 16     # b's last 16 bytes
            add(9, **{a: first})
            add(9, **{a: far[b] - size[a] // 16 * 16 + 16})
            add(0, **{a: far[b] + (size[b] + 15) // 16 * 16})
            add(0, **{a: far[b] - (size[a] + 15) // 16 * 16})
            if (a, b) != ("dx", "dx_add"):
                add(9, **{a: far[b]})
    got = record(calls, tmp_path)
    assert [s for s, _ in got] == want
    assert all(len(l) >= 2 if s == 0 else not l for (s, l) in got)


def test_long_ranges_take_the_paths_that_their_cases_name(tmp_path):
    """The shapes whose results the GPU tests compare run the launches meant."""
    got = record([router_bwd(dt, *c[:4], SPARSE) for c in RANGES for dt in (BF, F32)], tmp_path)
    for i, (status, ls) in enumerate(got):
        T, d, N, k, threads, ranges, pairs = RANGES[i // 2]
        groups_ = (ranges + 3) // 4
        assert status == 0
        assert len(ls) == pairs + 2 + (groups_ > 1), (RANGES[i // 2], ls)
        lists = ls[pairs]
        assert (lists.workgroups, lists.block[0]) == (ranges, threads), (RANGES[i // 2], ls)


def test_norm_streams_by_the_bytes_of_the_whole_list(tmp_path):
    """A list above 256 MB does not fit the last-level cache until the scaling
    reads it, however many tables of 112 tensors it takes."""
    def norm(counts):
        tensors = [[A + (i << 32), n, F32] for i, n in enumerate(counts)]
        return "bmoe_grad_norm", [len(tensors), tensors, A, A, LOTS, None]

    one_big, one_small = [70 << 20], [60 << 20] + [4] * 20
    got = record([norm(one_big), norm(one_small), norm([1 << 20] * 300), norm([1 << 17] * 300),
                  norm([100] * 112 + [70 << 20]), norm([100] * 9)], tmp_path)
    assert all(s == 0 for s, _ in got)
    big, small, many_big, many_small, mixed, few = ([l.kernel for l in ls[:-1]] for _, ls in got)
    assert len(big) == 1 and len(small) == 1 and big != small and few == small
    assert many_big == big * 3 and mixed == big * 2
    assert set(many_small) == set(small)
