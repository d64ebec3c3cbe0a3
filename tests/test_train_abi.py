"""Host-side refusals of routing from logits, the router's backward, the
balance bias and the gradient lists: every one returns before any HIP call, so
they run without a GPU. Pointers are made-up addresses that nothing reads."""
import ctypes

import pytest
import torch

from butterfly_rotated_ternary_amd import bmoe

BF, F32 = bmoe.BMOE_BF16, bmoe.BMOE_F32
OK, NULL, SHAPE, DTYPE, WS, ALIGN, VALUE = 0, 1, 2, 3, 6, 8, 9
A = 0x10000  # an aligned address


def spec(**kw):
    s = bmoe.RouteSpec()
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def route(dt=F32, T=4, N=8, k=2, sp=None, logits=A, bias=None, ids=A, gates=A):
    return bmoe.lib().bmoe_route(dt, T, N, k, sp or spec(), logits, bias, ids, gates, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=7)), (SHAPE, dict(N=0)), (SHAPE, dict(N=4097)), (SHAPE, dict(k=0)),
    (SHAPE, dict(k=9)), (SHAPE, dict(N=200, k=65)), (SHAPE, dict(T=-1)),
    (SHAPE, dict(T=1 << 30, k=2)), (OK, dict(T=0, logits=None)), (NULL, dict(logits=None)),
    (NULL, dict(ids=None)), (NULL, dict(gates=None)), (ALIGN, dict(logits=A + 4)),
    (ALIGN, dict(bias=A + 4)), (ALIGN, dict(ids=A + 8)), (ALIGN, dict(gates=A + 8)),
    (VALUE, dict(sp=spec(score=2))), (VALUE, dict(sp=spec(group_score=-1))),
    (VALUE, dict(sp=spec(scale=float("nan")))), (VALUE, dict(sp=spec(scale=float("inf")))),
    (VALUE, dict(sp=spec(n_groups=0))), (VALUE, dict(sp=spec(n_groups=3))),
    (VALUE, dict(N=130, sp=spec(n_groups=65))), (VALUE, dict(sp=spec(n_groups=4, topk_groups=0))),
    (VALUE, dict(sp=spec(n_groups=4, topk_groups=5))),
    (VALUE, dict(k=3, sp=spec(n_groups=4, topk_groups=1))),
])
def test_route_refuses(want, kw):
    assert route(**kw) == want


def test_route_needs_a_spec():
    assert bmoe.lib().bmoe_route(F32, 4, 8, 2, None, A, None, A, A, None) == NULL


def test_route_backward_refuses():
    def call(dt=F32, T=4, N=8, k=2, sp=None, p=(A, A, A, A)):
        return bmoe.lib().bmoe_route_backward(dt, T, N, k, sp or spec(), *p, None)
    assert call(dt=5) == DTYPE
    assert call(k=9) == SHAPE
    assert call(sp=spec(score=9)) == VALUE
    assert call(T=0, p=(None,) * 4) == OK
    for i in range(4):
        assert call(p=[None if j == i else A for j in range(4)]) == NULL
        assert call(p=[A + 4 if j == i else A for j in range(4)]) == ALIGN


def test_balance_refuses():
    n = bmoe.bmoe_route_balance_workspace_bytes
    assert n(4, 0, 2) == 0 and n(4, 4097, 2) == 0 and n(-1, 8, 2) == 0 and n(1 << 30, 8, 2) == 0
    assert n(4, 8, 2) > 0 and n(0, 8, 2) > 0
    big = n(4, 8, 2)

    def call(T=4, N=8, k=2, ids=A, rate=0.1, load=A, bias=A, ws=A, wb=big):
        return bmoe.lib().bmoe_route_balance(T, N, k, ids, 0, rate, load, bias, ws, wb, None)
    assert call(N=0) == SHAPE and call(k=0) == SHAPE and call(T=-1) == SHAPE
    assert call(ids=None) == NULL and call(load=None) == NULL
    assert call(rate=float("nan")) == VALUE and call(rate=float("inf")) == VALUE
    assert call(ws=None) == WS and call(wb=big - 1) == WS
    assert call(ids=A + 4) == ALIGN and call(load=A + 4) == ALIGN and call(bias=A + 4) == ALIGN


def test_router_backward_refuses():
    n = bmoe.bmoe_router_backward_workspace_bytes
    assert n(9, 4, 64, 8, 2) == 0 and n(F32, 4, 48, 8, 2) == 0 and n(F32, 4, 8, 8, 2) == 0
    assert n(F32, 4, 64, 8, 9) == 0 and n(F32, 4, 64, 128, 65) == 0
    big = n(BF, 4, 64, 8, 2)
    assert big > 0

    def call(dt=BF, T=4, d=64, N=8, k=2, sp=None, x=A, w=A, lg=A, ids=A, dg=A, add=None, dx=A,
             dw=A, ws=A, wb=big):
        return bmoe.lib().bmoe_router_backward(dt, T, d, N, k, sp or spec(), x, w, lg, ids, dg,
                                               add, dx, dw, ws, wb, None)
    B = A + 0x10000
    assert call(dt=3) == DTYPE and call(d=100) == SHAPE and call(N=0) == SHAPE
    assert call(sp=spec(n_groups=3)) == VALUE
    for name in ("x", "w", "lg", "ids", "dg", "dx", "dw"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: A + 8}) == ALIGN, name
    assert call(add=A + 8) == ALIGN
    assert call(ws=None) == WS and call(wb=16) == WS
    # dx on x, or on part of dx_add (4 x 64 bf16 values are 512 bytes)
    assert call() == VALUE and call(dx=B, x=B + 496) == VALUE and call(dx=B, x=B - 496) == VALUE
    assert call(dx=B, add=B + 256) == VALUE and call(dx=B, add=B - 496) == VALUE


def test_router_logits_refuses():
    f = bmoe.lib().bmoe_router_logits
    assert f(4, 4, 64, 8, A, A, A, None) == DTYPE
    assert f(F32, 4, 100, 8, A, A, A, None) == SHAPE
    assert f(F32, 4, 64, 4097, A, A, A, None) == SHAPE
    assert f(F32, 0, 64, 8, None, None, None, None) == OK
    assert f(F32, 4, 64, 8, None, A, A, None) == NULL
    assert f(F32, 4, 64, 8, A, A + 4, A, None) == ALIGN


def tensors(*entries):
    arr = (bmoe.BmoeTensor * max(1, len(entries)))()
    for e, (p, n, dt) in zip(arr, entries):
        e.data, e.count, e.dtype = p, n, dt
    return arr


def test_grad_lists_refuse():
    L = bmoe.lib()
    wb = bmoe.bmoe_grad_workspace_bytes(3)
    assert wb > 0 and bmoe.bmoe_grad_workspace_bytes(-1) == 0
    assert bmoe.bmoe_grad_workspace_bytes(0) > 0

    def clip(g, n=None, out=None, m=1.0, norm=A, ws=A, b=wb):
        return L.bmoe_grad_clip(len(g) if n is None else n, g, out, m, norm, ws, b, None)
    one = tensors((A, 100, F32))
    assert clip(one, n=-1) == SHAPE
    assert L.bmoe_grad_clip(1, None, None, 1.0, A, A, wb, None) == NULL
    assert clip(tensors((None, 4, F32))) == NULL
    assert clip(tensors((A, 4, 6))) == DTYPE
    assert clip(tensors((A + 2, 4, F32))) == ALIGN and clip(tensors((A + 1, 4, BF))) == ALIGN
    assert clip(tensors((A, 1 << 63, F32))) == SHAPE
    for m in (0.0, -1.0, float("nan")):
        assert clip(one, m=m) == VALUE
        assert L.bmoe_grad_scale(1, one, None, A, m, None) == VALUE
    assert clip(one, norm=None) == NULL and clip(one, norm=A + 2) == ALIGN
    assert clip(one, ws=None) == WS and clip(one, b=wb - 1) == WS and clip(one, ws=A + 8) == ALIGN
    assert L.bmoe_grad_scale(1, one, None, None, 1.0, None) == NULL
    assert L.bmoe_grad_norm(1, one, None, A, wb, None) == NULL
    assert L.bmoe_grad_norm(1, one, A, A, wb - 1, None) == WS
    # out: same types and counts
    assert clip(one, out=tensors((A, 100, BF))) == DTYPE
    assert clip(one, out=tensors((A, 99, F32))) == SHAPE
    assert clip(one, out=tensors((None, 100, F32))) == NULL
    assert clip(one, out=tensors((A + 1, 100, F32))) == ALIGN


def test_written_tensors_may_not_share_memory():
    """With ws too small the call stops right after these checks, so the
    accepted lists reach BMOE_E_WORKSPACE and nothing is launched."""
    def clip(g, out=None):
        return bmoe.lib().bmoe_grad_clip(len(g), g, out, 1.0, A, A, 1, None)
    B = A + 0x1000
    ok = tensors((B, 16, F32), (A, 0x400, F32), (B + 64, 16, BF), (None, 0, F32))
    assert clip(ok) == WS
    assert clip(tensors((A, 8, F32), (A, 8, F32))) == VALUE           # listed twice
    assert clip(tensors((A, 8, F32), (A + 28, 8, BF))) == VALUE       # last entry shared
    assert clip(tensors((A, 8, F32), (A + 32, 8, BF))) == WS
    two = tensors((A, 8, F32), (B, 8, F32))
    assert clip(two, tensors((A, 8, F32), (B, 8, F32))) == WS         # in place, spelled out
    assert clip(two, tensors((B, 8, F32), (A, 8, F32))) == VALUE      # swapped
    assert clip(two, tensors((A + 64, 8, F32), (A + 64, 8, F32))) == VALUE
    assert clip(two, tensors((A + 64, 8, F32), (B + 16, 8, F32))) == VALUE  # part of its own grad
    same = tensors((A, 8, F32), (A, 8, F32))
    assert clip(same, tensors((B, 8, F32), (B + 64, 8, F32))) == WS   # read twice, written apart
    # a long written span in front of several others
    assert clip(tensors((A, 100, F32), (A + 8, 1, F32), (A + 0x500, 1, F32))) == VALUE
    # the norm alone only reads: any sharing will do
    assert bmoe.lib().bmoe_grad_norm(2, same, A, A, 1, None) == WS


def test_wrappers_refuse_before_the_library():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        bmoe.RouteSpec("tanh")
    with pytest.raises(ValueError):
        bmoe.RouteSpec(group_score="mean")
    with pytest.raises(ValueError):
        bmoe.route_logits(x, 2)                 # on the CPU
    with pytest.raises(ValueError):
        bmoe.route_logits(x.t(), 2)             # strided
    with pytest.raises(TypeError):
        bmoe.route_logits(x.half(), 2)
    with pytest.raises(ValueError):
        bmoe.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        bmoe.clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        bmoe.clip_grads([x, x.t()], 1.0)
    with pytest.raises(ValueError):
        bmoe.router_backward(x, torch.zeros(5, 7), x, torch.zeros(4, 2, dtype=torch.int32),
                             torch.zeros(4, 2))


def test_workspace_sizes_at_the_largest_token_counts():
    """Sizes for token counts next to 2^31 neither wrap nor shrink."""
    n = bmoe.bmoe_router_backward_workspace_bytes
    top = 2 ** 31 - 1
    for dt in (BF, F32):
        last = 0
        for T in (1, 1000, 1 << 20, 1 << 30, top - 4096, top):
            got = n(dt, T, 16, 8, 1)
            assert got >= max(last, T * 8 * 4), (dt, T)
            last = got
    assert bmoe.bmoe_route_balance_workspace_bytes(top, 64, 1) >= 64 * 4
