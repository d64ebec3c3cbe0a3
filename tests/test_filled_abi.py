"""The calls that set rows of no group to 0: refusals and grids (CPU)."""
import shutil

import pytest

from butterfly_rotated_ternary_amd import bmoe
from test_block_abi import at, spec
from test_block_launches import LOTS, TOP, at as far, record

BF, F32 = bmoe.BMOE_BF16, bmoe.BMOE_F32


def test_refusals_are_those_of_the_plain_calls():
    L = bmoe.lib()
    assert L.bmoe_grouped_product_filled(BF, 8, 16, 24, 4, None, 5, at(1), 2, at(2), at(3), at(4), None) == 1
    assert L.bmoe_grouped_product_filled(BF, 8, 0, 24, 4, at(0), 5, at(1), 2, at(2), at(3), at(4), None) == 2
    assert L.bmoe_grouped_product_filled(BF, 8, 16, 24, 4, at(0), 5, at(1), 2, at(2), at(3), at(0), None) == 9
    big = bmoe.bmoe_grouped_product_backward_workspace_bytes(BF, 8, 16, 24, 4)
    args = [BF, 8, 16, 24, 4, at(0), 5, at(1), 2, at(2), at(3), at(4), at(5), at(6), at(7)]
    assert L.bmoe_grouped_product_backward_filled(*args, big - 1, None) == 6
    args[12] = at(4)
    assert L.bmoe_grouped_product_backward_filled(*args, big, None) == 9


def test_norm_gradient_needs_room_for_its_marks():
    n, more = bmoe.bmoe_residual_norm_backward_workspace_bytes, bmoe.bmoe_residual_norm_backward_filled_workspace_bytes
    assert more(5, 4, 16, 8) == 0 and more(BF, 4, 8193, 8) == 0 and more(BF, 4, 16, -1) == 0
    assert more(BF, 4, 16, 1000) >= n(BF, 4, 16) + 4000
    assert more(BF, 4, 16, TOP) >= n(BF, 4, 16) + 4 * TOP

    def call(u_rows=1000, u=at(0), du=at(8), wb=more(BF, 4, 16, 1000), T=4):
        return bmoe.lib().bmoe_residual_norm_backward_filled(
            BF, T, 16, 2, spec(), u, u_rows, at(1), at(2), at(3), at(4), at(5), at(6), at(7), du,
            at(9), at(10), at(11), at(12), at(20), wb, None)
    assert call(wb=more(BF, 4, 16, 1000) - 1) == 6 and call(wb=n(BF, 4, 16)) == 6
    assert call(u_rows=-1) == 2 and call(u_rows=-1, u=None, T=0) == 2
    assert call(du=at(20) + more(BF, 4, 16, 1000) - 16) == 9      # du among the marks


@pytest.mark.skipif(not shutil.which("g++"), reason="g++ not available")
def test_grids(tmp_path):
    """Room for tiles of rows before and behind the groups, and legal at the largest."""
    def product(name, M, O, G, *more):
        return f"bmoe_grouped_product{name}", [BF, M, 64, O, G, far(0), M, far(1), 1, far(2), far(3),
                                               *more, None]

    def norm(T, d, k, rows, **kw):
        p = dict(inv=far(1), g=far(2), dpost=far(11), dpre=far(12))
        p.update(kw)
        return "bmoe_residual_norm_backward_filled", [
            BF, T, d, k, "norm", far(0), rows, p["inv"], p["g"], far(3), far(4), far(5), far(6), far(7),
            far(8), far(9) if p["g"] else None, far(10), p["dpost"], p["dpre"], far(13), LOTS, None]
    calls = [product("", 5000, 4096, 7, far(4)), product("_filled", 5000, 4096, 7, far(4)),
             product("_filled", TOP, 8, 1, far(4)),
             product("_backward_filled", TOP, 8, 4096, far(4), far(5), far(6), far(7), LOTS),
             norm(TOP, 1, 1, TOP), norm(1 << 23, 8192, 2, 1 << 24), norm(8, 2048, 2, 16),
             norm(8, 2048, 2, 16, dpost=None, dpre=None)]
    got = record(calls, str(tmp_path))
    for call, (status, launches) in zip(calls, got):
        assert status == 0 and launches and all(x.legal() for x in launches), (call, launches)
    plain, filled = got[0][1][0], got[1][1][0]
    assert filled.workgroups >= plain.workgroups
    assert [x.grid[1] for x in got[6][1]][-1] == 3 and len(got[7][1]) == 2
