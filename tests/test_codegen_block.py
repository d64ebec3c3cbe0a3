"""The generated gfx950 code of the grouped and Newton-Schulz products keeps what
their counted waits rely on, and the kernels that are bound by memory or the
matrix units do not spill (CPU only: compiles the sources to AMD assembly)."""
import pytest

from test_codegen import _asm, _counted_waits, _functions, _kernels, pytestmark  # noqa: F401


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    out = {}

    def get(src):
        if src not in out:
            out[src] = _functions(_asm(src, tmp_path_factory.mktemp("asm")))
        return out[src]
    return get


@pytest.mark.parametrize("src,name", [("grouped.hip", "grouped_kernel"),
                                      ("grouped.hip", "grouped_dw_kernel"),
                                      ("norm.hip", "11norm_kernel"),
                                      ("group_rows.hip", "group_scatter_kernel")])
def test_kernels_do_not_spill(code, src, name):
    for k, ins in _kernels(code(src), name).items():
        assert not any(s.startswith("scratch_") for s in ins), k


@pytest.mark.parametrize("src,name", [("grouped.hip", "grouped_kernel"),
                                      ("grouped.hip", "grouped_dw_kernel"),
                                      ("ortho.hip", "ortho_product_kernel")])
def test_rings_count_only_dma(code, src, name):
    """The N newest vector-memory operations before a counted wait are the steps
    still in flight: DMA (a spill's among them would only wait for more)."""
    checked = 0
    for k, ins in _kernels(code(src), name).items():
        for n, ops in _counted_waits(ins):
            if not any("lds" in o for o in ops):
                continue  # rows that are not aligned: loads to registers, waited for by the compiler
            assert all(o == "global_load_lds_dwordx4" or o.startswith("scratch_") for o in ops), (k, n, ops)
            checked += 1
    assert checked > 0


def test_odd_rows_take_whole_accesses(code):
    """Rows that are no multiple of 16 bytes are read 16 bytes at a time too."""
    for src, name in (("norm.hip", "11norm_kernel"), ("grouped.hip", "grouped_kernel")):
        for k, ins in _kernels(code(src), name).items():
            assert any(s.startswith(("global_load_dwordx4", "global_load_lds_dwordx4")) for s in ins), k
