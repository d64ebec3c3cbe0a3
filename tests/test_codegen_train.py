"""The training-step kernels that are bound by memory or the matrix units do
not spill in the generated gfx950 code (CPU only: compiles the sources to AMD
assembly). A spill's reload is a vector-memory operation in their load
streams."""
import pytest

from test_codegen import _asm, _functions, _kernels, pytestmark  # noqa: F401


@pytest.mark.parametrize("src,names", [
    ("grads.hip", ["grad_sq_kernel", "grad_scale_kernel"]),
    ("route.hip", ["route_kernel", "route_bwd_kernel", "route_exact_kernel"]),
    ("router_bwd.hip", ["router_sparse_kernel", "router_dx_mfma_kernel", "router_dw_mfma_kernel",
                        "router_dx_f32_kernel", "router_dw_f32_kernel"]),
])
def test_kernels_do_not_spill(src, names, tmp_path):
    funcs = _functions(_asm(src, tmp_path))
    for name in names:
        for k, ins in _kernels(funcs, name).items():
            assert not any(s.startswith("scratch_") for s in ins), k


def test_dense_dw_leaves_the_next_step_in_flight(tmp_path):
    """Inside its loop the kernel waits for all but the newest step's seven
    loads, never for all of them."""
    import re
    funcs = _functions(_asm("router_bwd.hip", tmp_path))
    for k, ins in _kernels(funcs, "router_dw_mfma_kernel").items():
        first = next(i for i, s in enumerate(ins) if s.startswith("v_mfma"))
        last = max(i for i, s in enumerate(ins) if s.startswith("v_mfma"))
        waits = [int(m.group(1)) for s in ins[first:last]
                 for m in [re.match(r"s_waitcnt.*vmcnt\((\d+)\)", s)] if m]
        assert waits and min(waits) >= 5, (k, waits)
