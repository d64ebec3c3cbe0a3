"""Thin ctypes binding of libbmoe.so (declared in include/bmoe.h).

Argument marshalling only: every step of the forward runs in the library's
HIP kernels. torch supplies device memory and the current stream. There is
no CPU fallback: if the library is missing, loading it raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbmoe.so")
_lib = None

BMOE_F32 = 0
BMOE_BF16 = 1
BMOE_E_TERNARY = 4
BMOE_E_EXPERT = 5

STATUS = {
    0: "BMOE_OK", 1: "BMOE_E_NULL", 2: "BMOE_E_SHAPE", 3: "BMOE_E_DTYPE",
    4: "BMOE_E_TERNARY", 5: "BMOE_E_EXPERT", 6: "BMOE_E_WORKSPACE", 7: "BMOE_E_HIP",
    8: "BMOE_E_ALIGN", 9: "BMOE_E_VALUE",
}

BMOE_SCORE_SOFTMAX = 0
BMOE_SCORE_SIGMOID = 1
BMOE_GROUP_MAX = 0
BMOE_GROUP_TOP2 = 1
_SCORES = {"softmax": BMOE_SCORE_SOFTMAX, "sigmoid": BMOE_SCORE_SIGMOID}
_GROUP_SCORES = {"max": BMOE_GROUP_MAX, "top2": BMOE_GROUP_TOP2}


class RouteSpec(ctypes.Structure):
    """bmoe_route_spec: how scores, groups and gates are formed."""
    _fields_ = [("score", ctypes.c_int), ("renorm", ctypes.c_int), ("scale", ctypes.c_float),
                ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int),
                ("group_score", ctypes.c_int)]

    def __init__(self, score: str = "softmax", *, renorm: bool = True, scale: float = 1.0,
                 n_groups: int = 1, topk_groups: int = 1, group_score: str = "top2"):
        if score not in _SCORES or group_score not in _GROUP_SCORES:
            raise ValueError("score is 'softmax' or 'sigmoid', group_score 'max' or 'top2'")
        super().__init__(_SCORES[score], bool(renorm), scale, n_groups, topk_groups,
                         _GROUP_SCORES[group_score])


class NormSpec(ctypes.Structure):
    """bmoe_norm_spec: r' = res_scale * r + out_scale * z, eps of both norms."""
    _fields_ = [("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("out_scale", ctypes.c_float)]

    def __init__(self, *, eps: float = 1e-6, res_scale: float = 1.0, out_scale: float = 1.0):
        super().__init__(eps, res_scale, out_scale)


class OrthoSpec(ctypes.Structure):
    """bmoe_ortho_spec: Newton-Schulz steps with the coefficients (a, b, c)."""
    _fields_ = [("steps", ctypes.c_int), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float)]

    def __init__(self, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), *, eps: float = 1e-7):
        super().__init__(steps, *coeffs, eps)


class OrthoUpdate(ctypes.Structure):
    """bmoe_ortho_update: the scalars of one orthogonal_step()."""
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float), ("nesterov", ctypes.c_int),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float)]


class BmoeTensor(ctypes.Structure):
    """bmoe_tensor: one entry of a gradient list."""
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_size_t), ("dtype", ctypes.c_int)]


class BmoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({lib().bmoe_status_str(code).decode()})")
        self.code = code


def lib():
    """Load libbmoe.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m butterfly_rotated_ternary_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        c_int, c_sz, vp, c_f = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
        L.bmoe_packed_words.argtypes = [c_int]
        L.bmoe_packed_words.restype = c_sz
        L.bmoe_param_count.argtypes = [c_int, c_int]
        L.bmoe_param_count.restype = c_sz
        L.bmoe_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_workspace_bytes.restype = c_sz
        L.bmoe_pack_workspace_bytes.argtypes = []
        L.bmoe_pack_workspace_bytes.restype = c_sz
        L.bmoe_pack_ternary.argtypes = [vp, c_int, vp, vp, c_sz, vp]
        L.bmoe_pack_ternary.restype = c_int
        L.bmoe_packed3_bytes.argtypes = [c_int]
        L.bmoe_packed3_bytes.restype = c_sz
        L.bmoe_pack_ternary_b3.argtypes = [vp, c_int, vp, vp, c_sz, vp]
        L.bmoe_pack_ternary_b3.restype = c_int
        L.bmoe_unpack_ternary_b3.argtypes = [vp, c_int, vp, vp, c_sz, vp]
        L.bmoe_unpack_ternary_b3.restype = c_int
        L.bmoe_unpack_ternary_b3_timed.argtypes = [vp, c_int, vp, vp, c_sz, vp, vp]
        L.bmoe_unpack_ternary_b3_timed.restype = c_int
        L.bmoe_forward.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp, c_f,
                                   vp, vp, c_sz, vp, vp]
        L.bmoe_forward.restype = c_int
        L.bmoe_forward_noalloc.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp,
                                           vp, c_f, vp, vp, vp, vp]
        L.bmoe_forward_noalloc.restype = c_int
        c_dp = ctypes.POINTER(ctypes.c_double)
        for name in ("bmoe_ceiling_mfma_bf16", "bmoe_ceiling_valu_f32"):
            getattr(L, name).argtypes = [c_int, vp, vp, vp, c_dp]
            getattr(L, name).restype = c_int
        L.bmoe_ceiling_copy.argtypes = [vp, vp, c_sz, vp, vp]
        L.bmoe_ceiling_copy.restype = c_int
        L.bmoe_product.argtypes = [c_int, c_int, vp, vp, c_int, c_f, vp, vp, vp]
        L.bmoe_product.restype = c_int
        L.bmoe_forward_timed.argtypes = L.bmoe_forward.argtypes + [vp]
        L.bmoe_forward_timed.restype = c_int
        L.bmoe_forward_kernel_count.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_forward_kernel_count.restype = c_int
        L.bmoe_forward_kernel_name.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
        L.bmoe_forward_kernel_name.restype = ctypes.c_char_p
        L.bmoe_sync_status.argtypes = [vp, vp]
        L.bmoe_sync_status.restype = c_int
        L.bmoe_status_str.argtypes = [c_int]
        L.bmoe_status_str.restype = ctypes.c_char_p
        L.bmoe_backward_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_backward_workspace_bytes.restype = c_sz
        L.bmoe_backward.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp,
                                    c_f, vp, vp, vp, vp, vp, vp, vp, c_sz, vp]
        L.bmoe_backward.restype = c_int
        L.bmoe_forward_keep_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_forward_keep_workspace_bytes.restype = c_sz
        L.bmoe_forward_keep.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp,
                                        vp, c_f, vp, vp, c_sz, vp]
        L.bmoe_forward_keep.restype = c_int
        L.bmoe_backward_kept.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, c_f, vp,
                                         vp, vp, vp, vp, vp, vp, c_sz, vp, c_sz, vp]
        L.bmoe_backward_kept.restype = c_int
        L.bmoe_backward_kept_timed.argtypes = L.bmoe_backward_kept.argtypes + [vp]
        L.bmoe_backward_kept_timed.restype = c_int
        L.bmoe_rotate_in_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_rotate_in_workspace_bytes.restype = c_sz
        L.bmoe_rotate_in.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, c_sz,
                                     vp]
        L.bmoe_rotate_in.restype = c_int
        L.bmoe_quant_error.argtypes = [c_int, c_int, c_int, vp, c_int, c_int, vp, vp, vp]
        L.bmoe_quant_error.restype = c_int
        L.bmoe_router_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_router_workspace_bytes.restype = c_sz
        L.bmoe_router.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp, c_sz,
                                  vp]
        L.bmoe_router.restype = c_int
        L.bmoe_router_timed.argtypes = L.bmoe_router.argtypes + [vp]
        L.bmoe_router_timed.restype = c_int
        L.bmoe_router_logits.argtypes = [c_int, c_int, c_int, c_int, vp, vp, vp, vp]
        L.bmoe_router_logits.restype = c_int
        L.bmoe_route.argtypes = [c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp]
        L.bmoe_route.restype = c_int
        L.bmoe_route_backward.argtypes = [c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp, vp]
        L.bmoe_route_backward.restype = c_int
        L.bmoe_route_balance_workspace_bytes.argtypes = [c_int, c_int, c_int]
        L.bmoe_route_balance_workspace_bytes.restype = c_sz
        L.bmoe_route_balance.argtypes = [c_int, c_int, c_int, vp, c_int, c_f, vp, vp, vp, c_sz, vp]
        L.bmoe_route_balance.restype = c_int
        L.bmoe_router_backward_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_router_backward_workspace_bytes.restype = c_sz
        L.bmoe_router_backward.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp,
                                           vp, vp, vp, vp, vp, c_sz, vp]
        L.bmoe_router_backward.restype = c_int
        L.bmoe_grad_workspace_bytes.argtypes = [c_int]
        L.bmoe_grad_workspace_bytes.restype = c_sz
        L.bmoe_grad_norm.argtypes = [c_int, vp, vp, vp, c_sz, vp]
        L.bmoe_grad_norm.restype = c_int
        L.bmoe_grad_scale.argtypes = [c_int, vp, vp, vp, c_f, vp]
        L.bmoe_grad_scale.restype = c_int
        L.bmoe_grad_clip.argtypes = [c_int, vp, vp, c_f, vp, vp, c_sz, vp]
        L.bmoe_grad_clip.restype = c_int
        L.bmoe_group_rows_workspace_bytes.argtypes = [c_int, c_int, c_int]
        L.bmoe_group_rows_workspace_bytes.restype = c_sz
        L.bmoe_group_rows.argtypes = [c_int, c_int, c_int, vp, vp, vp, vp, vp, c_sz, vp]
        L.bmoe_group_rows.restype = c_int
        L.bmoe_grouped_product.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, c_int, vp, c_int,
                                           vp, vp, vp, vp]
        L.bmoe_grouped_product.restype = c_int
        L.bmoe_grouped_product_filled.argtypes = L.bmoe_grouped_product.argtypes
        L.bmoe_grouped_product_filled.restype = c_int
        L.bmoe_grouped_product_backward_workspace_bytes.argtypes = [c_int] * 5
        L.bmoe_grouped_product_backward_workspace_bytes.restype = c_sz
        L.bmoe_grouped_product_backward.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, c_int,
                                                    vp, c_int, vp, vp, vp, vp, vp, vp, c_sz, vp]
        L.bmoe_grouped_product_backward.restype = c_int
        L.bmoe_grouped_product_backward_filled.argtypes = L.bmoe_grouped_product_backward.argtypes
        L.bmoe_grouped_product_backward_filled.restype = c_int
        L.bmoe_residual_norm.argtypes = [c_int, c_int, c_int, c_int, vp, vp, c_int, vp, vp, vp, vp,
                                         vp, vp, vp, vp]
        L.bmoe_residual_norm.restype = c_int
        L.bmoe_residual_norm_backward_workspace_bytes.argtypes = [c_int, c_int, c_int]
        L.bmoe_residual_norm_backward_workspace_bytes.restype = c_sz
        L.bmoe_residual_norm_backward.argtypes = ([c_int, c_int, c_int, c_int, vp, vp, c_int] +
                                                  [vp] * 13 + [c_sz, vp])
        L.bmoe_residual_norm_backward.restype = c_int
        L.bmoe_residual_norm_backward_filled_workspace_bytes.argtypes = [c_int] * 4
        L.bmoe_residual_norm_backward_filled_workspace_bytes.restype = c_sz
        L.bmoe_residual_norm_backward_filled.argtypes = L.bmoe_residual_norm_backward.argtypes
        L.bmoe_residual_norm_backward_filled.restype = c_int
        L.bmoe_orthogonalize_workspace_bytes.argtypes = [c_int, c_int, c_int]
        L.bmoe_orthogonalize_workspace_bytes.restype = c_sz
        L.bmoe_orthogonalize.argtypes = [c_int, c_int, c_int, c_int, vp, vp, vp, vp, c_sz, vp]
        L.bmoe_orthogonalize.restype = c_int
        L.bmoe_orthogonal_step.argtypes = [c_int, c_int, c_int, c_int, c_int, vp, vp, vp, vp, vp,
                                           vp, c_sz, vp]
        L.bmoe_orthogonal_step.restype = c_int
        L.bmoe_backward_timed.argtypes = L.bmoe_backward.argtypes + [vp]
        L.bmoe_backward_timed.restype = c_int
        L.bmoe_backward_kernel_count.argtypes = [c_int, c_int, c_int, c_int, c_int]
        L.bmoe_backward_kernel_count.restype = c_int
        L.bmoe_backward_kernel_name.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
        L.bmoe_backward_kernel_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# The current stream's handle without the Stream object around it: 0.1 us of a
# call instead of 2.7 us (the lookup torch's own generated code uses).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is None and _raw_stream is not None and torch.cuda.is_initialized():
        return _raw_stream(torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _on(stream=None):
    """Make `stream` torch's current stream while a wrapper allocates and
    launches: the caching allocator then ties the temporary workspace and the
    outputs to the stream the kernels run on, so memory freed when the wrapper
    returns is not handed to other work before those kernels finish."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _check(code: int, what: str):
    if code != 0:
        raise BmoeError(code, what)


# ---- the C entry points, same names -------------------------------------

def bmoe_packed_words(d: int) -> int:
    return lib().bmoe_packed_words(d)


def bmoe_param_count(d: int, n_experts: int) -> int:
    return lib().bmoe_param_count(d, n_experts)


def bmoe_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_pack_workspace_bytes() -> int:
    return lib().bmoe_pack_workspace_bytes()


def bmoe_pack_ternary(w: torch.Tensor, d: int, packed: torch.Tensor, ws: torch.Tensor,
                      stream=None) -> int:
    return lib().bmoe_pack_ternary(_ptr(w), d, _ptr(packed), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream))


def bmoe_packed3_bytes(d: int) -> int:
    return lib().bmoe_packed3_bytes(d)


def bmoe_pack_ternary_b3(w: torch.Tensor, d: int, packed3: torch.Tensor, ws: torch.Tensor,
                         stream=None) -> int:
    return lib().bmoe_pack_ternary_b3(_ptr(w), d, _ptr(packed3), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream))


def bmoe_unpack_ternary_b3(packed3: torch.Tensor, d: int, packed: torch.Tensor,
                           ws: torch.Tensor, stream=None) -> int:
    return lib().bmoe_unpack_ternary_b3(_ptr(packed3), d, _ptr(packed), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream))


def bmoe_unpack_ternary_b3_timed(packed3: torch.Tensor, d: int, packed: torch.Tensor,
                                 ws: torch.Tensor, stream=None, events=None) -> int:
    ev = None
    if events is not None:
        ev = (ctypes.c_void_p * len(events))(*events)
    return lib().bmoe_unpack_ternary_b3_timed(_ptr(packed3), d, _ptr(packed), _ptr(ws),
                                              ws.numel() * ws.element_size(), _stream(stream), ev)


def bmoe_forward(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta, phi,
                 w_packed, alpha: float, y, ws, route_out=None, stream=None) -> int:
    return lib().bmoe_forward(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates), _ptr(theta),
                              _ptr(phi), _ptr(w_packed), float(alpha), _ptr(y), _ptr(ws),
                              ws.numel() * ws.element_size(), _ptr(route_out), _stream(stream))


def bmoe_forward_timed(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta, phi,
                       w_packed, alpha: float, y, ws, route_out=None, stream=None,
                       events=None) -> int:
    """``events``: raw hipEvent_t handles (ints), two per kernel: the start and
    stop events of kernel i are events[2i] and events[2i+1]."""
    ev = None
    if events is not None:
        ev = (ctypes.c_void_p * len(events))(*events)
    return lib().bmoe_forward_timed(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates),
                                    _ptr(theta), _ptr(phi), _ptr(w_packed), float(alpha), _ptr(y),
                                    _ptr(ws), ws.numel() * ws.element_size(), _ptr(route_out),
                                    _stream(stream), ev)


def bmoe_forward_noalloc(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta,
                         phi, w_packed, alpha: float, y, route_out=None, status=None,
                         stream=None) -> int:
    return lib().bmoe_forward_noalloc(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates),
                                      _ptr(theta), _ptr(phi), _ptr(w_packed), alpha, _ptr(y),
                                      _ptr(route_out), _ptr(status), _stream(stream))


BMOE_NOALLOC_MAX_WORKSPACE = 64 << 20


BMOE_W_2BIT = 0
BMOE_W_BASE3 = 1


def bmoe_product(M: int, d: int, z, w, fmt: int, alpha: float, h, stream=None,
                 events=None) -> int:
    return lib().bmoe_product(M, d, _ptr(z), _ptr(w), fmt, alpha, _ptr(h), _stream(stream),
                              _events_arg(events))


BMOE_CEILING_SINK_FLOATS = 256 * 8 * 256


def _events_arg(events):
    return None if events is None else (ctypes.c_void_p * len(events))(*events)


def bmoe_ceiling_mfma_bf16(iters: int, sink, stream=None, events=None):
    """(status, flops executed)."""
    f = ctypes.c_double()
    rc = lib().bmoe_ceiling_mfma_bf16(iters, _ptr(sink), _stream(stream), _events_arg(events),
                                      ctypes.byref(f))
    return rc, f.value


def bmoe_ceiling_valu_f32(iters: int, sink, stream=None, events=None):
    """(status, flops executed)."""
    f = ctypes.c_double()
    rc = lib().bmoe_ceiling_valu_f32(iters, _ptr(sink), _stream(stream), _events_arg(events),
                                     ctypes.byref(f))
    return rc, f.value


def bmoe_ceiling_copy(src, dst, nbytes: int, stream=None, events=None) -> int:
    return lib().bmoe_ceiling_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream),
                                   _events_arg(events))


def bmoe_forward_kernel_count(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_forward_kernel_count(dt, T, d, n_experts, k)


def bmoe_forward_kernel_name(dt: int, T: int, d: int, n_experts: int, k: int, i: int) -> str:
    return lib().bmoe_forward_kernel_name(dt, T, d, n_experts, k, i).decode()


def bmoe_sync_status(ws: torch.Tensor, stream=None) -> int:
    return lib().bmoe_sync_status(_ptr(ws), _stream(stream))


def bmoe_status_str(code: int) -> str:
    return lib().bmoe_status_str(code).decode()


def bmoe_backward_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_backward_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_backward(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta, phi,
                  w_packed, alpha: float, dy, dx, dgates, dtheta, dphi, dw, ws,
                  stream=None) -> int:
    return lib().bmoe_backward(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates),
                               _ptr(theta), _ptr(phi), _ptr(w_packed), float(alpha), _ptr(dy),
                               _ptr(dx), _ptr(dgates), _ptr(dtheta), _ptr(dphi), _ptr(dw),
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def bmoe_backward_timed(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta,
                        phi, w_packed, alpha: float, dy, dx, dgates, dtheta, dphi, dw, ws,
                        stream=None, events=None) -> int:
    """``events``: raw hipEvent_t handles (ints), two per launch (start, stop)."""
    ev = None
    if events is not None:
        ev = (ctypes.c_void_p * len(events))(*events)
    return lib().bmoe_backward_timed(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates),
                                     _ptr(theta), _ptr(phi), _ptr(w_packed), float(alpha),
                                     _ptr(dy), _ptr(dx), _ptr(dgates), _ptr(dtheta), _ptr(dphi),
                                     _ptr(dw), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream), ev)


def bmoe_backward_kernel_count(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_backward_kernel_count(dt, T, d, n_experts, k)


def bmoe_backward_kernel_name(dt: int, T: int, d: int, n_experts: int, k: int, i: int) -> str:
    return lib().bmoe_backward_kernel_name(dt, T, d, n_experts, k, i).decode()


def bmoe_forward_keep_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_forward_keep_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_forward_keep(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, gates, theta, phi,
                      w_packed, alpha: float, y, ws, stream=None) -> int:
    return lib().bmoe_forward_keep(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(gates),
                                   _ptr(theta), _ptr(phi), _ptr(w_packed), float(alpha), _ptr(y),
                                   _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def bmoe_backward_kept(dt: int, T: int, d: int, n_experts: int, k: int, x, gates, w_packed,
                       alpha: float, dy, dx, dgates, dtheta, dphi, dw, fwd_ws, ws,
                       stream=None) -> int:
    return lib().bmoe_backward_kept(dt, T, d, n_experts, k, _ptr(x), _ptr(gates),
                                    _ptr(w_packed), float(alpha), _ptr(dy), _ptr(dx),
                                    _ptr(dgates), _ptr(dtheta), _ptr(dphi), _ptr(dw),
                                    _ptr(fwd_ws), fwd_ws.numel() * fwd_ws.element_size(),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def bmoe_backward_kept_timed(dt: int, T: int, d: int, n_experts: int, k: int, x, gates,
                             w_packed, alpha: float, dy, dx, dgates, dtheta, dphi, dw, fwd_ws,
                             ws, stream=None, events=None) -> int:
    ev = None
    if events is not None:
        ev = (ctypes.c_void_p * len(events))(*events)
    return lib().bmoe_backward_kept_timed(dt, T, d, n_experts, k, _ptr(x), _ptr(gates),
                                          _ptr(w_packed), float(alpha), _ptr(dy), _ptr(dx),
                                          _ptr(dgates), _ptr(dtheta), _ptr(dphi), _ptr(dw),
                                          _ptr(fwd_ws), fwd_ws.numel() * fwd_ws.element_size(),
                                          _ptr(ws), ws.numel() * ws.element_size(),
                                          _stream(stream), ev)


def bmoe_rotate_in_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_rotate_in_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_rotate_in(dt: int, T: int, d: int, n_experts: int, k: int, x, ids, theta, z, ws,
                   stream=None) -> int:
    return lib().bmoe_rotate_in(dt, T, d, n_experts, k, _ptr(x), _ptr(ids), _ptr(theta), _ptr(z),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))


def bmoe_quant_error(dt: int, rows: int, d: int, src, m: int, mode: int, err, crest=None,
                     stream=None) -> int:
    return lib().bmoe_quant_error(dt, rows, d, _ptr(src), m, mode, _ptr(err), _ptr(crest),
                                  _stream(stream))


def bmoe_router_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_router_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_router(dt: int, T: int, d: int, n_experts: int, k: int, x, w_router, ids, gates,
                logits=None, ws=None, stream=None) -> int:
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    return lib().bmoe_router(dt, T, d, n_experts, k, _ptr(x), _ptr(w_router), _ptr(ids),
                             _ptr(gates), _ptr(logits), _ptr(ws), nb, _stream(stream))


def bmoe_router_timed(dt: int, T: int, d: int, n_experts: int, k: int, x, w_router, ids, gates,
                      logits=None, ws=None, stream=None, events=None) -> int:
    """``events``: 4 raw hipEvent_t handles (start/stop of the logits and
    top-k launches)."""
    ev = None
    if events is not None:
        ev = (ctypes.c_void_p * len(events))(*events)
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    return lib().bmoe_router_timed(dt, T, d, n_experts, k, _ptr(x), _ptr(w_router), _ptr(ids),
                                   _ptr(gates), _ptr(logits), _ptr(ws), nb, _stream(stream), ev)


def bmoe_router_logits(dt: int, T: int, d: int, n_experts: int, x, w_router, logits,
                       stream=None) -> int:
    return lib().bmoe_router_logits(dt, T, d, n_experts, _ptr(x), _ptr(w_router), _ptr(logits),
                                    _stream(stream))


def bmoe_route(dt: int, T: int, n_experts: int, k: int, spec, logits, bias, ids, gates,
               stream=None) -> int:
    return lib().bmoe_route(dt, T, n_experts, k, _ref(spec), _ptr(logits), _ptr(bias), _ptr(ids),
                            _ptr(gates), _stream(stream))


def bmoe_route_backward(dt: int, T: int, n_experts: int, k: int, spec, logits, ids, dgates,
                        dlogits, stream=None) -> int:
    return lib().bmoe_route_backward(dt, T, n_experts, k, _ref(spec), _ptr(logits), _ptr(ids),
                                     _ptr(dgates), _ptr(dlogits), _stream(stream))


def bmoe_route_balance_workspace_bytes(T: int, n_experts: int, k: int) -> int:
    return lib().bmoe_route_balance_workspace_bytes(T, n_experts, k)


def bmoe_route_balance(T: int, n_experts: int, k: int, ids, accumulate: bool, rate: float, load,
                       bias, ws, stream=None) -> int:
    return lib().bmoe_route_balance(T, n_experts, k, _ptr(ids), int(accumulate), rate, _ptr(load),
                                    _ptr(bias), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_router_backward_workspace_bytes(dt: int, T: int, d: int, n_experts: int, k: int) -> int:
    return lib().bmoe_router_backward_workspace_bytes(dt, T, d, n_experts, k)


def bmoe_router_backward(dt: int, T: int, d: int, n_experts: int, k: int, spec, x, w_router,
                         logits, ids, dgates, dx_add, dx, dw, ws, stream=None) -> int:
    return lib().bmoe_router_backward(dt, T, d, n_experts, k, _ref(spec), _ptr(x), _ptr(w_router),
                                      _ptr(logits), _ptr(ids), _ptr(dgates), _ptr(dx_add),
                                      _ptr(dx), _ptr(dw), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_grad_workspace_bytes(n: int) -> int:
    return lib().bmoe_grad_workspace_bytes(n)


def bmoe_grad_norm(n: int, grads, norm, ws, stream=None) -> int:
    """``grads`` (and ``out`` below): ctypes arrays of BmoeTensor, or None."""
    return lib().bmoe_grad_norm(n, grads, _ptr(norm), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_grad_scale(n: int, grads, out, norm, max_norm: float, stream=None) -> int:
    return lib().bmoe_grad_scale(n, grads, out, _ptr(norm), max_norm, _stream(stream))


def bmoe_grad_clip(n: int, grads, out, max_norm: float, norm, ws, stream=None) -> int:
    return lib().bmoe_grad_clip(n, grads, out, max_norm, _ptr(norm), _ptr(ws), _nbytes(ws),
                                _stream(stream))


def bmoe_group_rows_workspace_bytes(T: int, n_experts: int, k: int) -> int:
    return lib().bmoe_group_rows_workspace_bytes(T, n_experts, k)


def bmoe_group_rows(T: int, n_experts: int, k: int, ids, offsets, perm, inv, ws,
                    stream=None) -> int:
    return lib().bmoe_group_rows(T, n_experts, k, _ptr(ids), _ptr(offsets), _ptr(perm), _ptr(inv),
                                 _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_grouped_product(dt: int, M: int, K: int, O: int, n_groups: int, a, a_rows: int, perm,
                         k: int, w, offsets, c, stream=None) -> int:
    return lib().bmoe_grouped_product(dt, M, K, O, n_groups, _ptr(a), a_rows, _ptr(perm), k,
                                      _ptr(w), _ptr(offsets), _ptr(c), _stream(stream))


def bmoe_grouped_product_filled(dt: int, M: int, K: int, O: int, n_groups: int, a, a_rows: int,
                                perm, k: int, w, offsets, c, stream=None) -> int:
    return lib().bmoe_grouped_product_filled(dt, M, K, O, n_groups, _ptr(a), a_rows, _ptr(perm), k,
                                             _ptr(w), _ptr(offsets), _ptr(c), _stream(stream))


def bmoe_grouped_product_backward_workspace_bytes(dt: int, M: int, K: int, O: int,
                                                  n_groups: int) -> int:
    return lib().bmoe_grouped_product_backward_workspace_bytes(dt, M, K, O, n_groups)


def bmoe_grouped_product_backward(dt: int, M: int, K: int, O: int, n_groups: int, a, a_rows: int,
                                  perm, k: int, w, offsets, dc, da, dw, ws, stream=None) -> int:
    return lib().bmoe_grouped_product_backward(dt, M, K, O, n_groups, _ptr(a), a_rows, _ptr(perm),
                                               k, _ptr(w), _ptr(offsets), _ptr(dc), _ptr(da),
                                               _ptr(dw), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_grouped_product_backward_filled(dt: int, M: int, K: int, O: int, n_groups: int, a,
                                         a_rows: int, perm, k: int, w, offsets, dc, da, dw, ws,
                                         stream=None) -> int:
    return lib().bmoe_grouped_product_backward_filled(
        dt, M, K, O, n_groups, _ptr(a), a_rows, _ptr(perm), k, _ptr(w), _ptr(offsets), _ptr(dc),
        _ptr(da), _ptr(dw), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_residual_norm(dt: int, T: int, d: int, k: int, spec, u, u_rows: int, inv, gates, r, w_post,
                       w_pre, r_out, n, stream=None) -> int:
    return lib().bmoe_residual_norm(dt, T, d, k, _ref(spec), _ptr(u), u_rows, _ptr(inv),
                                    _ptr(gates), _ptr(r), _ptr(w_post), _ptr(w_pre), _ptr(r_out),
                                    _ptr(n), _stream(stream))


def bmoe_residual_norm_backward_workspace_bytes(dt: int, T: int, d: int) -> int:
    return lib().bmoe_residual_norm_backward_workspace_bytes(dt, T, d)


def bmoe_residual_norm_backward(dt: int, T: int, d: int, k: int, spec, u, u_rows: int, inv, gates,
                                r_out, w_post, w_pre, dr_out, dn, du, dgates, dr, dw_post, dw_pre,
                                ws, stream=None) -> int:
    return lib().bmoe_residual_norm_backward(dt, T, d, k, _ref(spec), _ptr(u), u_rows, _ptr(inv),
                                             _ptr(gates), _ptr(r_out), _ptr(w_post), _ptr(w_pre),
                                             _ptr(dr_out), _ptr(dn), _ptr(du), _ptr(dgates),
                                             _ptr(dr), _ptr(dw_post), _ptr(dw_pre), _ptr(ws),
                                             _nbytes(ws), _stream(stream))


def bmoe_residual_norm_backward_filled_workspace_bytes(dt: int, T: int, d: int, u_rows: int) -> int:
    return lib().bmoe_residual_norm_backward_filled_workspace_bytes(dt, T, d, u_rows)


def bmoe_residual_norm_backward_filled(dt: int, T: int, d: int, k: int, spec, u, u_rows: int, inv,
                                       gates, r_out, w_post, w_pre, dr_out, dn, du, dgates, dr,
                                       dw_post, dw_pre, ws, stream=None) -> int:
    return lib().bmoe_residual_norm_backward_filled(
        dt, T, d, k, _ref(spec), _ptr(u), u_rows, _ptr(inv), _ptr(gates), _ptr(r_out), _ptr(w_post),
        _ptr(w_pre), _ptr(dr_out), _ptr(dn), _ptr(du), _ptr(dgates), _ptr(dr), _ptr(dw_post),
        _ptr(dw_pre), _ptr(ws), _nbytes(ws), _stream(stream))


def bmoe_orthogonalize_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return lib().bmoe_orthogonalize_workspace_bytes(batch, rows, cols)


def bmoe_orthogonalize(dt: int, batch: int, rows: int, cols: int, spec, u, o, ws,
                       stream=None) -> int:
    return lib().bmoe_orthogonalize(dt, batch, rows, cols, _ref(spec), _ptr(u), _ptr(o), _ptr(ws),
                                    _nbytes(ws), _stream(stream))


def bmoe_orthogonal_step(w_dt: int, grad_dt: int, batch: int, rows: int, cols: int, spec, update,
                         grad, momentum, w, ws, stream=None) -> int:
    return lib().bmoe_orthogonal_step(w_dt, grad_dt, batch, rows, cols, _ref(spec), _ref(update),
                                      _ptr(grad), _ptr(momentum), _ptr(w), _ptr(ws), _nbytes(ws),
                                      _stream(stream))


# ---- conveniences over the entry points (allocation + error checks) -------

def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BMOE_BF16
    if t.dtype == torch.float32:
        return BMOE_F32
    raise TypeError(f"x must be float32 or bfloat16, got {t.dtype}")


def pack_ternary(w: torch.Tensor) -> torch.Tensor:
    """int8 [d][d] device tensor -> packed uint32 words (as int32 storage)."""
    d = w.shape[0]
    n = bmoe_packed_words(d)
    if n == 0:
        raise BmoeError(2, "bmoe_pack_ternary")
    packed = torch.empty(n, dtype=torch.int32, device=w.device)
    ws = torch.empty(bmoe_pack_workspace_bytes(), dtype=torch.uint8, device=w.device)
    _check(bmoe_pack_ternary(w.contiguous(), d, packed, ws), "bmoe_pack_ternary")
    _check(bmoe_sync_status(ws), "bmoe_pack_ternary")
    return packed


class Workspace:
    """Caller-owned workspace sized for one shape (reused across calls)."""

    def __init__(self, dt: int, T: int, d: int, n_experts: int, k: int, device="cuda"):
        n = bmoe_workspace_bytes(dt, T, d, n_experts, k)
        if n == 0:
            raise BmoeError(2, "bmoe_workspace_bytes")
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.key = (dt, T, d, n_experts, k)


def forward(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, theta: torch.Tensor,
            phi: torch.Tensor, w_packed: torch.Tensor, alpha: float, *, y=None, ws=None,
            route_out=None, stream=None) -> torch.Tensor:
    with _on(stream):
        T, d = x.shape
        k = ids.shape[1]
        N = theta.shape[0]
        dt = dtype_code(x)
        if y is None:
            y = torch.empty_like(x)
        if ws is None:
            ws = Workspace(dt, T, d, N, k, device=x.device)
        _check(bmoe_forward(dt, T, d, N, k, x, ids, gates, theta, phi, w_packed, alpha, y, ws.buf,
                            route_out, stream), "bmoe_forward")
        return y


def backward(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, theta: torch.Tensor,
             phi: torch.Tensor, w_packed: torch.Tensor, alpha: float, dy: torch.Tensor, *,
             want_dw: bool = True, stream=None) -> dict:
    """Gradients of sum(dy * y) for the layer bmoe_forward computes: dict of
    dx (dtype of x), dgates, dtheta, dphi and (want_dw) dw, all fp32 but dx."""
    with _on(stream):
        T, d = x.shape
        k = ids.shape[1]
        N = theta.shape[0]
        dt = dtype_code(x)
        n = bmoe_backward_workspace_bytes(dt, T, d, N, k)
        if n == 0:
            raise BmoeError(2, "bmoe_backward_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        out = {
            "dx": torch.empty_like(x),
            "dgates": torch.empty(T, k, dtype=torch.float32, device=x.device),
            "dtheta": torch.empty_like(theta),
            "dphi": torch.empty_like(phi),
            "dw": torch.empty(d, d, dtype=torch.float32, device=x.device) if want_dw else None,
        }
        _check(bmoe_backward(dt, T, d, N, k, x, ids, gates, theta, phi, w_packed, alpha, dy,
                             out["dx"], out["dgates"], out["dtheta"], out["dphi"], out["dw"], ws,
                             stream), "bmoe_backward")
        return out


def route(x: torch.Tensor, w_router: torch.Tensor, k: int, *, want_logits: bool = False,
          stream=None):
    """Router: (ids int32 [T][k], gates fp32 [T][k]) for bmoe_forward, plus
    the fp32 [T][N] logits when want_logits."""
    with _on(stream):
        T, d = x.shape
        N = w_router.shape[0]
        dt = dtype_code(x)
        if w_router.dtype != x.dtype or w_router.shape[1] != d:
            raise ValueError("w_router must be [N][d] in x's dtype")
        ids = torch.empty(T, k, dtype=torch.int32, device=x.device)
        gates = torch.empty(T, k, dtype=torch.float32, device=x.device)
        logits = torch.empty(T, N, dtype=torch.float32, device=x.device) if want_logits else None
        ws = None
        if logits is None:
            n = bmoe_router_workspace_bytes(dt, T, d, N, k)
            if n == 0:
                raise BmoeError(2, "bmoe_router_workspace_bytes")
            ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        _check(bmoe_router(dt, T, d, N, k, x, w_router, ids, gates, logits, ws, stream),
               "bmoe_router")
        return (ids, gates, logits) if want_logits else (ids, gates)


def pack_ternary_b3(w: torch.Tensor) -> torch.Tensor:
    """int8 [d][d] in {-1,0,+1} on the GPU -> uint8 base-3 stream (raises on
    a bad entry)."""
    d = w.shape[0]
    n = bmoe_packed3_bytes(d)
    if n == 0 or w.shape != (d, d) or w.dtype != torch.int8:
        raise ValueError("w must be int8 [d][d] with a supported d")
    # 8 bytes of slack past the stream, as bmoe_product reads whole dwords
    out = torch.zeros((n + 8 + 15) // 16 * 16, dtype=torch.uint8, device=w.device)
    ws = torch.empty(bmoe_pack_workspace_bytes(), dtype=torch.uint8, device=w.device)
    _check(bmoe_pack_ternary_b3(w, d, out, ws), "bmoe_pack_ternary_b3")
    _check(bmoe_sync_status(ws), "bmoe_pack_ternary_b3 (device)")
    return out[:n]


def unpack_ternary_b3(packed3: torch.Tensor, d: int) -> torch.Tensor:
    """Base-3 stream -> the 2-bit words bmoe_forward takes (raises on a byte
    above 242)."""
    out = torch.empty(d, d // 16, dtype=torch.int32, device=packed3.device)
    ws = torch.empty(bmoe_pack_workspace_bytes(), dtype=torch.uint8, device=packed3.device)
    _check(bmoe_unpack_ternary_b3(packed3, d, out, ws), "bmoe_unpack_ternary_b3")
    _check(bmoe_sync_status(ws), "bmoe_unpack_ternary_b3 (device)")
    return out


def rotate_in(x: torch.Tensor, ids: torch.Tensor, theta: torch.Tensor) -> torch.Tensor:
    """z [T*k][d] (x's dtype), row t*k + j = B(theta_{ids[t][j]})^T x[t]."""
    T, d = x.shape
    k = ids.shape[1]
    N = theta.shape[0]
    dt = dtype_code(x)
    n = bmoe_rotate_in_workspace_bytes(dt, T, d, N, k)
    if n == 0:
        raise BmoeError(2, "bmoe_rotate_in_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    z = torch.empty(T * k, d, dtype=x.dtype, device=x.device)
    _check(bmoe_rotate_in(dt, T, d, N, k, x, ids, theta, z, ws), "bmoe_rotate_in")
    _check(bmoe_sync_status(ws), "bmoe_rotate_in (device)")
    return z


def quant_error(v: torch.Tensor, m: int, mode: int = 0):
    """(err, crest) fp32 [rows] for the rows of v (bf16 or fp32)."""
    rows, d = v.shape
    err = torch.empty(rows, dtype=torch.float32, device=v.device)
    crest = torch.empty(rows, dtype=torch.float32, device=v.device)
    _check(bmoe_quant_error(dtype_code(v), rows, d, v, m, mode, err, crest), "bmoe_quant_error")
    return err, crest


def forward_keep(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, theta: torch.Tensor,
                 phi: torch.Tensor, w_packed: torch.Tensor, alpha: float, stream=None):
    """(y, kept workspace): the forward on the unfused path, with its routing
    tables, cos/sin tables, Z and H left in the returned workspace for
    backward_kept."""
    with _on(stream):
        T, d = x.shape
        k = ids.shape[1]
        N = theta.shape[0]
        dt = dtype_code(x)
        n = bmoe_forward_keep_workspace_bytes(dt, T, d, N, k)
        if n == 0:
            raise BmoeError(2, "bmoe_forward_keep_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        y = torch.empty_like(x)
        _check(bmoe_forward_keep(dt, T, d, N, k, x, ids, gates, theta, phi, w_packed, alpha, y, ws,
                                 stream), "bmoe_forward_keep")
        return y, ws


def backward_kept(x: torch.Tensor, gates: torch.Tensor, n_experts: int, w_packed: torch.Tensor,
                  alpha: float, dy: torch.Tensor, kept: torch.Tensor, *, want_dw: bool = True,
                  stream=None) -> dict:
    """As backward(), reading the forward's intermediates from forward_keep's
    workspace instead of recomputing them."""
    with _on(stream):
        T, d = x.shape
        k = gates.shape[1]
        N = n_experts
        dt = dtype_code(x)
        L = int(d).bit_length() - 1
        n = bmoe_backward_workspace_bytes(dt, T, d, N, k)
        if n == 0:
            raise BmoeError(2, "bmoe_backward_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        out = {
            "dx": torch.empty_like(x),
            "dgates": torch.empty(T, k, dtype=torch.float32, device=x.device),
            "dtheta": torch.empty(N, L, d // 2, dtype=torch.float32, device=x.device),
            "dphi": torch.empty(N, L, d // 2, dtype=torch.float32, device=x.device),
            "dw": torch.empty(d, d, dtype=torch.float32, device=x.device) if want_dw else None,
        }
        _check(bmoe_backward_kept(dt, T, d, N, k, x, gates, w_packed, alpha, dy, out["dx"],
                                  out["dgates"], out["dtheta"], out["dphi"], out["dw"], kept, ws,
                                  stream), "bmoe_backward_kept")
        return out


# ---- routing from logits and the rest of a training step ---------------------

@contextlib.contextmanager
def _device_of(device, stream):
    with torch.cuda.device(device), _on(stream):
        yield


def _at(t: torch.Tensor, stream):
    """Make t's device (and `stream`, one of that device) current for a call."""
    if not t.is_cuda:
        raise ValueError("the library works on GPU tensors")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {t.device}")
    if stream is None and t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return _device_of(t.device, stream)


def _like(name: str, t: torch.Tensor, dtype, shape, device) -> torch.Tensor:
    """t itself, checked: dtype, shape, device and contiguous storage."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', strided'}")
    return t


def _matrix(name: str, t: torch.Tensor) -> torch.Tensor:
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix, got shape {tuple(t.shape)}")
    return t


def router_logits(x: torch.Tensor, w_router: torch.Tensor, *, logits=None,
                  stream=None) -> torch.Tensor:
    """fp32 [T][N] = x w_router^T: the logits of route(), for route_logits()."""
    T, d = _matrix("x", x).shape
    N = w_router.shape[0]
    dt = dtype_code(x)
    _like("w_router", w_router, x.dtype, (N, d), x.device)
    with _at(x, stream):
        if logits is None:
            logits = torch.empty(T, N, dtype=torch.float32, device=x.device)
        else:
            _like("logits", logits, torch.float32, (T, N), x.device)
        _check(bmoe_router_logits(dt, T, d, N, x, w_router, logits, stream), "bmoe_router_logits")
        return logits


def route_logits(logits: torch.Tensor, k: int, spec: Optional[RouteSpec] = None, *, bias=None,
                 ids=None, gates=None, stream=None):
    """(ids int32 [T][k], gates fp32 [T][k]) of the k experts each row of
    logits (fp32 or bf16 [T][N]) chooses under `spec` (default: softmax gates
    renormalised over the chosen, as route()); `bias` fp32 [N] moves the choice."""
    T, N = _matrix("logits", logits).shape
    dt = dtype_code(logits)
    dev = logits.device
    if spec is None:
        spec = RouteSpec()
    with _at(logits, stream):
        if bias is not None:
            _like("bias", bias, torch.float32, (N,), dev)
        if ids is None:
            ids = torch.empty(T, k, dtype=torch.int32, device=dev)
        else:
            _like("ids", ids, torch.int32, (T, k), dev)
        if gates is None:
            gates = torch.empty(T, k, dtype=torch.float32, device=dev)
        else:
            _like("gates", gates, torch.float32, (T, k), dev)
        _check(bmoe_route(dt, T, N, k, spec, logits, bias, ids, gates, stream), "bmoe_route")
        return ids, gates


def route_logits_backward(logits: torch.Tensor, ids: torch.Tensor, dgates: torch.Tensor,
                          spec: Optional[RouteSpec] = None, *, dlogits=None,
                          stream=None) -> torch.Tensor:
    """dlogits fp32 [T][N] of sum(dgates * gates) for route_logits()'s gates."""
    T, N = _matrix("logits", logits).shape
    k = _matrix("ids", ids).shape[1]
    dt = dtype_code(logits)
    dev = logits.device
    if spec is None:
        spec = RouteSpec()
    _like("ids", ids, torch.int32, (T, k), dev)
    _like("dgates", dgates, torch.float32, (T, k), dev)
    with _at(logits, stream):
        if dlogits is None:
            dlogits = torch.empty(T, N, dtype=torch.float32, device=dev)
        else:
            _like("dlogits", dlogits, torch.float32, (T, N), dev)
        _check(bmoe_route_backward(dt, T, N, k, spec, logits, ids, dgates, dlogits, stream),
               "bmoe_route_backward")
        return dlogits


def route_balance(ids: torch.Tensor, load: torch.Tensor, *, bias=None, rate: float = 0.0,
                  accumulate: bool = False, stream=None) -> torch.Tensor:
    """Counts ids [T][k] into load int32 [N] (added to it with `accumulate`)
    and, with a bias fp32 [N], moves it by `rate` against the loads, in place.
    Returns load."""
    T, k = _matrix("ids", ids).shape
    N = load.numel()
    _like("ids", ids, torch.int32, (T, k), load.device)
    _like("load", load, torch.int32, (N,), load.device)
    with _at(load, stream):
        if bias is not None:
            _like("bias", bias, torch.float32, (N,), load.device)
        n = bmoe_route_balance_workspace_bytes(T, N, k)
        if n == 0:
            raise BmoeError(2, "bmoe_route_balance_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=load.device)
        _check(bmoe_route_balance(T, N, k, ids, accumulate, rate, load, bias, ws, stream),
               "bmoe_route_balance")
        return load


def router_backward(x: torch.Tensor, w_router: torch.Tensor, logits: torch.Tensor,
                    ids: torch.Tensor, dgates: torch.Tensor, spec: Optional[RouteSpec] = None, *,
                    dx_add=None, dx=None, dw=None, stream=None) -> dict:
    """Gradients of sum(dgates * gates) for gates = route_logits(x w_router^T):
    dict of dx (dtype of x; plus `dx_add`, e.g. backward()'s dx) and dw fp32
    [N][d]. logits: the fp32 ones of router_logits() or route()."""
    T, d = _matrix("x", x).shape
    N = w_router.shape[0]
    k = _matrix("ids", ids).shape[1]
    dt = dtype_code(x)
    dev = x.device
    if spec is None:
        spec = RouteSpec()
    _like("w_router", w_router, x.dtype, (N, d), dev)
    _like("logits", logits, torch.float32, (T, N), dev)
    _like("ids", ids, torch.int32, (T, k), dev)
    _like("dgates", dgates, torch.float32, (T, k), dev)
    with _at(x, stream):
        if dx_add is not None:
            _like("dx_add", dx_add, x.dtype, (T, d), dev)
        if dx is None:
            dx = torch.empty_like(x)
        else:
            _like("dx", dx, x.dtype, (T, d), dev)
        if dw is None:
            dw = torch.empty(N, d, dtype=torch.float32, device=dev)
        else:
            _like("dw", dw, torch.float32, (N, d), dev)
        n = bmoe_router_backward_workspace_bytes(dt, T, d, N, k)
        if n == 0:
            raise BmoeError(2, "bmoe_router_backward_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        _check(bmoe_router_backward(dt, T, d, N, k, spec, x, w_router, logits, ids, dgates,
                                    dx_add, dx, dw, ws, stream), "bmoe_router_backward")
        return {"dx": dx, "dw": dw}


_CODES = {torch.float32: BMOE_F32, torch.bfloat16: BMOE_BF16}


def _grad_list(name: str, tensors, device):
    for t in tensors:
        if t.dtype not in _CODES:
            raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        if t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous tensors on one device")
    return (BmoeTensor * len(tensors))(*[(t.data_ptr(), t.numel(), _CODES[t.dtype])
                                         for t in tensors])


def _grad_call(grads, out, stream):
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    dev = grads[0].device
    arr = _grad_list("grads", grads, dev)
    if out is None:
        return grads, arr, None
    out = list(out)
    if len(out) != len(grads):
        raise ValueError("out must have one tensor per gradient")
    return grads, arr, _grad_list("out", out, dev)


def grad_norm(grads, *, stream=None) -> torch.Tensor:
    """fp32 scalar tensor: the 2-norm over all entries of all `grads` (fp32 or
    bf16 tensors of one GPU), summed in 64 bits."""
    grads, arr, _ = _grad_call(grads, None, stream)
    with _at(grads[0], stream):
        norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
        ws = torch.empty(bmoe_grad_workspace_bytes(len(arr)), dtype=torch.uint8, device=norm.device)
        _check(bmoe_grad_norm(len(arr), arr, norm, ws, stream), "bmoe_grad_norm")
        return norm


def scale_grads(grads, norm: torch.Tensor, max_norm: float, *, out=None, stream=None) -> None:
    """grads * max_norm / norm where max_norm < norm < inf, in place or to
    `out`: clip_grads() with a norm at hand (e.g. summed over ranks)."""
    grads, arr, oarr = _grad_call(grads, out, stream)
    _like("norm", norm, torch.float32, (), grads[0].device)
    with _at(grads[0], stream):
        _check(bmoe_grad_scale(len(arr), arr, oarr, norm, max_norm, stream), "bmoe_grad_scale")


def clip_grads(grads, max_norm: float, *, out=None, stream=None) -> torch.Tensor:
    """Scale `grads` so that their global 2-norm is at most max_norm, in place
    or to `out` (tensors of the same types and sizes). Returns the norm before
    clipping; one that is not finite leaves the gradients as they are."""
    grads, arr, oarr = _grad_call(grads, out, stream)
    with _at(grads[0], stream):
        norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
        ws = torch.empty(bmoe_grad_workspace_bytes(len(arr)), dtype=torch.uint8, device=norm.device)
        _check(bmoe_grad_clip(len(arr), arr, oarr, max_norm, norm, ws, stream), "bmoe_grad_clip")
        return norm


# ---- around a block: dense experts, norms, orthogonalised updates ---------------

def _fits(*counts: int):
    """Refuses counts that the library's ints would wrap."""
    if max(counts) > 0x7FFFFFFF:
        raise ValueError(f"counts are at most 2^31 - 1, got {max(counts)}")


def _workspace(n: int, what: str, device) -> torch.Tensor:
    if n == 0:
        raise BmoeError(2, what)
    return torch.empty(n, dtype=torch.uint8, device=device)


def group_rows(ids: torch.Tensor, n_experts: int, *, stream=None):
    """(offsets int32 [N+1], perm int32 [T*k], inv int32 [T*k]): the routed rows
    r = t*k + j of ids int32 [T][k] grouped by expert, in order within one. An id
    outside [0, N) is a padded pick: behind the last expert, inv = -1."""
    T, k = _matrix("ids", ids).shape
    dev = ids.device
    _like("ids", ids, torch.int32, (T, k), dev)
    _fits(T * k, n_experts)
    with _at(ids, stream):
        ws = _workspace(bmoe_group_rows_workspace_bytes(T, n_experts, k),
                        "bmoe_group_rows_workspace_bytes", dev)
        offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * k, dtype=torch.int32, device=dev)
        inv = torch.empty(T * k, dtype=torch.int32, device=dev)
        _check(bmoe_group_rows(T, n_experts, k, ids, offsets, perm, inv, ws, stream),
               "bmoe_group_rows")
        return offsets, perm, inv


def _grouped(a, w, offsets, perm, k):
    """(dt, M, K, O, groups) of a grouped product's checked inputs."""
    R, K = _matrix("a", a).shape
    dt = dtype_code(a)
    if w.dim() != 3:
        raise ValueError(f"w must be [groups][O][K], got shape {tuple(w.shape)}")
    G, O = w.shape[:2]
    _like("w", w, a.dtype, (G, O, K), a.device)
    _like("offsets", offsets, torch.int32, (G + 1,), a.device)
    _fits(R, K, O, k)
    if perm is None:
        return dt, R, K, O, G
    _like("perm", perm, torch.int32, (perm.numel(),), a.device)
    if k < 1:
        raise ValueError("k must be at least 1")
    _fits(perm.numel())
    return dt, perm.numel(), K, O, G


def grouped_product(a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, perm=None,
                    k: int = 1, out=None, stream=None) -> torch.Tensor:
    """c [M][O], c[q] = w[e] a[row(q)] for the rows q of group e = offsets[e] ..
    offsets[e+1] (int32, on the GPU). a [R][K], w [groups][O][K] (one type, fp32
    or bf16); row(q) = perm[q] // k with group_rows()'s perm, else q. Rows of no
    group (padded picks) are 0; those of a given `out` are left as they were."""
    dt, M, K, O, G = _grouped(a, w, offsets, perm, k)
    with _at(a, stream):
        if out is None:
            call, out = bmoe_grouped_product_filled, torch.empty(M, O, dtype=a.dtype, device=a.device)
        else:
            call = bmoe_grouped_product
            _like("out", out, a.dtype, (M, O), a.device)
        _check(call(dt, M, K, O, G, a, a.shape[0], perm, k, w, offsets, out, stream),
               "bmoe_grouped_product")
        return out


def grouped_product_backward(a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                             dc: torch.Tensor, *, perm=None, k: int = 1, da=None, dw=None,
                             want_da: bool = True, want_dw: bool = True, stream=None) -> dict:
    """Gradients of sum(dc * c) for grouped_product()'s c: dict of da [M][K] (one
    row per row of the product, type of a) and dw fp32 [groups][O][K]. With
    `perm`, residual_norm(da, k=k, inv=inv) sums a token's k rows. Rows of no group
    are 0 in da; those of a given `da` are left as they were."""
    dt, M, K, O, G = _grouped(a, w, offsets, perm, k)
    _like("dc", dc, a.dtype, (M, O), a.device)
    with _at(a, stream):
        call = bmoe_grouped_product_backward
        if da is not None:
            _like("da", da, a.dtype, (M, K), a.device)
        elif want_da:
            call = bmoe_grouped_product_backward_filled
            da = torch.empty(M, K, dtype=a.dtype, device=a.device)
        if dw is not None:
            _like("dw", dw, torch.float32, (G, O, K), a.device)
        elif want_dw:
            dw = torch.empty(G, O, K, dtype=torch.float32, device=a.device)
        ws = _workspace(bmoe_grouped_product_backward_workspace_bytes(dt, M, K, O, G),
                        "bmoe_grouped_product_backward_workspace_bytes", a.device)
        _check(call(dt, M, K, O, G, a, a.shape[0], perm, k, w, offsets, dc, da, dw, ws, stream),
               "bmoe_grouped_product_backward")
        return {"da": da, "dw": dw}


def _norm_inputs(x, T, d, u, k, inv, gates, w_post, w_pre):
    """Checks what both directions of residual_norm() read; the rows of u."""
    dev = x.device
    _fits(T * k, d)
    if u is not None:
        _fits(u.shape[0])
        if u.dim() != 2 or u.shape[1] != d:
            raise ValueError(f"u must be [rows][{d}], got shape {tuple(u.shape)}")
        _like("u", u, x.dtype, u.shape, dev)
        if inv is not None:
            _like("inv", inv, torch.int32, (T * k,), dev)
        elif u.shape[0] != T * k:
            raise ValueError(f"u must have {T * k} rows without inv, got {u.shape[0]}")
        if gates is not None:
            _like("gates", gates, torch.float32, (T, k), dev)
    elif inv is not None or gates is not None or w_post is not None:
        raise ValueError("inv, gates and w_post belong to u")
    for name, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            _like(name, w, torch.float32, (d,), dev)
    return 0 if u is None else u.shape[0]


def residual_norm(u, r, spec: Optional[NormSpec] = None, *, k: int = 1, inv=None, gates=None,
                  w_post=None, w_pre=None, r_out=None, n=None, stream=None):
    """(r', n): r' = res_scale * r + out_scale * z with z the (w_post: RMS-normed)
    sum of a token's k gate-weighted rows of u, n the RMS norm of r' (None without
    w_pre). u [rows][d]: grouped_product()'s c with inv (int32 [T*k] of
    group_rows()) and gates fp32 [T][k], or a layer's y; None: n of r alone. r
    [T][d] or None (0). r_out may be r."""
    if u is None and r is None:
        raise ValueError("u or r has to be given")
    x = u if r is None else r
    _matrix("r" if r is not None else "u", x)
    if k < 1:
        raise ValueError("k must be at least 1")
    d = x.shape[1]
    if r is not None:
        T = r.shape[0]
    elif inv is not None:
        T = inv.numel() // k
    else:
        T = u.shape[0] // k
    dt = dtype_code(x)
    rows = _norm_inputs(x, T, d, u, k, inv, gates, w_post, w_pre)
    if spec is None:
        spec = NormSpec()
    with _at(x, stream):
        if r_out is not None:
            _like("r_out", r_out, x.dtype, (T, d), x.device)
        else:
            r_out = torch.empty(T, d, dtype=x.dtype, device=x.device)
        if n is not None and w_pre is None:
            raise ValueError("n needs w_pre")
        if n is not None:
            _like("n", n, x.dtype, (T, d), x.device)
        elif w_pre is not None:
            n = torch.empty(T, d, dtype=x.dtype, device=x.device)
        _check(bmoe_residual_norm(dt, T, d, k, spec, u, rows, inv, gates, r, w_post, w_pre, r_out,
                                  n, stream), "bmoe_residual_norm")
        return r_out, n


def residual_norm_backward(u, r_out: torch.Tensor, spec: Optional[NormSpec] = None, *, k: int = 1,
                           inv=None, gates=None, w_post=None, w_pre=None, dr_out=None, dn=None,
                           du=None, dr=None, stream=None) -> dict:
    """Gradients of sum(dr_out * r') + sum(dn * n) for residual_norm(): dict of
    dr, du, dgates, dw_post and dw_pre (None where the input is). r_out: its r' as
    stored. Rows of u that no pick names (padded picks') are 0 in du; those of a
    given `du` are left as they were."""
    T, d = _matrix("r_out", r_out).shape
    dev = r_out.device
    dt = dtype_code(r_out)
    if k < 1:
        raise ValueError("k must be at least 1")
    rows = _norm_inputs(r_out, T, d, u, k, inv, gates, w_post, w_pre)
    if (dn is None) != (w_pre is None):
        raise ValueError("dn belongs to w_pre")
    if dr_out is None and w_pre is None:
        raise ValueError("dr_out is needed without w_pre")
    if spec is None:
        spec = NormSpec()
    for name, t in (("dr_out", dr_out), ("dn", dn), ("dr", dr)):
        if t is not None:
            _like(name, t, r_out.dtype, (T, d), dev)
    if du is not None:
        if u is None:
            raise ValueError("du belongs to u")
        _like("du", du, u.dtype, u.shape, dev)
    with _at(r_out, stream):
        # without inv every row of u is a pick's
        fill = du is None and inv is not None
        if du is None and u is not None:
            du = torch.empty_like(u)
        if dr is None:
            dr = torch.empty_like(r_out)
        dgates = None if gates is None else torch.empty_like(gates)
        dw_post = None if w_post is None else torch.empty_like(w_post)
        dw_pre = None if w_pre is None else torch.empty_like(w_pre)
        ws = _workspace(bmoe_residual_norm_backward_filled_workspace_bytes(dt, T, d, rows) if fill
                        else bmoe_residual_norm_backward_workspace_bytes(dt, T, d),
                        "bmoe_residual_norm_backward_workspace_bytes", dev)
        call = bmoe_residual_norm_backward_filled if fill else bmoe_residual_norm_backward
        _check(call(dt, T, d, k, spec, u, rows, inv, gates, r_out, w_post, w_pre, dr_out, dn, du,
                    dgates, dr, dw_post, dw_pre, ws, stream), "bmoe_residual_norm_backward")
        return {"dr": dr, "du": du, "dgates": dgates, "dw_post": dw_post, "dw_pre": dw_pre}


def _matrices(name: str, t: torch.Tensor):
    """(batch, rows, cols) of one matrix or a batch of them."""
    if t.dim() not in (2, 3) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix or a batch of matrices, got shape "
                         f"{tuple(t.shape)}")
    _fits(*t.shape)
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


def orthogonalize(u: torch.Tensor, spec: Optional[OrthoSpec] = None, *, out=None,
                  stream=None) -> torch.Tensor:
    """The Newton-Schulz iterate of u / |u| for a matrix or a batch of matrices
    (fp32 or bf16): u's singular vectors with singular values near 1. out may be
    u."""
    B, rows, cols = _matrices("u", u)
    dt = dtype_code(u)
    if spec is None:
        spec = OrthoSpec()
    with _at(u, stream):
        if out is None:
            out = torch.empty_like(u)
        else:
            _like("out", out, u.dtype, u.shape, u.device)
        ws = _workspace(bmoe_orthogonalize_workspace_bytes(B, rows, cols),
                        "bmoe_orthogonalize_workspace_bytes", u.device)
        _check(bmoe_orthogonalize(dt, B, rows, cols, spec, u, out, ws, stream),
               "bmoe_orthogonalize")
        return out


def orthogonal_step(w: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, lr: float,
                    spec: Optional[OrthoSpec] = None, *, beta: float = 0.95, nesterov: bool = True,
                    weight_decay: float = 0.0, scale: float = 1.0, stream=None) -> torch.Tensor:
    """One step of the weights w (a matrix or a batch, fp32 or bf16) by the
    orthogonalised momentum of grad (fp32 or bf16), in place: momentum (fp32) =
    beta * momentum + grad; w = (1 - lr * weight_decay) * w - lr * scale *
    orthogonalize(grad + beta * momentum, or momentum without nesterov)."""
    B, rows, cols = _matrices("w", w)
    w_dt, g_dt = dtype_code(w), dtype_code(grad)
    _like("grad", grad, grad.dtype, w.shape, w.device)
    _like("momentum", momentum, torch.float32, w.shape, w.device)
    if spec is None:
        spec = OrthoSpec()
    update = OrthoUpdate(lr, beta, bool(nesterov), weight_decay, scale)
    with _at(w, stream):
        ws = _workspace(bmoe_orthogonalize_workspace_bytes(B, rows, cols),
                        "bmoe_orthogonalize_workspace_bytes", w.device)
        _check(bmoe_orthogonal_step(w_dt, g_dt, B, rows, cols, spec, update, grad, momentum, w, ws,
                                    stream), "bmoe_orthogonal_step")
        return w
