"""ctypes binding of the prefill's gradients (include/kata_backward.h).

Argument marshalling only, like _binding.py; tensors are checked here, because
the C ABI sees plain pointers.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as kb
from ._binding import KataError, _check, _dt
from ._calls import bind, on_stream, want, workspace_for

_vp, _i, _f, _sz = C.c_void_p, C.c_int, C.c_float, C.c_size_t

# name -> (restype, argtypes), mirroring include/kata_backward.h
SIGNATURES = {
    "kata_prefill_backward_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "kata_prefill_backward": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp,
                                   _sz, _vp]),
}


def lib() -> C.CDLL:
    """libkata.so with this header's entry points; raises if it has not been built."""
    return bind(SIGNATURES)


def prefill_backward_workspace_bytes(B, H, T, d, dtype) -> int:
    return int(lib().kata_prefill_backward_workspace_bytes(B, H, T, d, kb._DTYPE[dtype]))


def _inputs(q, k, v, do):
    """The tensors' type code and shape; raises unless they fit each other. One
    expression for the ordinary case: a short call is bound by the host."""
    try:
        shape, dtype, dev = q.shape, q.dtype, q.get_device()
        if (len(shape) == 4 and dev >= 0 and dtype in kb._DTYPE and q.is_contiguous()
                and k.shape == shape and k.dtype is dtype and k.get_device() == dev
                and k.is_contiguous() and v.shape == shape and v.dtype is dtype
                and v.get_device() == dev and v.is_contiguous() and do.shape == shape
                and do.dtype is dtype and do.get_device() == dev and do.is_contiguous()):
            return kb._DTYPE[dtype], shape
    except AttributeError:
        pass
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        if t is None:
            raise KataError(f"{name} must not be None")
    if q.dim() != 4:
        raise KataError(f"q has {q.dim()} dimensions, expected 4")
    dt = _dt(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        want(name, t, q.shape, q.dtype, q)
    return dt, q.shape


def prefill_backward(q, k, v, do, eps: float = 1e-6, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of prefill's output from a zero state, for the
    output's gradient ``do``. All [B, H, T, d] in q's dtype; any T. (prefill's own
    output is fp32 for bf16 inputs as well: its gradient has to be cast.)"""
    dt, shape = _inputs(q, k, v, do)
    B, H, T, d = shape
    if workspace is not None:
        want("workspace", workspace, None, None, q)
    L = lib()
    with on_stream(q, stream) as s:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        if workspace is None:
            workspace = workspace_for(L, "kata_prefill_backward_workspace_bytes",
                                      (B, H, T, d, dt), q)
        _check("kata_prefill_backward", L.kata_prefill_backward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, B, H, T, d, eps, do.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.nbytes, s))
    return dq, dk, dv
