"""ctypes binding of the gated delta rule (include/kata_delta.h).

Argument marshalling only, like _binding.py. Tensors are checked for type,
shape, device and contiguity here, because the C ABI sees plain pointers.
Outputs and workspaces that are not given are allocated on the call's stream.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as kb
from ._binding import KataError, _check, _dt, _ptr
from ._calls import bind, fits, on_stream, want, workspace_for

_vp, _i, _f, _sz = C.c_void_p, C.c_int, C.c_float, C.c_size_t

# name -> (restype, argtypes), mirroring include/kata_delta.h
SIGNATURES = {
    "kata_delta_prefill_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "kata_delta_prefill": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp,
                                _vp, _sz, _vp]),
    "kata_delta_decode_step": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _f, _vp, _vp, _vp]),
    "kata_delta_backward_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "kata_delta_backward": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}


def lib() -> C.CDLL:
    """libkata.so with this header's entry points; raises if it has not been built."""
    return bind(SIGNATURES)


def _inputs(q, k, v, g, beta, ndim):
    """The tensors' type code and q's shape; raises unless they fit each other.
    One expression for the ordinary case: a call for single tokens is bound by
    the host."""
    f32 = torch.float32
    try:
        shape, dtype, dev = q.shape, q.dtype, q.get_device()
        rows = shape[:-1]
        if (len(shape) == ndim and dev >= 0 and dtype in kb._DTYPE and q.is_contiguous()
                and k.shape == shape and k.dtype is dtype and k.get_device() == dev
                and k.is_contiguous() and v.shape == shape and v.dtype is dtype
                and v.get_device() == dev and v.is_contiguous() and g.shape == rows
                and g.dtype is f32 and g.get_device() == dev and g.is_contiguous()
                and beta.shape == rows and beta.dtype is f32 and beta.get_device() == dev
                and beta.is_contiguous()):
            return kb._DTYPE[dtype], shape
    except AttributeError:
        pass
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if t is None:
            raise KataError(f"{name} must not be None")
    if q.dim() != ndim:
        raise KataError(f"q has {q.dim()} dimensions, expected {ndim}")
    dt = _dt(q)
    rows = q.shape[:-1]
    want("q", q, None, None, q)
    want("k", k, q.shape, q.dtype, q)
    want("v", v, q.shape, q.dtype, q)
    want("g", g, rows, f32, q)
    want("beta", beta, rows, f32, q)
    return dt, q.shape


def delta_prefill_workspace_bytes(B, H, T, d, dtype) -> int:
    return int(lib().kata_delta_prefill_workspace_bytes(B, H, T, d, kb._DTYPE[dtype]))


def delta_prefill(q, k, v, g, beta, scale: float | None = None, S_in=None, state: bool = True,
                  output: bool = True, o=None, S_out=None, workspace=None, stream=None):
    """The gated delta rule over q, k, v [B, H, T, d] with log decays g and
    writing strengths beta [B, H, T] (fp32), from the state S_in [B, H, d, d]
    (fp32, None: zero). ``scale`` defaults to d**-0.5. Returns (o, S): o in q's
    dtype, None when ``output`` is False and no buffer ``o`` is given; the last
    state, None when ``state`` is False and no ``S_out`` is given (it may be
    S_in). No autograd graph is recorded: delta_backward gives the gradients."""
    dt, shape = _inputs(q, k, v, g, beta, 4)
    B, H, T, d = shape
    st = (B, H, d, d)
    if S_in is not None:
        want("S_in", S_in, st, torch.float32, q)
    if S_out is not None:
        want("S_out", S_out, st, torch.float32, q)
    if o is not None:
        want("o", o, shape, q.dtype, q)
    if workspace is not None:
        want("workspace", workspace, None, None, q)
    scale = d ** -0.5 if scale is None else scale
    L = lib()
    with on_stream(q, stream) as s:
        if output and o is None:
            o = torch.empty_like(q)
        if state and S_out is None:
            S_out = g.new_empty(st)
        if workspace is None:
            workspace = workspace_for(L, "kata_delta_prefill_workspace_bytes", (B, H, T, d, dt), g)
        _check("kata_delta_prefill", L.kata_delta_prefill(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, g.data_ptr(), beta.data_ptr(), B, H, T,
            d, scale, _ptr(S_in), _ptr(o), _ptr(S_out), workspace.data_ptr(), workspace.nbytes, s))
    return o, S_out


def delta_decode_step(q, k, v, g, beta, S, scale: float | None = None, o=None, stream=None):
    """One token of the gated delta rule: q, k, v [B, H, d], g and beta [B, H]
    (fp32), the state S [B, H, d, d] (fp32) updated in place. Returns o in q's
    dtype. No autograd graph is recorded."""
    dt, shape = _inputs(q, k, v, g, beta, 3)
    B, H, d = shape
    if S is None:
        raise KataError("S must not be None")
    if not fits(S, (B, H, d, d), torch.float32, q.get_device()):
        want("S", S, (B, H, d, d), torch.float32, q)
    if o is not None:
        want("o", o, shape, q.dtype, q)
    scale = d ** -0.5 if scale is None else scale
    with on_stream(q, stream) as s:
        if o is None:
            o = torch.empty_like(q)
        _check("kata_delta_decode_step", lib().kata_delta_decode_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, g.data_ptr(), beta.data_ptr(), B, H, d,
            scale, S.data_ptr(), o.data_ptr(), s))
    return o


def delta_backward_workspace_bytes(B, H, T, d, dtype) -> int:
    return int(lib().kata_delta_backward_workspace_bytes(B, H, T, d, kb._DTYPE[dtype]))


def delta_backward(q, k, v, g, beta, do, scale: float | None = None, S_in=None, dS=None,
                   state_grad: bool = False, workspace=None, stream=None):
    """Gradients of delta_prefill for the gradient ``do`` of its output and
    ``dS`` [B, H, d, d] (fp32, None: zero) of its last state. Returns (dq, dk,
    dv, dg, dbeta, dS_in): the first three in q's dtype, the rest fp32; dS_in,
    the gradient of the first state, is None unless ``state_grad``."""
    dt, shape = _inputs(q, k, v, g, beta, 4)
    B, H, T, d = shape
    st = (B, H, d, d)
    if do is None:
        raise KataError("do must not be None")
    want("do", do, shape, q.dtype, q)
    if S_in is not None:
        want("S_in", S_in, st, torch.float32, q)
    if dS is not None:
        want("dS", dS, st, torch.float32, q)
    if workspace is not None:
        want("workspace", workspace, None, None, q)
    scale = d ** -0.5 if scale is None else scale
    L = lib()
    with on_stream(q, stream) as s:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        dg, db = torch.empty_like(g), torch.empty_like(beta)
        dS_in = g.new_empty(st) if state_grad else None
        if workspace is None:
            workspace = workspace_for(L, "kata_delta_backward_workspace_bytes", (B, H, T, d, dt), g)
        _check("kata_delta_backward", L.kata_delta_backward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, g.data_ptr(), beta.data_ptr(), B, H, T,
            d, scale, _ptr(S_in), do.data_ptr(), _ptr(dS), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), dg.data_ptr(), db.data_ptr(), _ptr(dS_in), workspace.data_ptr(),
            workspace.nbytes, s))
    return dq, dk, dv, dg, db, dS_in
