"""What the bindings of kata_delta.h and kata_backward.h share: binding the
entry points, checking tensors, and running a call on a device and stream."""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as kb
from ._binding import KataError

_bound = set()


def bind(signatures: dict) -> C.CDLL:
    """libkata.so with these entry points typed; raises if it has not been built."""
    handle = kb.lib()
    if id(signatures) not in _bound:
        for name, (res, args) in signatures.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _bound.add(id(signatures))
    return handle


def want(name: str, t, shape, dtype, like: torch.Tensor) -> None:
    """Raise unless t (None passes) is a contiguous tensor of this shape and
    type (None: any) on like's device."""
    if t is None:
        return
    if not t.is_cuda or not t.is_contiguous():
        raise KataError(f"{name}: tensors must be contiguous CUDA tensors")
    if ((shape is not None and t.shape != shape) or (dtype is not None and t.dtype != dtype)
            or t.device != like.device):
        raise KataError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected "
                        f"{None if shape is None else tuple(shape)} {dtype} on {like.device}")


class on_stream:
    """Runs a call on t's device and on `stream` (default: that device's current
    one), and gives the stream's handle. What the call allocates inside belongs
    to that stream."""

    def __init__(self, t: torch.Tensor, stream):
        if stream is not None and stream.device != t.device:
            raise KataError(f"stream of {stream.device}, tensors on {t.device}")
        self.inner = []
        if t.device.index != torch.cuda.current_device():
            self.inner.append(torch.cuda.device(t.device))
        if stream is not None:
            self.inner.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.inner:
            c.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        for c in reversed(self.inner):
            c.__exit__(*exc)
