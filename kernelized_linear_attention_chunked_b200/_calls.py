"""What the bindings of kata_delta.h and kata_backward.h share: binding the
entry points, checking tensors, and running a call on a device and stream."""
from __future__ import annotations

import contextlib
import ctypes as C
import functools

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


def fits(t, shape, dtype, dev) -> bool:
    """t is a contiguous tensor of this shape and type on CUDA device `dev`."""
    return (t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous())


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


@functools.lru_cache(maxsize=256)
def _bytes(lib, query: str, *sizes) -> int:
    return int(getattr(lib, query)(*sizes))


def workspace_for(lib, query: str, sizes, like: torch.Tensor) -> torch.Tensor:
    """A workspace of lib.query(*sizes) bytes beside the tensor `like` (that
    gives its device and type: 1 us less than naming them)."""
    item = like.element_size()
    return like.new_empty(max(1, -(-_bytes(lib, query, *sizes) // item)))


class on_stream:
    """Runs a call on t's device and on `stream` (default: that device's current
    one), and gives the stream's handle. What the call allocates inside belongs
    to that stream."""

    __slots__ = ("dev", "inner")

    def __init__(self, t: torch.Tensor, stream):
        self.dev = t.get_device()
        self.inner = None
        if stream is not None and stream.device != t.device:
            raise KataError(f"stream of {stream.device}, tensors on {t.device}")
        if stream is not None or self.dev != torch._C._cuda_getDevice():
            self.inner = contextlib.ExitStack()
            self.inner.enter_context(torch.cuda.device(self.dev))
            if stream is not None:
                self.inner.enter_context(torch.cuda.stream(stream))

    def __enter__(self):
        # torch.cuda.current_stream().cuda_stream without its Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(self.dev)

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)
