"""The entry points of kata_delta.h and kata_backward.h: exported, bound as
declared, and refusing invalid arguments with a status before any launch (CPU)."""
import ctypes as C
import re
from pathlib import Path

import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from kernelized_linear_attention_chunked_b200 import _backward, _binding, _delta

INCLUDE = Path(__file__).resolve().parent.parent / "include"
HEADERS = [("kata_delta.h", _delta.SIGNATURES), ("kata_backward.h", _backward.SIGNATURES)]
FAKE = C.c_void_p(1 << 20)  # aligned, never dereferenced: validation fails first
OTHER = C.c_void_p(1 << 21)
MISALIGNED = C.c_void_p((1 << 20) + 4)
ODD = C.c_void_p((1 << 20) + 2)


@pytest.mark.parametrize("header,signatures", HEADERS)
def test_declared_exported_and_bound(header, signatures):
    text = (INCLUDE / header).read_text()
    names = re.findall(r"KATA_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == set(signatures) and len(names) == len(set(names))
    assert not set(names) & set(_binding.SIGNATURES)
    for name, (_, args) in signatures.items():
        assert hasattr(kata.lib(), name)
        params = re.search(r"KATA_API[^;(]*\b" + name + r"\(([^)]*)\)", text).group(1)
        assert len([p for p in params.split(",") if p.strip()]) == len(args), name


def delta_prefill(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, g=FAKE, beta=FAKE, B=1, H=1, T=100, d=64, scale=1.0,
             S_in=None, o=OTHER, S_out=OTHER, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return _delta.lib().kata_delta_prefill(*a.values(), None)


def delta_step(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, g=FAKE, beta=FAKE, B=1, H=1, d=64, scale=1.0, S=OTHER,
             o=OTHER)
    a.update(kw)
    return _delta.lib().kata_delta_decode_step(*a.values(), None)


def delta_backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, g=FAKE, beta=FAKE, B=1, H=1, T=100, d=64, scale=1.0,
             S_in=None, d_o=FAKE, dS_out=None, dq=OTHER, dk=OTHER, dv=OTHER, dg=OTHER, dbeta=OTHER,
             dS_in=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return _delta.lib().kata_delta_backward(*a.values(), None)


def prefill_backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=1, B=1, H=1, T=100, d=64, eps=1e-6, d_o=FAKE, dq=OTHER,
             dk=OTHER, dv=OTHER, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return _backward.lib().kata_prefill_backward(*a.values(), None)


COMMON = [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(q=MISALIGNED), 1),
          (dict(v=MISALIGNED), 1), (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(B=0), 1),
          (dict(H=-1), 1), (dict(B=1 << 15, H=1 << 15), 1), (dict(d=0), 2), (dict(d=24), 2),
          (dict(d=256), 2)]
SEQUENCE = [(dict(T=0), 1), (dict(T=-5), 1), (dict(T=(1 << 24) + 1), 1),
            (dict(B=1 << 10, H=1 << 10, T=1 << 24), 1), (dict(ws=None), 5), (dict(ws_bytes=100), 5),
            (dict(ws=MISALIGNED), 1)]
RULE = [(dict(g=None), 1), (dict(beta=None), 1), (dict(g=ODD), 1), (dict(beta=ODD), 1),
        (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1)]


@pytest.mark.parametrize("kw,status", COMMON + SEQUENCE + RULE + [
    (dict(o=None, S_out=None), 1), (dict(S_in=MISALIGNED), 1), (dict(o=MISALIGNED), 1),
    (dict(S_out=MISALIGNED), 1), (dict(o=FAKE), 1)])
def test_delta_prefill_refuses(kw, status):
    before = kata.launch_count()
    assert delta_prefill(**kw) == status
    assert kata.lib().kata_last_error() and kata.launch_count() == before


@pytest.mark.parametrize("kw,status", COMMON + RULE + [
    (dict(S=None), 1), (dict(o=None), 1), (dict(S=MISALIGNED), 1), (dict(o=FAKE), 1)])
def test_delta_step_refuses(kw, status):
    before = kata.launch_count()
    assert delta_step(**kw) == status
    assert kata.lib().kata_last_error() and kata.launch_count() == before


@pytest.mark.parametrize("kw,status", COMMON + SEQUENCE + RULE + [
    (dict(d_o=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1),
    (dict(dg=None), 1), (dict(dbeta=None), 1), (dict(dS_out=MISALIGNED), 1),
    (dict(dS_in=MISALIGNED), 1), (dict(dg=ODD), 1)])
def test_delta_backward_refuses(kw, status):
    before = kata.launch_count()
    assert delta_backward(**kw) == status
    assert kata.lib().kata_last_error() and kata.launch_count() == before


@pytest.mark.parametrize("kw,status", COMMON + SEQUENCE + [
    (dict(d=128), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(d_o=None), 1),
    (dict(dq=None), 1), (dict(dk=MISALIGNED), 1), (dict(dv=None), 1)])
def test_prefill_backward_refuses(kw, status):
    before = kata.launch_count()
    assert prefill_backward(**kw) == status
    assert kata.lib().kata_last_error() and kata.launch_count() == before


def test_workspace_queries():
    bf = torch.bfloat16
    for fn in (kata.delta_prefill_workspace_bytes, kata.delta_backward_workspace_bytes,
               kata.prefill_backward_workspace_bytes):
        assert fn(2, 8, 1000, 64, bf) > 0
        assert fn(2, 8, 0, 64, bf) == 0 and fn(0, 8, 10, 64, bf) == 0 and fn(2, 8, 10, 24, bf) == 0
        # sizes are 64 bits wide
        assert fn(8, 64, 1 << 20, 64, bf) > 1 << 32
        # a chunk's worth more for the token after a whole number of chunks, never less
        assert fn(1, 1, 65, 64, bf) >= fn(1, 1, 64, 64, bf)
    assert kata.delta_prefill_workspace_bytes(1, 1, 65, 128, bf) == \
        2 * kata.delta_prefill_workspace_bytes(1, 1, 64, 128, bf)


@pytest.mark.parametrize("call", [
    lambda x: kata.delta_prefill(x, x, x, x[..., 0], x[..., 0]),
    lambda x: kata.delta_backward(x, x, x, x[..., 0], x[..., 0], x),
    lambda x: kata.delta_decode_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], x[:, :, 0, 0], x[:, :, 0, 0],
                                     None),
    lambda x: kata.prefill_backward(x, x, x, x)])
def test_host_tensors_are_refused(call):
    with pytest.raises(kata.KataError):
        call(torch.zeros(1, 1, 4, 16))
