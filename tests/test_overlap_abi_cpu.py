"""Buffers of the delta rule's calls and of the gradients that overlap are refused before any
launch, at the same address or in part; the pairs that the headers allow are not (CPU).

Calls that pass the check of the outputs against the inputs stop at a workspace that is too
small, so that none of them can launch anything."""
import ctypes as C

import pytest

import kernelized_linear_attention_chunked_b200 as kata
from kernelized_linear_attention_chunked_b200 import _backward, _delta

INVALID, SHORT = 1, 5
B, H, T, d = 1, 2, 100, 32
X, Y, Z = B * H * T * d * 2, B * H * T * 4, B * H * d * d * 4  # bytes of q (bf16), g and a state


def call(library, fn, sizes, order, **kw):
    """Every buffer (never dereferenced) a megabyte from the next unless kw places it."""
    at = {n: (i + 1) << 20 for i, n in enumerate(sizes)}
    at.update(kw)
    before = kata.launch_count()
    status = getattr(library, fn)(*[C.c_void_p(at[n]) if n in at else n for n in order], None)
    assert kata.launch_count() == before
    return status, (kata.lib().kata_last_error() or b"").decode()


def prefill(ws_bytes, **kw):
    sizes = dict(q=X, k=X, v=X, g=Y, beta=Y, S_in=Z, o=X, S_out=Z, ws=0)
    return call(_delta.lib(), "kata_delta_prefill", sizes,
                ["q", "k", "v", 1, "g", "beta", B, H, T, d, 1.0, "S_in", "o", "S_out", "ws", ws_bytes], **kw)


def backward(ws_bytes, **kw):
    sizes = dict(q=X, k=X, v=X, g=Y, beta=Y, S_in=Z, d_o=X, dS_out=Z, dq=X, dk=X, dv=X, dg=Y, dbeta=Y,
                 dS_in=Z, ws=0)
    return call(_delta.lib(), "kata_delta_backward", sizes,
                ["q", "k", "v", 1, "g", "beta", B, H, T, d, 1.0, "S_in", "d_o", "dS_out", "dq", "dk", "dv",
                 "dg", "dbeta", "dS_in", "ws", ws_bytes], **kw)


def attention(ws_bytes, **kw):
    sizes = dict(q=X, k=X, v=X, d_o=X, dq=X, dk=X, dv=X, ws=0)
    return call(_backward.lib(), "kata_prefill_backward", sizes,
                ["q", "k", "v", 1, B, H, T, d, 1e-6, "d_o", "dq", "dk", "dv", "ws", ws_bytes], **kw)


BYTES = dict(g=Y, beta=Y, dg=Y, dbeta=Y, S_in=Z, S_out=Z, dS_in=Z, dS_out=Z, S=Z)
CALLS = [(prefill, ("q", "k", "v", "g", "beta", "S_in"), ("o", "S_out"), {("S_out", "S_in")}),
         (backward, ("q", "k", "v", "g", "beta", "S_in", "d_o", "dS_out"),
          ("dq", "dk", "dv", "dg", "dbeta", "dS_in"), {("dS_in", "dS_out")}),
         (attention, ("q", "k", "v", "d_o"), ("dq", "dk", "dv"), set())]
PAIRS = [(fn, o, i, (o, i) in allowed) for fn, ins, outs, allowed in CALLS for o in outs for i in ins]
BASE = 1 << 30


@pytest.mark.parametrize("fn,out,inp,allowed", PAIRS)
def test_outputs_over_inputs(fn, out, inp, allowed):
    no, ni = BYTES.get(out, X), BYTES.get(inp, X)
    status, message = fn(0, **{out: BASE, inp: BASE})
    assert status == (SHORT if allowed else INVALID)
    if not allowed:
        assert f"{out} must not overwrite {inp}" == message
    for shift in (16, ni - 16, -16, 16 - no):  # in part, from either side
        assert fn(0, **{out: BASE + shift, inp: BASE})[0] == INVALID, shift
    for shift in (ni, -no):  # next to each other
        assert fn(0, **{out: BASE + shift, inp: BASE})[0] == SHORT, shift


@pytest.mark.parametrize("fn,names", [(fn, outs) for fn, _, outs, _ in CALLS])
def test_outputs_over_each_other(fn, names):
    for i, a in enumerate(names):
        for b in names[:i]:
            for shift in (0, 16):
                status, message = fn(1 << 40, **{a: BASE + shift, b: BASE})
                assert status == INVALID and "must not overwrite" in message


@pytest.mark.parametrize("fn,names", [(fn, ins + outs) for fn, ins, outs, _ in CALLS])
def test_workspace_over_anything(fn, names):
    for n in names:
        for at in (BASE, BASE + 1024):
            status, message = fn(1 << 40, ws=BASE, **{n: at})
            assert status == INVALID and message == f"workspace must not overwrite {n}"


@pytest.mark.parametrize("out", ["S", "o"])
@pytest.mark.parametrize("inp", ["q", "k", "v", "g", "beta", "S"])
def test_step(out, inp):
    if out == inp:
        return
    x, y, z = B * H * d * 2, B * H * 4, Z
    sizes = dict(q=x, k=x, v=x, g=y, beta=y, S=z, o=x)
    for shift in (0, 16 if inp in "qkvS" else 0, 16 - sizes[out]):
        status, message = call(_delta.lib(), "kata_delta_decode_step", sizes,
                               ["q", "k", "v", 1, "g", "beta", B, H, d, 1.0, "S", "o"],
                               **{out: BASE + shift, inp: BASE})
        assert status == INVALID and message == f"{out} must not overwrite {inp}"
