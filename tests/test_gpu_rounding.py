"""bf16 results against the 64-bit values rounded once (GPU).

The gradients of the prefill are held element by element: their largest rows are few and
far above the others, so a norm would be that of some hundred elements. With n the error of
an element before its rounding, |got - want| <= 2^-8 (|want| + |n|) + |n|. The operands P
and dS are in two bf16 parts, off by 2^-16 at most (half a step, 2^-8, of a rest that is
itself at most 2^-8 of the value), and fp32 sums of up to 2048 terms, sixteen at a time in
an accumulator that drops bits, by at most 128 * 2^-23 = 2^-16 of the terms' absolute sum.
The scores s and dP are sums of at most 64 exact products, off by at most 8 * 2^-23 = 2^-20
of the products' absolute sums; a row's 1 / den and delta as much again. So, with |S| and
|dP| the absolute sums (2^-19: the score itself and its row's sums),
    dV: |n| <= sum_i (2^-15 |P| + 2^-19 2 |s| |S| / den) |dO_i|
    dK: |n| <= sum_i (2^-15 |dS| + 2^-19 2 (|S| |dP - delta| + |s| (|dP| + |delta|)) / den) |q_i|
and dQ likewise. An operand rounded to 8 bits is off by up to 2^-8: small elements that
are sums of large ones fail.

The delta rule's are held by a norm. A result differs from the rounded 64-bit value only
where its error carries it over a border between two roundings, and then by one step. With
steps u_i <= 2^-7 |x_i| and values that lie evenly between the borders, that is the case
with probability |n_i| / u_i, so the expected square of the difference is sum |n_i| u_i <=
2^-7 |n| |x|: relative to |x| it is sqrt(2^-7 |n| / |x|). Operands in two bf16 parts give
|n| / |x| <= 2^-15 (twice their 2^-16, for sums that cancel a little), operands in two tf32
parts less: sqrt(2^-22) = 2^-11. With 24 such elements or more expected, a sample's norm is
at most 1.35 times the expected one (four standard deviations). Operands cut to 11 bits
(2^-10) would give 2^-9.
"""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import delta_forward, delta_grads, delta_inputs, prefill_grads, rel

pytestmark = pytest.mark.gpu


def check(got, want, name=""):
    assert got.dtype == torch.bfloat16
    assert rel(got, want.to(torch.bfloat16)) < 1.35 * 2**-11, name


def prefill_errors(q, k, v, do, eps):
    """The bounds above on the errors of dq, dk and dv before their rounding."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    s, S = (q @ k.mT).tril(), (q.abs() @ k.abs().mT).tril()
    dp, DP = do @ v.mT, do.abs() @ v.abs().mT
    den = (s**2).sum(-1, keepdim=True) + eps
    delta = (s**2 * dp).sum(-1, keepdim=True) / den
    ds = 2 * s * (dp - delta) / den
    nds = 2**-15 * ds.abs() + 2**-19 * 2 * (S * (dp - delta).abs() + s.abs() * (DP + delta.abs())) / den
    np = 2**-15 * s**2 / den + 2**-19 * 2 * s.abs() * S / den
    return nds @ k.abs(), nds.mT @ q.abs(), np.mT @ do.abs()


@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("B,H,T", [(2, 3, 200), (1, 3, 1030), (1, 2, 2048)])
def test_prefill_gradients(B, H, T, d):
    gen = torch.Generator().manual_seed(T + d)
    n = lambda: torch.randn(B, H, T, d, generator=gen)
    x = [t.bfloat16().cuda() for t in (n() * d**-0.5, n() * d**-0.5, n(), n())]
    got = kata.prefill_backward(*x)
    kata.sync_status()
    for name, a, b, e in zip(("dq", "dk", "dv"), got, prefill_grads(*x, 1e-6), prefill_errors(*x, 1e-6)):
        assert a.dtype == torch.bfloat16
        over = (a.double() - b).abs() - (2**-8 * (b.abs() + e) + e)
        assert not (over > 0).any(), (name, int((over > 0).sum()), a.numel())


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H,T", [(2, 3, 63), (2, 3, 200), (1, 2, 1000)])
def test_delta_prefill(B, H, T, d):
    x = delta_inputs(B, H, T, d, torch.bfloat16, seed=T + d)
    o, _ = kata.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], S_in=x["S"])
    kata.sync_status()
    check(o, delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], d**-0.5, x["S"])[0])


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H,T", [(2, 3, 63), (2, 3, 200), (1, 2, 500)])
def test_delta_gradients(B, H, T, d):
    x = delta_inputs(B, H, T, d, torch.bfloat16, seed=T + d)
    got = kata.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], S_in=x["S"],
                              dS=x["dS"])
    kata.sync_status()
    want = delta_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], d**-0.5, x["do"], x["S"], x["dS"])
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        check(a, b, name)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_delta_step(d):
    x = delta_inputs(40, 7, 1, d, torch.bfloat16, seed=d)
    S = x["S"].clone()
    o = kata.delta_decode_step(*(x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")), S)
    kata.sync_status()
    want = delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], d**-0.5, x["S"])[0]
    check(o, want[:, :, 0])
