"""Gradients of the kernelized prefill at rows whose denominators are next to nothing (GPU).
Inputs N(0, 1) scaled so that the squared scores reach the end of fp32's range."""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import prefill_grads, rel

pytestmark = pytest.mark.gpu

# as for ordinary scores: the last rounding and the operands' (bf16), products in split
# tf32 (fp32); the scale itself is a power of two and changes no rounding
TOL = {torch.float32: 2e-5, torch.bfloat16: 6e-3}


def inputs(T, d, dtype, scale):
    gen = torch.Generator().manual_seed(T)
    n = lambda s: (torch.randn(1, 3, T, d, generator=gen) * s).to(dtype).cuda()
    return n(scale * d**-0.5), n(scale * d**-0.5), n(1.0), n(1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_denominators_below_the_range(dtype, T):
    # scores of 2^-70 and less: squares below 2^-126 in rows of few keys, whose 1 / den has
    # no fp32 value; those rows give no gradient, and no row an infinity or a NaN
    for scale in (2.0**-33, 2.0**-35, 2.0**-36, 2.0**-60):
        x = inputs(T, 32, dtype, scale)
        for a in kata.prefill_backward(*x, eps=0.0):
            assert bool(torch.isfinite(a).all())
        assert not kata.prefill_backward(*inputs(T, 32, dtype, 2.0**-60), eps=0.0)[0].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [70, 300])
def test_small_scores_without_eps(dtype, T):
    # scores about 2^-40, squares about 2^-80, down to 2^-100 in single keys: in the range
    x = inputs(T, 32, dtype, 2.0**-20)
    for a, b in zip(kata.prefill_backward(*x, eps=0.0), prefill_grads(*x, 0.0)):
        assert rel(a, b) < TOL[dtype]
