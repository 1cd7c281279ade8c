"""The delta rule and the gradients where offsets pass 32 bits (GPU): more than 2^31
elements per tensor, whose last heads give the same bits as those heads by themselves."""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata

pytestmark = pytest.mark.gpu

B, H, T, d = 32, 1050, 1000, 64  # 2.15e9 elements; fifteen 64-token chunks and a part
LAST = (slice(B - 1, B), slice(H - 3, H))


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130e9:
        pytest.skip("needs 130 GB")
    yield
    torch.cuda.empty_cache()


def rows(n, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.empty(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        x[b].normal_(0, scale, generator=gen)
    assert x.numel() > 1 << 31
    return x


def part(t):
    return t[LAST].contiguous()


def same(whole, alone):
    kata.sync_status()
    for a, b in zip(whole, alone):
        assert torch.equal(part(a), b)
        assert bool(torch.isfinite(b).all()) and b.any()


def rule():
    q, k, v = rows(1), rows(2, d**-0.5), rows(3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = -0.3 * torch.rand(B, H, T, device="cuda", generator=gen)
    beta = torch.rand(B, H, T, device="cuda", generator=gen)
    return q, k, v, g, beta


def test_delta_prefill():
    x = rule()
    same(kata.delta_prefill(*x), kata.delta_prefill(*map(part, x)))


def test_delta_backward():
    x = (*rule(), rows(5))
    same(kata.delta_backward(*x)[:5], kata.delta_backward(*map(part, x))[:5])


def test_prefill_backward():
    x = rows(1, d**-0.5), rows(2, d**-0.5), rows(3), rows(5)
    same(kata.prefill_backward(*x), kata.prefill_backward(*map(part, x)))


def test_step():
    heads, w = (B, 4100), 128  # 2.15e9 elements of the state
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*heads, *s, device="cuda", generator=gen)
    S = n(w, w)
    assert S.numel() > 1 << 31
    x = [n(w).bfloat16(), (n(w) * w**-0.5).bfloat16(), n(w).bfloat16(), -n().abs(), n().sigmoid()]
    last = slice(heads[0] - 1, heads[0]), slice(heads[1] - 3, heads[1])
    S1 = S[last].clone()
    o = kata.delta_decode_step(*x, S)
    o1 = kata.delta_decode_step(*(t[last].contiguous() for t in x), S1)
    kata.sync_status()
    assert torch.equal(o[last], o1) and torch.equal(S[last], S1)
    assert bool(torch.isfinite(o1).all()) and o1.any()
