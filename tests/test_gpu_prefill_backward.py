"""Gradients of the kernelized prefill against the definition differentiated in
64 bits, and against differences (GPU).

Tolerances on the relative 2-norm. bf16 gradients: the last rounding (eps/2 =
2^-8) and, where the weights' gradients are rounded to bf16 for the tensor
cores, one more of the same size on independent terms: 2^-8 * sqrt(2), held to
6e-3. fp32 gradients: two products in a row, each under 2^-19 of its norm (terms
off by 2^-21, sums by at most 16 roundings of 2^-24 per tile and one per tile
after), and scores off by as much entering with the third power: 8 * 2^-19 =
1.5e-5, held to 2e-5.
"""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import prefill_forward, prefill_grads, rel

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 6e-3}
DTYPES = [torch.float32, torch.bfloat16]
NAMES = ("dq", "dk", "dv")


def inputs(B, H, T, d, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda: torch.randn(B, H, T, d, generator=gen)
    return [x.to(dtype).cuda() for x in (n() * d**-0.5, n() * d**-0.5, n(), n())]


def check(q, k, v, do, eps=1e-6, got=None):
    got = kata.prefill_backward(q, k, v, do, eps=eps) if got is None else got
    kata.sync_status()
    for name, a, b in zip(NAMES, got, prefill_grads(q, k, v, do, eps)):
        assert a.dtype == q.dtype
        assert rel(a, b) < TOL[q.dtype], name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 32, 64])
@pytest.mark.parametrize("T", [1, 2, 3, 15, 63, 64, 65, 127, 128, 129, 200, 256, 257, 385])
def test_grads(dtype, d, T):
    check(*inputs(2, 3, T, d, dtype, seed=d + T))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,T,d", [(1, 1, 1030, 64), (1, 2, 2048, 32), (7, 23, 70, 32),
                                     (3, 11, 140, 64)])
def test_larger(dtype, B, H, T, d):
    check(*inputs(B, H, T, d, dtype, seed=T))


@pytest.mark.parametrize("B,H,T,d", [(2, 8, 300, 16), (1, 4, 643, 64), (1, 5, 643, 32),
                                     (1, 1, 1025, 16), (1, 37, 512, 32)])
def test_shared_walks(B, H, T, d):
    # few rows: two, four, eight CTAs share a tile's walk, some of them without a
    # step of their own (the first rows); tiles of 32 and, in the last case, 64 rows
    x = inputs(B, H, T, d, torch.float32, seed=H + T)
    got = kata.prefill_backward(*x)
    check(*x, got=got)
    assert all(torch.equal(a, b) for a, b in zip(got, kata.prefill_backward(*x)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-2, 10.0])
def test_eps(dtype, eps):
    check(*inputs(1, 3, 150, 32, dtype, seed=3), eps=eps)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_key_dominates(dtype):
    # a key a hundred times the others: each later row is nearly that value, and
    # dP - delta is a small difference
    q, k, v, do = inputs(1, 2, 200, 32, dtype, seed=4)
    k[:, :, 20] *= 100
    check(q, k, v, do)


@pytest.mark.parametrize("dtype", DTYPES)
def test_orthogonal_first_keys(dtype):
    # rows 0 .. 3 see only keys with a score of exactly zero: o = 0, and with
    # eps their gradients are finite (zero, as the score enters squared)
    q, k, v, do = inputs(1, 2, 140, 32, dtype, seed=5)
    q[:, :, :4, :16] = 0
    k[:, :, :4, 16:] = 0
    check(q, k, v, do)
    for a in kata.prefill_backward(q, k, v, do, eps=0.0):
        assert bool(torch.isfinite(a).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_against_differences(dtype):
    q, k, v, do = inputs(1, 2, 100, 32, dtype, seed=6)
    got = kata.prefill_backward(q, k, v, do, eps=1e-3)
    xs = [x.double() for x in (q, k, v)]
    for i, name in enumerate(NAMES):
        r = torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).cuda().double()
        step = 1e-6
        up, dn = list(xs), list(xs)
        up[i], dn[i] = xs[i] + step * r, xs[i] - step * r
        want = float(((prefill_forward(*up, 1e-3) - prefill_forward(*dn, 1e-3)) * do.double()).sum())
        have = float((got[i].double() * r).sum())
        assert abs(have - want / (2 * step)) < TOL[dtype] * float(got[i].double().norm() * r.norm()), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_causal(dtype):
    # the last rows' upstream gradients reach no later key, and no later token
    # changes an earlier row's dq
    q, k, v, do = inputs(1, 2, 300, 64, dtype, seed=7)
    do2 = do.clone()
    do2[:, :, 100:] = 0
    dq, dk, dv = kata.prefill_backward(q, k, v, do2)
    assert not dq[:, :, 100:].any() and not dk[:, :, 100:].any() and not dv[:, :, 100:].any()
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 260:] *= 3
    v2[:, :, 260:] += 1
    assert torch.equal(kata.prefill_backward(q, k, v, do)[0][:, :, :260],
                       kata.prefill_backward(q, k2, v2, do)[0][:, :, :260])


@pytest.mark.parametrize("dtype", DTYPES)
def test_deterministic_and_given_workspace(dtype):
    x = inputs(2, 3, 333, 64, dtype, seed=8)
    want = kata.prefill_backward(*x)
    ws = torch.empty(kata.prefill_backward_workspace_bytes(2, 3, 333, 64, dtype), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(255)
    for a, b in zip(want, kata.prefill_backward(*x, workspace=ws)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_training_step(dtype):
    # forward and gradients together, as an autograd function would pair them
    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            ctx.save_for_backward(q, k, v)
            return kata.prefill(q, k, v, chunk=64, state=False)[0].to(q.dtype)

        @staticmethod
        def backward(ctx, do):
            return kata.prefill_backward(*ctx.saved_tensors, do.contiguous())

    q, k, v, do = inputs(1, 2, 256, 32, dtype, seed=9)
    xs = [x.clone().requires_grad_(True) for x in (q, k, v)]
    (Attend.apply(*xs) * do).sum().backward()
    check(q, k, v, do, got=[x.grad for x in xs])


@pytest.mark.parametrize("dtype", DTYPES)
def test_streams_and_graph(dtype):
    x = inputs(2, 2, 300, 64, dtype, seed=10)
    want = kata.prefill_backward(*x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [kata.prefill_backward(*x, stream=s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kata.prefill_backward(*x)
    y = inputs(2, 2, 300, 64, dtype, seed=11)
    for a, b in zip(x, y):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, kata.prefill_backward(*y)))


def test_refusals():
    q, k, v, do = inputs(1, 2, 64, 32, torch.bfloat16, seed=12)
    before = kata.launch_count()
    bad = [(dict(q=q.half()), "not float32"), (dict(k=k.float()), "k:"), (dict(v=v[:, :, :32]), "v:"),
           (dict(do=do.float()), "do:"), (dict(do=None), "do must not be None"),
           (dict(q=q[0]), "dimensions"), (dict(k=k.mT), "k:"), (dict(v=v.cpu()), "v:"),
           (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
           (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), "WORKSPACE")]
    for kw, message in bad:
        with pytest.raises(kata.KataError, match=message):
            kata.prefill_backward(**{**dict(q=q, k=k, v=v, do=do), **kw})
    for d in (8, 128):
        with pytest.raises(kata.KataError, match="UNSUPPORTED"):
            kata.prefill_backward(*inputs(1, 1, 4, d, torch.float32, seed=13))
    with pytest.raises(kata.KataError, match="INVALID_ARG"):
        kata.prefill_backward(*(t[:, :, :0].contiguous() for t in (q, k, v, do)))
    assert kata.launch_count() == before
