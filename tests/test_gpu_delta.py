"""The gated delta rule (prefill, one-token step, gradients) against its
definition in 64 bits, token by token, at the sizes and values where it can go
wrong (GPU).

Tolerances on the relative 2-norm. bf16 results: the final rounding is at most
2^-9 of the value's binade, that is eps/2 = 2^-8 relative; o may add one tf32
part's truncation (2^-10) on each factor of its two products. fp32 results
pass at most six products in a row; a product's terms are off by 2^-21 and its
sums by at most 16 roundings of 2^-24, together under 2^-19 of its norm; the
inverse of a chunk may amplify them a few times: 6 * 2^-19 * 2 = 2.3e-5, held
to 2e-5.
"""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import delta_forward, delta_grads, delta_inputs, rel

pytestmark = pytest.mark.gpu

F32 = 2e-5
TOL = {torch.float32: F32, torch.bfloat16: 2**-8}
DTYPES = [torch.float32, torch.bfloat16]
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS_in")


def prefill(x, **kw):
    return kata.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], S_in=x["S"], **kw)


def backward(x, **kw):
    return kata.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], S_in=x["S"],
                               dS=x["dS"], state_grad=True, **kw)


def check_prefill(x, tol_o=None, tol_s=F32, scale=None):
    d = x["q"].shape[-1]
    sc = d ** -0.5 if scale is None else scale
    o, S = prefill(x, scale=scale)
    kata.sync_status()
    ro, rS = delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], sc, x["S"])
    assert o.dtype == x["q"].dtype and S.dtype == torch.float32
    assert rel(o, ro) < (tol_o or TOL[x["q"].dtype])
    assert rel(S, rS) < tol_s


def check_backward(x, tol=F32, scale=None):
    d = x["q"].shape[-1]
    sc = d ** -0.5 if scale is None else scale
    got = backward(x, scale=scale)
    kata.sync_status()
    want = delta_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], sc, x["do"], x["S"], x["dS"])
    for name, a, b in zip(NAMES, got, want):
        t = max(tol, TOL[a.dtype]) if a.dtype == torch.bfloat16 else tol
        assert rel(a, b) < t, name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 15, 63, 64, 65, 130, 200])
def test_prefill(dtype, d, T):
    check_prefill(delta_inputs(2, 3, T, d, dtype, seed=d + T, state=T % 2 == 1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 17, 64, 65, 150])
def test_backward(dtype, d, T):
    check_backward(delta_inputs(1, 3, T, d, dtype, seed=d + T + 7, state=T % 2 == 1))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_backward_against_differences(d):
    # the gradient along a random direction of each input against central
    # differences of the 64-bit definition (step 1e-5: an error of 1e-10)
    x = delta_inputs(1, 2, 70, d, torch.float32, seed=d + 31)
    got = backward(x)
    scale = d ** -0.5
    xs = [x[n].double() for n in ("q", "k", "v", "g", "beta", "S")]

    def loss(a):
        o, S = delta_forward(*a[:5], scale, a[5])
        return float((o * x["do"].double()).sum() + (S * x["dS"].double()).sum())

    for i, name in enumerate(NAMES):
        r = torch.randn(xs[i].shape, generator=torch.Generator().manual_seed(i)).cuda().double()
        up, dn = list(xs), list(xs)
        up[i], dn[i] = xs[i] + 1e-5 * r, xs[i] - 1e-5 * r
        want = (loss(up) - loss(dn)) / 2e-5
        have = float((got[i].double() * r).sum())
        norm = float(got[i].double().norm() * r.norm())
        assert abs(have - want) < F32 * norm, name


@pytest.mark.parametrize("dtype", DTYPES)
def test_long(dtype):
    check_prefill(delta_inputs(1, 2, 4097, 64, dtype, seed=5))


def test_long_backward():
    check_backward(delta_inputs(1, 2, 1000, 32, torch.bfloat16, seed=6))


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_heads(dtype):
    check_prefill(delta_inputs(9, 35, 66, 32, dtype, seed=7))
    check_backward(delta_inputs(5, 35, 66, 16, dtype, seed=8))


@pytest.mark.parametrize("dtype", DTYPES)
def test_repeated_keys_full_strength(dtype):
    # the same few keys over and over, written at beta = 1 without decay: the
    # chunk's triangular system at its worst conditioning
    x = delta_inputs(1, 2, 300, 64, dtype, seed=9, keys=5)
    x["beta"].fill_(1.0)
    x["g"].zero_()
    check_prefill(x)
    check_backward(x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_decay_long(dtype):
    x = delta_inputs(1, 1, 2048, 32, dtype, seed=10)
    x["g"].zero_()
    check_prefill(x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", [-30.0, -1e4, -3.0e38, float("-inf")])
def test_strong_decay(dtype, low):
    # a decay to nothing in the middle of a chunk starts the state anew, and
    # later small decays keep their digits
    x = delta_inputs(1, 2, 150, 32, dtype, seed=11)
    x["g"][:, :, [0, 40, 41, 64, 127]] = low
    check_prefill(x)
    got = backward(x)
    y = dict(x, g=x["g"].clamp(min=-200.0))  # exp of either is 0 in fp32
    want = delta_grads(y["q"], y["k"], y["v"], y["g"], y["beta"], 32 ** -0.5, y["do"], y["S"], y["dS"])
    for name, a, b in zip(NAMES, got, want):
        if name == "dS_in":  # under exp(-30) or nothing at all
            assert float((a.double() - b).abs().max()) <= F32 * float(x["dS"].abs().max())
        else:
            assert rel(a, b) < TOL[a.dtype], name


def test_zero_strength_changes_nothing():
    # padding tokens (beta = 0, g = 0) behind a sequence leave its state and its
    # outputs bit for bit, and get no gradient but v's zeros
    x = delta_inputs(2, 2, 128, 64, torch.bfloat16, seed=12)
    x["beta"][:, :, 70:] = 0.0
    x["g"][:, :, 70:] = 0.0
    o, S = prefill(x)
    short = {n: (t[:, :, :70].contiguous() if t.dim() >= 3 and t.shape[2] == 128 else t)
             for n, t in x.items()}
    o2, S2 = prefill(short)
    assert torch.equal(o[:, :, :70], o2)
    assert rel(S, S2) < 1e-6
    ro, rS = delta_forward(short["q"], short["k"], short["v"], short["g"], short["beta"], 0.125,
                           short["S"])
    assert rel(S, rS) < F32
    assert not backward(x)[2][:, :, 70:].any()


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_scale(scale):
    x = delta_inputs(1, 2, 70, 32, torch.float32, seed=13)
    o, S = prefill(x, scale=scale)
    ro, rS = delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["S"])
    assert rel(S, rS) < F32
    if scale:
        assert rel(o, ro) < F32
        check_backward(x, scale=scale)
    else:
        assert not o.any()


def test_large_and_small_values():
    for f in (1e4, 1e-4):
        x = delta_inputs(1, 2, 100, 32, torch.float32, seed=14)
        x["v"] *= f
        x["S"] *= f
        check_prefill(x)


def test_outputs_on_request():
    x = delta_inputs(2, 2, 100, 64, torch.bfloat16, seed=15)
    o, S = prefill(x)
    o1, none = prefill(x, state=False)
    none2, S1 = prefill(x, output=False)
    assert none is None and none2 is None
    assert torch.equal(o, o1) and torch.equal(S, S1)
    assert kata.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"])[5] is None


def test_state_in_place_and_given_buffers():
    x = delta_inputs(2, 2, 100, 64, torch.bfloat16, seed=16)
    o, S = prefill(x)
    buf, out = x["S"].clone(), torch.empty_like(o)
    ws = torch.empty(kata.delta_prefill_workspace_bytes(2, 2, 100, 64, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # NaN everywhere: nothing in it is read before it is written
    o2, S2 = kata.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], S_in=buf, S_out=buf,
                                o=out, workspace=ws)
    assert S2 is buf and o2 is out
    assert torch.equal(o, o2) and torch.equal(S, S2)
    want = backward(x)
    ws = torch.empty(kata.delta_backward_workspace_bytes(2, 2, 100, 64, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    for a, b in zip(want, backward(x, workspace=ws)):
        assert torch.equal(a, b)


def test_rows_behind_the_last_are_left():
    # the buffers continue after the last row: nothing there is written
    x = delta_inputs(1, 1, 65, 16, torch.bfloat16, seed=17)
    room = torch.full((1, 1, 129, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    o = room[:, :, :65]
    kata.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], S_in=x["S"], o=o)
    assert bool((room[:, :, 65:] == 7.0).all()) and rel(o, prefill(x)[0]) == 0.0


def test_deterministic():
    x = delta_inputs(3, 4, 333, 64, torch.bfloat16, seed=18)
    assert all(torch.equal(a, b) for a, b in zip(prefill(x), prefill(x)))
    assert all(torch.equal(a, b) for a, b in zip(backward(x), backward(x)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (40, 7)])
def test_decode(dtype, d, B, H):
    steps = 5
    x = delta_inputs(B, H, steps, d, dtype, seed=d + B)
    x["g"][:, :, 2] = float("-inf")
    S = x["S"].clone()
    out = []
    for t in range(steps):
        out.append(kata.delta_decode_step(*(x[n][:, :, t].contiguous()
                                            for n in ("q", "k", "v", "g", "beta")), S))
    kata.sync_status()
    ro, rS = delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], d ** -0.5, x["S"])
    # fp32: at most d roundings of 2^-24 per sum and step
    assert rel(torch.stack(out, 2), ro) < (1e-6 if dtype == torch.float32 else 2**-8)
    assert rel(S, rS) < 1e-6


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [32, 128])
def test_prefill_then_decode_then_prefill(dtype, d):
    # a served sequence: a prompt, some tokens, another prompt
    T, cut, more = 150, 83, 9
    x = delta_inputs(2, 2, T, d, dtype, seed=d + 40)
    part = lambda a, b: [x[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")]
    o1, S = kata.delta_prefill(*part(0, cut), S_in=x["S"])
    mid = [kata.delta_decode_step(*(p.squeeze(2) for p in part(t, t + 1)), S)
           for t in range(cut, cut + more)]
    o3, S = kata.delta_prefill(*part(cut + more, T), S_in=S, S_out=S)
    o = torch.cat([o1, torch.stack(mid, 2), o3], 2)
    ro, rS = delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], d ** -0.5, x["S"])
    assert rel(o, ro) < TOL[dtype] and rel(S, rS) < F32


def test_gradient_chains_over_parts():
    # gradients of a sequence taken in two parts through the state between them
    d, T, cut = 32, 140, 75
    x = delta_inputs(1, 2, T, d, torch.float32, seed=50)
    names = ("q", "k", "v", "g", "beta", "do")
    part = lambda a, b: {n: x[n][:, :, a:b].contiguous() for n in names}
    a, b = part(0, cut), part(cut, T)
    _, mid = prefill(dict(a, S=x["S"]))
    gb = backward(dict(b, S=mid, dS=x["dS"]))
    ga = backward(dict(a, S=x["S"], dS=gb[5]))
    want = delta_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], d ** -0.5, x["do"], x["S"], x["dS"])
    for i in range(5):
        assert rel(torch.cat([ga[i], gb[i]], 2), want[i]) < F32
    assert rel(ga[5], want[5]) < F32


def test_autograd_training_step():
    # as a training loop uses the pair: inside an autograd function
    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, g, beta):
            ctx.save_for_backward(q, k, v, g, beta)
            return kata.delta_prefill(q, k, v, g, beta, state=False)[0]

        @staticmethod
        def backward(ctx, do):
            return kata.delta_backward(*ctx.saved_tensors, do.contiguous())[:5]

    x = delta_inputs(2, 2, 90, 32, torch.float32, seed=60, state=False)
    xs = [x[n].clone().requires_grad_(True) for n in ("q", "k", "v", "g", "beta")]
    (Rule.apply(*xs) * x["do"]).sum().backward()
    want = delta_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], 32 ** -0.5, x["do"])
    for a, b in zip(xs, want):
        assert rel(a.grad, b) < F32


def test_on_another_stream():
    x = delta_inputs(2, 2, 200, 64, torch.bfloat16, seed=61)
    want, grads = prefill(x), backward(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, got_g = prefill(x, stream=s), backward(x, stream=s)
    S = x["S"].clone()
    s.wait_stream(torch.cuda.current_stream())
    o = kata.delta_decode_step(*(x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")),
                               S, stream=torch.cuda.current_stream())
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(grads, got_g))
    first = delta_forward(*(x[n][:, :, :1] for n in ("q", "k", "v", "g", "beta")), 0.125, x["S"])
    assert rel(o, first[0][:, :, 0]) < 2**-8 and rel(S, first[1]) < 1e-6


def test_two_calls_at_once():
    # two streams, each with its own buffers
    xs = [delta_inputs(2, 4, 500, 64, torch.bfloat16, seed=70 + i) for i in range(2)]
    want = [(prefill(x), backward(x)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = [(prefill(x, stream=s), backward(x, stream=s)) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w[0] + w[1], g[0] + g[1]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_back_to_back(dtype):
    # every call right after the kernels that write its inputs and right before
    # those that overwrite them, the framework's own others between: the same bits
    # as with a pause after each
    base = delta_inputs(2, 4, 333, 32, dtype, seed=21)

    def run(pause):
        out = []
        for i in range(8):
            x = {n: t.clone() for n, t in base.items()}
            x["v"].mul_(1 + i / 8)
            pause()
            o, S = prefill(x)
            pause()
            last = [x[n][:, :, -1].contiguous() for n in ("q", "k", "v", "g", "beta")]
            o1 = kata.delta_decode_step(*last, S)
            pause()
            x["do"].copy_(o)
            grads = backward(x)
            pause()
            y = [x[n][:, :, :256].contiguous() for n in ("q", "k", "v")]
            w = kata.prefill(*y, chunk=64, state=False)[0].to(dtype)
            pause()
            more = kata.prefill_backward(*y, w)
            pause()
            for t in (*x.values(), *y, w):
                t.zero_()
            pause()
            out += [o, S, o1, *grads, *more]
        torch.cuda.synchronize()
        kata.sync_status()
        return out

    for a, b in zip(run(torch.cuda.synchronize), run(lambda: None)):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    x = delta_inputs(2, 2, 200, 64, torch.bfloat16, seed=80)
    names = ("q", "k", "v", "g", "beta")
    S = x["S"].clone()
    step = {n: x[n][:, :, 0].contiguous() for n in names}
    prefill(x), backward(x), kata.delta_decode_step(*step.values(), S.clone())  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, last = prefill(x)
        grads = backward(x)
        od = kata.delta_decode_step(*step.values(), S)
    for seed in (81, 82):
        y = delta_inputs(2, 2, 200, 64, torch.bfloat16, seed=seed)
        for n in x:
            x[n].copy_(y[n])
        for n in names:
            step[n].copy_(y[n][:, :, 0])
        S.copy_(y["S"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((o, last) + grads, prefill(y) + backward(y)))
        S2 = y["S"].clone()
        assert torch.equal(od, kata.delta_decode_step(*step.values(), S2)) and torch.equal(S, S2)


@pytest.mark.parametrize("change,message", [
    (dict(q=lambda x: x["q"].half()), "not float32 or bfloat16"),
    (dict(k=lambda x: x["k"].float()), "k:"),
    (dict(v=lambda x: x["v"][:, :, :50]), "v:"),
    (dict(g=lambda x: x["g"].double()), "g:"),
    (dict(g=lambda x: x["g"].bfloat16()), "g:"),
    (dict(beta=lambda x: x["beta"][:, :1]), "beta:"),
    (dict(beta=lambda x: None), "beta must not be None"),
    (dict(S=lambda x: x["S"].double()), "S_in:"),
    (dict(S=lambda x: x["S"].mT), "S_in:"),
    (dict(q=lambda x: x["q"].cpu()), "q:"),
    (dict(g=lambda x: x["g"].cpu()), "g:"),
])
def test_refusals(change, message):
    x = delta_inputs(2, 2, 100, 32, torch.bfloat16, seed=90)
    x.update({n: f(x) for n, f in change.items()})
    before = kata.launch_count()
    with pytest.raises(kata.KataError, match=message):
        prefill(x)
    with pytest.raises(kata.KataError, match=message):
        backward(x)
    assert kata.launch_count() == before


def test_refusals_of_sizes():
    for d in (8, 24, 48, 256):
        x = delta_inputs(1, 1, 4, d, torch.float32, seed=91)
        with pytest.raises(kata.KataError, match="KATA_ERR_UNSUPPORTED"):
            prefill(x)
        with pytest.raises(kata.KataError, match="KATA_ERR_UNSUPPORTED"):
            backward(x)
    x = delta_inputs(1, 1, 1, 32, torch.float32, seed=92)
    empty = {n: (t[:, :, :0].contiguous() if n not in ("S", "dS") else t) for n, t in x.items()}
    with pytest.raises(kata.KataError, match="KATA_ERR_INVALID_ARG"):
        prefill(empty)
    with pytest.raises(kata.KataError, match="KATA_ERR_WORKSPACE"):
        prefill(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kata.KataError, match="KATA_ERR_WORKSPACE"):
        backward(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kata.KataError, match="must not overwrite"):
        kata.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], o=x["v"])
    with pytest.raises(kata.KataError, match="S must not be None"):
        kata.delta_decode_step(*(x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g", "beta")), None)
