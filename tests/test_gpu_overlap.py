"""Calls that follow each other with no other kernel between them (GPU).

The delta rule's kernels and the gradients' are launched to start while the kernel
before them still runs, and wait for it themselves. Each test here runs the same calls
once with a pause after each and once without, and wants the same bits: a call that
reads or overwrites what the one before it is still writing or reading gives others.
"""
import pytest
import torch

import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import delta_inputs

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
NAMES = ("q", "k", "v", "g", "beta")


def token(x, t):
    return {n: x[n][:, :, t].contiguous() for n in NAMES}


def same(run, repeats=3):
    want = run(torch.cuda.synchronize)
    kata.sync_status()
    for _ in range(repeats):
        got = run(lambda: None)
        kata.sync_status()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,d", [(64, 16, 128), (40, 7, 64), (1, 1, 16)])
def test_steps_in_a_row(dtype, B, H, d):
    # many steps on one state, several waves of blocks each, and each one's q and v are
    # what the two before it have just written
    x = delta_inputs(B, H, 10, d, dtype, seed=d)
    tokens = [token(x, t) for t in range(10)]
    S = torch.empty_like(x["S"])

    def run(pause):
        S.copy_(x["S"])
        outs = [torch.empty_like(tokens[0]["q"]) for _ in tokens]
        pause()
        for i, t in enumerate(tokens):
            q = outs[i - 1] if i > 0 else t["q"]
            v = outs[i - 2] if i > 1 else t["v"]
            kata.delta_decode_step(q, t["k"], v, t["g"], t["beta"], S, o=outs[i])
            pause()
        return [S.clone(), *outs]

    same(run)


@pytest.mark.parametrize("dtype", DTYPES)
def test_step_then_everything(dtype):
    # what reads a step's output or state, or overwrites its inputs, right behind it
    B, H, T, d = 16, 8, 130, 64
    x = delta_inputs(B, H, T, d, dtype, seed=3)
    tokens = [token(x, t) for t in range(6)]
    seq = [x[n] for n in NAMES]
    S = torch.empty_like(x["S"])

    def run(pause):
        S.copy_(x["S"])
        outs = [torch.empty_like(tokens[0]["q"]) for _ in tokens]
        o = torch.empty_like(x["q"])
        pause()

        def step(i):
            t = tokens[i]
            kata.delta_decode_step(*t.values(), S, o=outs[i])
            pause()

        one = lambda t: t.unsqueeze(2)  # a sequence of one token
        step(0)
        kata.delta_prefill(*seq, S_in=S, S_out=S, o=o)
        pause()
        step(1)
        g1 = kata.delta_backward(one(outs[1]), *(one(tokens[1][n]) for n in NAMES[1:]), one(outs[0]),
                                 S_in=S, dS=S, state_grad=True)
        pause()
        step(2)
        g2 = kata.prefill_backward(one(outs[2]), one(tokens[2]["k"]), one(outs[1]), one(outs[0]))
        pause()
        step(3)
        g3 = kata.delta_backward(*seq, o, S_in=S)
        pause()
        step(4)
        g4 = kata.prefill_backward(x["q"], x["k"], x["v"], o)
        pause()
        step(5)
        return [S.clone(), o, *outs, *g1, *g2, *g3[:5], *g4]

    same(run)


@pytest.mark.parametrize("form", ["chunked", "auto"])
@pytest.mark.parametrize("T,d", [(128, 32), (256, 32), (128, 64), (256, 64), (512, 64), (1024, 64)])
def test_behind_the_prefill(T, d, form):
    # the chunked prefill reads its snapshots behind a wait of its own, and with one
    # interval there are none: its inputs and its state are another's right after it
    B, H = 8, 16
    x = delta_inputs(B, H, T, d, torch.bfloat16, seed=T + d)
    fresh = {n: torch.empty_like(x[n]) for n in ("q", "k", "v")}
    seq, last = [x[n] for n in NAMES], token(x, 0)
    D = d * (d + 1) // 2
    Hs = torch.empty(B, H, D, d, device="cuda")
    ss = torch.empty(B, H, D, device="cuda")
    # its last state's memory as the state of the rule (D d >= d d)
    S = Hs.view(-1)[: B * H * d * d].view(B, H, d, d)

    def run(pause):
        out = []

        def attend():
            for n, t in fresh.items():
                t.copy_(x[n])
            pause()
            o = kata.prefill(*fresh.values(), chunk=64, H_out=Hs, s_out=ss, form=form)[0]
            pause()
            return o

        o = attend()
        o2, S2 = kata.delta_prefill(*seq, o=fresh["k"])  # over the keys it has just read
        pause()
        out += [o, o2.clone(), S2, Hs.clone(), ss.clone()]
        o = attend()
        kata.delta_prefill(*seq, o=fresh["v"], S_out=S)  # over the values and the state
        pause()
        out += [o, fresh["v"].clone(), S.clone()]
        o = attend()
        kata.delta_decode_step(*last.values(), S, o=fresh["k"].view(-1)[: B * H * d].view(B, H, d))
        pause()
        out += [o, S.clone(), fresh["k"].clone()]
        o = attend()
        out += kata.prefill_backward(*fresh.values(), x["do"])
        pause()
        out += [o, Hs.clone(), ss.clone()]
        o = attend()
        out += kata.delta_backward(*fresh.values(), x["g"], x["beta"], x["do"], S_in=S)[:5]
        pause()
        out += [o, ss.clone()]
        return out

    same(run)


@pytest.mark.parametrize("form", ["chunked", "quadratic"])
def test_captured_behind_the_prefill(form):
    # the same in a graph, whose edges are taken from the stream's: chunked (a kernel that
    # starts early before it) and quadratic with the state (two branches that join)
    x = delta_inputs(2, 4, 256, 64, torch.bfloat16, seed=9)
    seq = [x[n] for n in NAMES]
    last = token(x, 1)
    S0 = x["S"].clone()

    def calls():
        o, Hs, ss = kata.prefill(*seq[:3], chunk=64, form=form)
        o2, S = kata.delta_prefill(*seq, S_in=x["S"])
        o3 = kata.delta_decode_step(*last.values(), S0)
        o4, Hs2, _ = kata.prefill(*seq[:3], chunk=64, form=form)
        return [o, Hs, ss, o2, S, o3, S0, o4, Hs2, *kata.prefill_backward(*seq[:3], o2)]

    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        S0.copy_(x["S"])
        graph.replay()
        torch.cuda.synchronize()
        kata.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
