"""Measured cases of the gated delta rule (chunked prefill, one-token step, gradients) and of
the gradients of the causal kernelized prefill.

The gated delta rule, per (batch, head), with the fp32 state S [d, d] (key rows, value
columns), the log decay g_t <= 0 and the writing strength beta_t:

    e_t = v_t - exp(g_t) S_{t-1}^T k_t
    S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T
    o_t = scale S_t^T q_t

The kernelized prefill, o_i = sum_{j<=i} (q_i.k_j)^2 v_j / (sum_{j<=i} (q_i.k_j)^2 + eps), is
differentiated with respect to q, k and v; its weights are recomputed, not kept.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64
EPS = 1e-6


def listed():
    return [
        # a short fp32 prompt of one head, from an empty state: the smallest call
        dict(name="delta_prefill_f32_T256_d16", op="delta_prefill", dtype="f32", B=1, H=1, T=256, d=16, state=False),
        # an ordinary prefill batch
        dict(name="delta_prefill_bf16_T2048_d32", op="delta_prefill", dtype="bf16", B=4, H=8, T=2048, d=32, state=False),
        # a long document continued from a kept state: the largest
        dict(name="delta_prefill_bf16_T16384_d64", op="delta_prefill", dtype="bf16", B=2, H=16, T=16384, d=64, state=True),
        # wide heads, a ragged number of heads and tokens, continued from a kept state
        dict(name="delta_prefill_bf16_T1531_d128", op="delta_prefill", dtype="bf16", B=3, H=5, T=1531, d=128, state=True),
        # one user's next token: latency
        dict(name="delta_decode_bf16_B1_d64", op="delta_decode", dtype="bf16", B=1, H=16, d=64),
        # a serving batch's next tokens
        dict(name="delta_decode_bf16_B64_d64", op="delta_decode", dtype="bf16", B=64, H=16, d=64),
        # a ragged batch with wide heads in fp32
        dict(name="delta_decode_f32_B37_d128", op="delta_decode", dtype="f32", B=37, H=12, d=128),
        # a training step's gradients over a batch of sequences
        dict(name="delta_backward_bf16_T4096_d64", op="delta_backward", dtype="bf16", B=2, H=16, T=4096, d=64, state=False),
        # a ragged fp32 piece of a longer sequence: gradients through the states at both its ends
        dict(name="delta_backward_f32_T777_d32", op="delta_backward", dtype="f32", B=1, H=6, T=777, d=32, state=True),
        # gradients of the headline prefill
        dict(name="prefill_backward_bf16_T2048_d32", op="prefill_backward", dtype="bf16", B=4, H=8, T=2048, d=32),
        # gradients of a long sequence
        dict(name="prefill_backward_bf16_T8192_d64", op="prefill_backward", dtype="bf16", B=2, H=8, T=8192, d=64),
        # a ragged fp32 sequence
        dict(name="prefill_backward_f32_T643_d64", op="prefill_backward", dtype="f32", B=1, H=4, T=643, d=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_prefill", "delta_prefill", "delta_decode", "delta_backward", "prefill_backward", "prefill_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, dtype=dtype, B=rng.randint(1, 4), H=rng.randint(1, 16))
    if op == "delta_decode":
        c.update(B=_log_int(rng, 1, 64), d=rng.choice([16, 32, 64, 128]))
        if c["d"] == 128:
            c.update(B=min(c["B"], 32))
        return c
    heads = c["B"] * c["H"]
    if op == "delta_prefill":
        d = rng.choice([16, 32, 64, 64, 128])
        c.update(d=d, T=_log_int(rng, 1, min(16384, (1 << 19) * 64 * 64 // (heads * d * d))), state=rng.random() < 0.5)
    elif op == "delta_backward":
        d = rng.choice([16, 32, 64, 64, 128])
        c.update(d=d, T=_log_int(rng, 1, min(4096, (1 << 17) * 64 * 64 // (heads * d * d))), state=rng.random() < 0.5)
    else:
        d = rng.choice([16, 32, 64])
        longest = 8192 if dtype == "bf16" else 4096
        c.update(d=d, T=_log_int(rng, 1, min(longest, int(math.sqrt(16 * 8192 * 8192 / heads)))))
    return c


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def unit(*shape):
        x = normal(*shape)
        return x / x.norm(dim=-1, keepdim=True)

    t = DTYPES[c["dtype"]]
    B, H, d = c["B"], c["H"], c["d"]
    s = {"case": c}
    if c["op"] == "prefill_backward":
        shape = (B, H, c["T"], d)
        for n in ("q", "k"):
            s[n] = (normal(*shape) * d**-0.5).to(t)
        for n in ("v", "do"):
            s[n] = normal(*shape).to(t)
        return s
    rows = (B, H) if c["op"] == "delta_decode" else (B, H, c["T"])
    # keys and queries are unit rows; each head has its own rate of decay, and each token its own share of it
    s["q"], s["k"], s["v"] = unit(*rows, d).to(t), unit(*rows, d).to(t), normal(*rows, d).to(t)
    rate = torch.exp(torch.rand(H, generator=gen, device="cuda") * 5.0 - 6.0).reshape((1, H) + (1,) * (len(rows) - 2))
    s["g"] = -rate * torch.nn.functional.softplus(normal(*rows))
    s["beta"] = torch.sigmoid(normal(*rows))
    s["S"] = 0.5 * normal(B, H, d, d) if c.get("state") or c["op"] == "delta_decode" else None
    if c["op"] == "delta_backward":
        s["do"] = normal(*rows, d).to(t)
        s["dS"] = 0.5 * normal(B, H, d, d) if c["state"] else None
    return s


def run(state):
    return {"delta_prefill": _delta_prefill, "delta_decode": _delta_decode, "delta_backward": _delta_backward,
            "prefill_backward": _prefill_backward}[state["case"]["op"]](state)


def _delta_prefill(s):
    if own:
        import kernelized_linear_attention_chunked_b200 as kata
        return kata.delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], S_in=s["S"])
    p = _chunked(s)
    o = torch.empty_like(p["q"])
    S = p["S"]
    for c in range(p["n"]):
        R = p["v"][:, c] - p["a"][:, c] * (p["k"][:, c] @ S)
        U = p["beta"][:, c] * (p["X"][:, c] @ R)
        o[:, c] = p["scale"] * (p["a"][:, c] * (p["q"][:, c] @ S) + p["M"][:, c] @ U)
        S = p["aC"][:, c] * S + p["k"][:, c].mT @ (p["c"][:, c] * U)
    return _whole(o, s["q"]), S.reshape(s["q"].shape[:2] + S.shape[1:])


def _chunked(s):
    """The sequence in chunks, in fp32, padded with tokens that change nothing, and what each chunk needs of itself alone."""
    B, H, T, d = s["q"].shape
    n = -(-T // CHUNK)

    def chunks(x):
        x = x.float().reshape(B * H, T, -1)
        return torch.nn.functional.pad(x, (0, 0, 0, n * CHUNK - T)).reshape(B * H, n, CHUNK, -1)

    q, k, v, beta = (chunks(s[x]) for x in ("q", "k", "v", "beta"))
    G = chunks(s["g"]).double().cumsum(2)  # log decay since the chunk's start
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp(torch.where(low, G - G.mT, -torch.inf)).float()
    N = (k @ k.mT * D).tril(-1)
    A = N * beta.mT
    X = torch.eye(CHUNK, device=q.device).repeat(B * H, n, 1, 1)  # (1 + A)^-1 by forward substitution
    for i in range(1, CHUNK):
        X[:, :, i, :i] = -(A[:, :, i : i + 1, :i] @ X[:, :, :i, :i]).squeeze(2)
    S = torch.zeros(B * H, d, d, device=q.device) if s["S"] is None else s["S"].reshape(B * H, d, d)
    return dict(q=q, k=k, v=v, beta=beta, n=n, D=D, N=N, X=X, M=q @ k.mT * D, S=S, scale=d**-0.5, a=torch.exp(G).float(),
                c=torch.exp(G[:, :, -1:] - G).float(), aC=torch.exp(G[:, :, -1:]).float())


def _whole(x, like):
    return x.reshape(like.shape[0] * like.shape[1], x.shape[1] * CHUNK, -1)[:, : like.shape[2]].reshape(like.shape).to(like.dtype)


def _delta_decode(s):
    if own:
        import kernelized_linear_attention_chunked_b200 as kata
        return kata.delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"]), s["S"]
    q, k, v = (s[n].float().unsqueeze(-2) for n in ("q", "k", "v"))
    S = torch.exp(s["g"])[..., None, None] * s["S"]
    S = S + k.mT @ (s["beta"][..., None, None] * (v - k @ S))
    s["S"].copy_(S)
    return (q.shape[-1] ** -0.5 * (q @ S)).squeeze(-2).to(s["q"].dtype), s["S"]


def _delta_backward(s):
    if own:
        import kernelized_linear_attention_chunked_b200 as kata
        return kata.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], S_in=s["S"], dS=s["dS"], state_grad=s["S"] is not None)
    p = _chunked(s)
    B, H, T, d = s["q"].shape
    n, beta, scale = p["n"], p["beta"], p["scale"]
    do = torch.nn.functional.pad(s["do"].float().reshape(B * H, T, d), (0, 0, 0, n * CHUNK - T)).reshape(B * H, n, CHUNK, d)
    S0, E, dSC, Z = (torch.empty(B * H, n, x, d, device=do.device) for x in (d, CHUNK, d, CHUNK))
    S = p["S"]
    for c in range(n):  # the states, and each token's error, forwards
        S0[:, c] = S
        E[:, c] = p["X"][:, c] @ (p["v"][:, c] - p["a"][:, c] * (p["k"][:, c] @ S))
        S = p["aC"][:, c] * S + p["k"][:, c].mT @ (p["c"][:, c] * beta[:, c] * E[:, c])
    dS = torch.zeros_like(S) if s["dS"] is None else s["dS"].reshape(B * H, d, d)
    for c in reversed(range(n)):  # their gradients, backwards
        dSC[:, c] = dS
        dU = scale * p["M"][:, c].mT @ do[:, c] + p["c"][:, c] * (p["k"][:, c] @ dS)
        Z[:, c] = p["X"][:, c].mT @ (beta[:, c] * dU)
        dS = p["aC"][:, c] * dS + p["q"][:, c].mT @ (scale * p["a"][:, c] * do[:, c]) - p["k"][:, c].mT @ (p["a"][:, c] * Z[:, c])
    U = beta * E
    F = scale * p["M"].mT @ do + p["c"] * (p["k"] @ dSC) - p["N"].mT @ Z
    PM = scale * (do @ U.mT) * p["D"]
    PN = (-(Z @ U.mT) * p["D"]).tril(-1)
    dq = PM @ p["k"] + scale * p["a"] * (do @ S0.mT)
    row = PN @ p["k"] - p["a"] * (Z @ S0.mT)
    col = PM.mT @ p["q"] + PN.mT @ p["k"] + p["c"] * (U @ dSC.mT)
    dG = (p["q"] * dq).sum(-1) + (p["k"] * (row - col)).sum(-1)
    end = (p["c"] * U * (p["k"] @ dSC)).sum((-1, -2)) + p["aC"][:, :, 0, 0] * (S0 * dSC).sum((-1, -2))
    dg = end[..., None] + dG.double().flip(-1).cumsum(-1).flip(-1).float()
    out = [_whole(dq, s["q"]), _whole(row + col, s["q"]), _whole(Z, s["q"])]
    out += [x.reshape(B, H, -1)[:, :, :T].contiguous() for x in (dg, (E * F).sum(-1))]
    return (*out, dS.reshape(B, H, d, d) if s["S"] is not None else None)


def _prefill_backward(s):
    if own:
        import kernelized_linear_attention_chunked_b200 as kata
        return kata.prefill_backward(s["q"], s["k"], s["v"], s["do"], eps=EPS)
    q, k, v, do = (s[n].float() for n in ("q", "k", "v", "do"))
    # scores next to zero, and rows of few keys, which leave next to nothing of dw - delta: 64 bits
    x = (q.double() @ k.double().mT).tril_()
    dw = do @ v.mT
    a = x.square()
    den = a.sum(-1, keepdim=True).add_(EPS)
    dv = a.div(den).float().mT @ do
    dw = dw - a.mul_(dw).sum(-1, keepdim=True).div_(den)
    dw = dw.mul_(x).mul_(2 / den).float()
    return tuple(y.to(s["q"].dtype) for y in (dw @ k, dw.mT @ q, dv))


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    rows, d, T = c["B"] * c["H"], c["d"], c.get("T", 1)
    tokens, states = rows * T, 4 * rows * d * d
    if c["op"] == "delta_prefill":  # q, k, v, o, g and beta; the last state, and the first where there is one
        return {"bytes": tokens * (4 * d * e + 8) + states * (2 if c["state"] else 1), "flops": tokens * 6 * d * d}
    if c["op"] == "delta_decode":
        return {"bytes": tokens * (4 * d * e + 8) + 2 * states, "flops": tokens * 6 * d * d}
    if c["op"] == "delta_backward":  # q, k, v, do and their gradients; the states and gradients at both ends
        return {"bytes": tokens * (7 * d * e + 16) + states * (3 if c["state"] else 0), "flops": tokens * 18 * d * d}
    return {"bytes": tokens * 7 * d * e, "flops": rows * (T * (T + 1) // 2) * 10 * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill_backward":
        return _exact_prefill_backward(s)
    back = case["op"] == "delta_backward"
    lead = s["q"].shape[:2]
    d, scale = case["d"], 1.0 / math.sqrt(case["d"])
    T = case.get("T", 1)

    def tokens(name):  # [T, heads, ...] in 64 bits
        return s[name].double().reshape(lead[0] * lead[1], T, -1).transpose(0, 1).contiguous()

    q, k, v, g, beta = (tokens(n) for n in ("q", "k", "v", "g", "beta"))
    S = torch.zeros(q.shape[1], d, d, dtype=torch.float64, device="cuda") if s["S"] is None else s["S"].double().reshape(-1, d, d)
    kept, o = [], torch.empty_like(q)
    if back and T * S.numel() * 8 > 48e9:
        return None
    for t in range(T):  # the definition, token by token
        if back:
            kept.append(S)
        S = S * torch.exp(g[t])[:, :, None]
        e = v[t] - torch.einsum("hab,ha->hb", S, k[t])
        S = S + torch.einsum("ha,hb->hab", k[t], beta[t] * e)
        o[t] = scale * torch.einsum("hab,ha->hb", S, q[t])

    def back_to(x):
        return x.transpose(0, 1).reshape(lead + (T, -1))

    if case["op"] == "delta_decode":
        return back_to(o).squeeze(2), S.reshape(lead + (d, d))
    if not back:
        return back_to(o), S.reshape(lead + (d, d))
    do = tokens("do")
    dS = torch.zeros_like(S) if s["dS"] is None else s["dS"].double().reshape(-1, d, d)
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    for t in reversed(range(T)):  # the chain rule through one token
        decay = torch.exp(g[t])[:, :, None]
        D = kept[t] * decay
        e = v[t] - torch.einsum("hab,ha->hb", D, k[t])
        u = beta[t] * e
        dq[t] = scale * torch.einsum("hab,hb->ha", D + torch.einsum("ha,hb->hab", k[t], u), do[t])
        dS = dS + scale * torch.einsum("ha,hb->hab", q[t], do[t])
        du = torch.einsum("hab,ha->hb", dS, k[t])
        db[t] = (du * e).sum(-1, keepdim=True)
        de = beta[t] * du
        dv[t] = de
        dk[t] = torch.einsum("hab,hb->ha", dS, u) - torch.einsum("hab,hb->ha", D, de)
        dD = dS - torch.einsum("ha,hb->hab", k[t], de)
        dg[t] = (dD * D).sum((-1, -2)).unsqueeze(-1)
        dS = dD * decay
    return (*(back_to(x) for x in (dq, dk, dv)), back_to(dg).squeeze(-1), back_to(db).squeeze(-1),
            dS.reshape(lead + (d, d)) if s["S"] is not None else None)


def _exact_prefill_backward(s):
    B, H, T, d = s["q"].shape
    grads = torch.empty(3, B * H, T, d, dtype=torch.float64, device="cuda")
    rows = [s[n].reshape(B * H, T, d) for n in ("q", "k", "v", "do")]
    for h in range(B * H):
        q, k, v, do = (x[h].double() for x in rows)
        for i in range(0, T, 1024):  # queries in blocks, against the keys up to theirs
            j = min(i + 1024, T)
            Q, K, V, dO = q[i:j], k[:j], v[:j], do[i:j]
            seen = torch.arange(j, device="cuda")[None, :] <= torch.arange(i, j, device="cuda")[:, None]
            x = torch.where(seen, Q @ K.T, 0.0)
            den = (x**2).sum(1, keepdim=True) + EPS
            o = (x**2 @ V) / den
            dx = 2 * x * (dO @ V.T - (dO * o).sum(1, keepdim=True)) / den
            grads[0, h, i:j] = dx @ K
            if i == 0:
                grads[1:, h] = 0
            grads[1, h, :j] += dx.T @ Q
            grads[2, h, :j] += (x**2 / den).T @ dO
    return tuple(x.reshape(B, H, T, d) for x in grads)
