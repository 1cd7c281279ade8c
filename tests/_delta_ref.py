"""The gated delta rule and the kernelized prefill's gradients from their
definitions, in 64 bits, token by token (test infrastructure)."""
import torch


def delta_forward(q, k, v, g, beta, scale, S=None):
    """q, k, v [B, H, T, d], g, beta [B, H, T] -> o, last state (float64)."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    B, H, T, d = q.shape
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if S is None else S.double()
    out = []
    for t in range(T):
        S = torch.exp(g[:, :, t, None, None]) * S
        e = v[:, :, t] - (S * k[:, :, t, :, None]).sum(-2)
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * e)[:, :, None, :]
        out.append(scale * (S * q[:, :, t, :, None]).sum(-2))
    return torch.stack(out, 2), S


def delta_grads(q, k, v, g, beta, scale, do, S=None, dS=None):
    """(dq, dk, dv, dg, dbeta, dS_in) in float64, by differentiating delta_forward."""
    S = torch.zeros(*q.shape[:2], q.shape[3], q.shape[3], device=q.device) if S is None else S
    xs = [x.detach().double().requires_grad_(True) for x in (q, k, v, g, beta, S)]
    with torch.enable_grad():
        o, last = delta_forward(*xs[:5], scale, xs[5])
        loss = (o * do.double()).sum()
        if dS is not None:
            loss = loss + (last * dS.double()).sum()
    return torch.autograd.grad(loss, xs)


def prefill_forward(q, k, v, eps):
    q, k, v = (x.double() for x in (q, k, v))
    a = torch.tril(q @ k.mT) ** 2
    return (a @ v) / (a.sum(-1, keepdim=True) + eps)


def prefill_grads(q, k, v, do, eps):
    """(dq, dk, dv) in float64, by differentiating prefill_forward."""
    xs = [x.detach().double().requires_grad_(True) for x in (q, k, v)]
    with torch.enable_grad():
        loss = (prefill_forward(*xs, eps) * do.double()).sum()
    return torch.autograd.grad(loss, xs)


def rel(got, want) -> float:
    got, want = got.detach().double(), want.detach().double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all())
    return float((got - want).norm() / want.norm().clamp_min(1e-300))


def delta_inputs(B, H, T, d, dtype, seed, state=True, keys=None, device="cuda"):
    """Unit queries and keys (the keys drawn from a pool of `keys` vectors if
    given), values N(0, 1), decays and strengths over their useful range."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q = unit(n(B, H, T, d))
    if keys is None:
        k = unit(n(B, H, T, d))
    else:
        k = unit(n(keys, d))[torch.randint(keys, (B, H, T), generator=gen)]
    x = dict(q=q.to(dtype), k=k.to(dtype), v=n(B, H, T, d).to(dtype),
             g=-torch.rand(B, H, T, generator=gen) * 0.3, beta=torch.rand(B, H, T, generator=gen),
             do=n(B, H, T, d).to(dtype))
    x["S"] = 0.5 * n(B, H, d, d) if state else None
    x["dS"] = 0.5 * n(B, H, d, d) if state else None
    return {a: (b.to(device) if b is not None else None) for a, b in x.items()}
