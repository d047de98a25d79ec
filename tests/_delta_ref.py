"""The gated delta rule and the RMS norm in float64 on the CPU, from their definitions, and the
seeded inputs of their tests."""
from __future__ import annotations

import torch

L2_EPS = 1e-6


def draw(b, L, H, G, P, N, dtype=torch.float32, seed=0, unit=True, decay="mixed", init=True,
         nseq=None):
    """CPU inputs in their storage types.  unit: keys and queries of norm 1 (before rounding)."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    q, k = normal(b, L, G, N), normal(b, L, G, N) + 0.2   # keys that point the same way a little
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    g = None
    if decay == "mixed":     # heads from almost no decay to a few tokens of memory
        rate = 10.0 ** torch.linspace(-4, 0.3, H)
        g = -rate * torch.rand((b, L, H), generator=gen)
    elif decay == "strong":  # some tokens wipe the state out
        g = -torch.rand((b, L, H), generator=gen) * 0.1
        g[torch.rand((b, L, H), generator=gen) < 0.2] = -200.0
    return dict(q=q.to(dtype), k=k.to(dtype), v=normal(b, L, H, P).to(dtype), g=g,
                beta=torch.sigmoid(normal(b, L, H)),
                init=0.3 * normal(nseq or b, H, P, N) if init else None)


def heads(t, H):
    return t.repeat_interleave(H // t.shape[-2], dim=-2)


def unit(t, on):
    return t / torch.sqrt((t * t).sum(-1, keepdim=True) + L2_EPS) if on else t


def delta_rule(q, k, v, g, beta, init, scale, l2norm):
    """float64 token recurrence; differentiable.  Returns o (b, L, H, P) and the final state."""
    q, k, v, beta = (x.double() for x in (q, k, v, beta))
    b, L, H, P = v.shape
    q, k = (heads(unit(x, l2norm), H) for x in (q, k))
    S = torch.zeros(b, H, P, q.shape[-1], dtype=torch.float64) if init is None else init.double()
    a = torch.exp(g.double()) if g is not None else torch.ones(b, L, H, dtype=torch.float64)
    o = []
    for t in range(L):
        S = a[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        o.append(scale * (S * q[:, t, :, None, :]).sum(-1))
    return (torch.stack(o, 1) if o else v[:, :0]), S


def silu(z):
    return z * torch.sigmoid(z)


def rms_norm(x, weight, eps, residual=None, z=None, gate="none"):
    """float64: (y, h); h is the stored sum where there is a residual, else x."""
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(x.dtype)
    n = h.double()
    if gate == "pre":
        n = n * silu(z.double())
    y = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + eps) * weight.double()
    if gate == "post":
        y = y * silu(z.double())
    return y, h


def rel(got, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    got, ref = got.detach().double().cpu(), ref.detach().double()
    return float((got - ref).norm() / ref.norm().clamp_min(1e-300))
