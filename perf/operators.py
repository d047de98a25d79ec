"""What the gated delta rule and the block's RMS norm have to compute, in plain torch operations, and
the calls of this package that compute the same: the cases on which the two are timed and compared.

The gated delta rule, per batch row and head (g = h // (H / G) is the head's group of q and k):

    S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T      state P x N
    o_t = scale S_t q_t

with q and k divided by their norm first where `l2norm` is set.  The RMS norm, per row:

    h = x + residual (as stored),  y = h / sqrt(mean(h^2) + eps) * weight

gated by silu(z) before ("pre") or after ("post") the norm, and stored as it is or as e4m3 values
with one float32 scale per `quant` elements.  Gradients are those of these formulas.
"""
import math

import torch

own = False   # set by whoever measures: False computes the plain forms

EPS = 1e-5        # of the RMS norm
L2_EPS = 1e-6     # under the root of q's and k's norms
CHUNK = 64        # of the plain form of the delta rule
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def _delta(name, op, b, L, H, G, P, N, dtype="bf16", init=True, l2norm=True, nseq=0):
    return dict(name=name, op=op, b=b, L=L, H=H, G=G, P=P, N=N, dtype=dtype, init=init,
                l2norm=l2norm, nseq=nseq)


def _norm(name, op, rows, dim, dtype="bf16", residual=False, gate="none", quant=0):
    return dict(name=name, op=op, rows=rows, dim=dim, dtype=dtype, residual=residual, gate=gate,
                quant=quant)


def listed():
    return [
        # a short prompt that continues from a kept state: few heads, a ragged last chunk
        _delta("delta_fwd_short", "delta_fwd", 1, 129, 8, 2, 64, 128),
        # training and prefill with wide heads, two value heads to a key head
        _delta("delta_fwd_p128", "delta_fwd", 2, 4096, 32, 16, 128, 128, init=False),
        # prefill of 12 packed prompts at the 2.7B layer's width (the packed workload's sizes)
        _delta("delta_fwd_packed", "delta_fwd", 1, 16384, 80, 1, 64, 128, nseq=12),
        # a training step's backward on a small odd case: keys that come normalised
        _delta("delta_bwd_odd", "delta_bwd", 1, 777, 6, 2, 64, 64, l2norm=False),
        # the backward at the 370M layer's sizes
        _delta("delta_bwd_370m", "delta_bwd", 2, 2048, 24, 1, 64, 128),
        # one token for one sequence: latency
        _delta("delta_step_b1", "delta_step", 1, 1, 24, 1, 64, 128),
        # one token for each of 128 sequences (the decode workload's sizes)
        _delta("delta_step_b128", "delta_step", 128, 1, 80, 1, 64, 128),
        # the pre-norm of the 2.7B layer (width 2560) over 16384 tokens, with the residual's sum
        _norm("norm_residual", "norm", 16384, 2560, residual=True),
        # the same for one token of each of 128 sequences, to 8 bits with a scale per row
        _norm("norm_step_e4m3", "norm", 128, 2560, residual=True, quant=2560),
        # the gated norm in front of the output projection (width 5120), to 8 bits by groups of 128
        _norm("norm_gated_e4m3", "norm", 8191, 5120, gate="pre", quant=128),
        # the pre-norm's backward, the residual stream's own gradient added in
        _norm("norm_bwd_residual", "norm_bwd", 16384, 2560, residual=True),
        # the backward of the norm over each head's output with the gate behind it
        _norm("norm_bwd_heads", "norm_bwd", 98304, 64, gate="post"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(("delta_fwd", "delta_fwd", "delta_bwd", "delta_step", "norm", "norm_bwd"))
    if op == "norm" or op == "norm_bwd":
        gate = rng.choice(("none", "pre", "post"))
        dim = rng.choice((64, 80, 128, 130, 1536, 1537, 2560, 5120, _log(rng, 16, 8192)))
        quant = 0
        if op == "norm" and rng.random() < 0.5:
            quant = 128 if dim % 128 == 0 and rng.random() < 0.5 else dim
        return _norm(op, op, _log(rng, 1, 4e7 / dim), dim, rng.choice(("bf16", "bf16", "f32")),
                     gate == "none" and rng.random() < 0.7, gate, quant)
    G = rng.choice((1, 1, 2, 4, 8))
    H = G * rng.choice((1, 2, 3, 4, 6, 10))
    P, N = rng.choice((64, 64, 128, 128, 48, 32)), rng.choice((128, 128, 64))
    l2norm, init = rng.random() < 0.7, rng.random() < 0.5
    if op == "delta_step":
        b = _log(rng, 1, 128 * 80 / H)
        return _delta(op, op, min(b, 512), 1, H, G, P, N, rng.choice(("bf16", "f32")), True, l2norm)
    dtype = "f32" if op == "delta_fwd" and rng.random() < 0.2 else "bf16"
    L = _log(rng, 1, 1500 if dtype == "f32" else 6000)
    nseq = 0
    if op == "delta_fwd" and L > 40 and rng.random() < 0.3:
        nseq = rng.randint(2, 12)
    most = 5e7 if op == "delta_fwd" else 1.2e7       # values of v
    b = 1 if nseq else max(1, min(rng.choice((1, 2, 3, 4)), int(most / (L * H * P))))
    return _delta(op, op, b, L, H, G, P, N, dtype, init, l2norm, nseq)


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _cuts(case, seed):
    """The first token of each packed sequence, and the end."""
    import random
    L, n = case["L"], case["nseq"]
    return [0] + sorted(random.Random(seed).sample(range(1, L), n - 1)) + [L]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    t = _dtype(case)

    def normal(*shape, to=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(to)

    if case["op"].startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        s = dict(case=case, x=normal(rows, dim, to=t), weight=1 + normal(dim, scale=0.2))
        if case["residual"]:
            s["residual"] = normal(rows, dim, to=t, scale=2.0)
        if case["gate"] != "none":
            s["z"] = normal(rows, dim, to=t)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, dim, to=t)
        return s
    b, L, H, G, P, N = (case[k] for k in "bLHGPN")
    # keys and queries as a convolution's SiLU leaves them: of one sign more often than not
    q, k = (torch.nn.functional.silu(normal(b, L, G, N)) for _ in range(2))
    if not case["l2norm"]:
        q, k = (v / v.norm(dim=-1, keepdim=True) for v in (q, k))
    dt = torch.nn.functional.softplus(normal(b, L, H) - 4).clamp(1e-3, 0.1)
    A = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(16))
    s = dict(case=case, q=q.to(t), k=k.to(t), v=normal(b, L, H, P, to=t), g=-dt * A,
             beta=torch.sigmoid(normal(b, L, H)), init=None, scale=N ** -0.5)
    if case["init"]:
        s["init"] = normal(case["nseq"] or b, H, P, N, scale=0.1)
    if case["nseq"]:
        s["cu_seqlens"] = torch.tensor(_cuts(case, seed), dtype=torch.int32, device="cuda")
    if case["op"] == "delta_step":
        s |= {n: s[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    if case["op"] == "delta_bwd":
        s["do"] = normal(b, L, H, P, to=t)
        s["dfinal"] = normal(b, H, P, N, scale=0.1)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"delta_fwd": _plain_fwd, "delta_bwd": _plain_bwd, "delta_step": _plain_step,
            "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[case["op"]](s, case)


def _run_own(s, case):
    from mamba_ssd_layer_scan_b200 import ssd
    if case["op"] == "norm":
        return ssd.rms_norm(s["x"], s["weight"], eps=EPS, residual=s.get("residual"),
                            z=s.get("z"), gate=case["gate"], quant_group=case["quant"])
    if case["op"] == "norm_bwd":
        # the forward's stored sum is the backward's input; `residual` is its gradient here
        return ssd.rms_norm_bwd(s["x"], s["weight"], s["dy"], eps=EPS, z=s.get("z"),
                                gate=case["gate"], dresidual=s.get("residual"))
    kw = dict(scale=s["scale"], qk_l2norm=case["l2norm"])
    args = [s[n] for n in ("q", "k", "v", "g", "beta")]
    if case["op"] == "delta_step":
        return ssd.delta_rule_update(s["init"], *args, **kw), s["init"]
    if case["op"] == "delta_bwd":
        return ssd.delta_rule_bwd(*args, s["do"], init_state=s["init"], dfinal=s["dfinal"], **kw)
    if case["nseq"]:
        return ssd.delta_rule_varlen_fwd(*args, s["cu_seqlens"], init_states=s["init"], **kw)
    return ssd.delta_rule_fwd(*args, init_state=s["init"], **kw)


# ---------------------------------------------------------------- plain forms: the delta rule
def _heads(t, H):
    """(..., G, N) to (..., H, N): each group's row for each of its heads."""
    return t.repeat_interleave(H // t.shape[-2], dim=-2)


def _unit(t, on):
    return t * torch.rsqrt((t * t).sum(-1, keepdim=True) + L2_EPS) if on else t


def _chunked(q, k, v, g, beta, S, scale):
    """q, k (b, L, H, N), v (b, L, H, P), g and beta (b, L, H), S (b, H, P, N), all float32:
    o (b, L, H, P) and the state after the last token, in chunks of CHUNK tokens."""
    b, L, H, P = v.shape
    n = -(-L // CHUNK)

    def cut(t):   # (b, L, H, ...) to (b, H, n, CHUNK, ...), zeros behind the end
        t = torch.nn.functional.pad(t, [0, 0] * (t.dim() - 2) + [0, n * CHUNK - L])
        return t.unflatten(1, (n, CHUNK)).movedim(3, 1)

    q, k, v, g, beta = (cut(t) for t in (q, k, v, g, beta))
    cs = g.cumsum(-1)
    at = torch.arange(CHUNK, device=v.device)
    upto = at[:, None] >= at[None, :]
    decay = torch.exp((cs[..., :, None] - cs[..., None, :]).masked_fill(~upto, -math.inf))
    # W, the part of v that the state does not predict: (I + A) W = V - exp(cs) K S^T, where A_ij
    # = exp(cs_i - cs_j) (k_i . k_j) beta_j below the diagonal; T = (I + A)^-1 row by row
    kk = k @ k.transpose(-1, -2)
    A = (kk * decay * beta[..., None, :]) * (at[:, None] > at[None, :])
    rows = [torch.eye(CHUNK, device=v.device).expand(A.shape[:-2] + (CHUNK, CHUNK))[..., 0, :]]
    for i in range(1, CHUNK):
        above = torch.stack(rows, -2)
        row = -(A[..., i:i + 1, :i] @ above).squeeze(-2)
        row = row + (at == i)
        rows.append(row)
    T = torch.stack(rows, -2)
    Tv = T @ v
    Tk = T @ (torch.exp(cs)[..., None] * k)
    att = (q @ k.transpose(-1, -2)) * decay * scale
    qe = q * (torch.exp(cs)[..., None] * scale)
    ke = k * torch.exp(cs[..., -1:] - cs)[..., None]
    last = torch.exp(cs[..., -1])[..., None, None]
    o = []
    for c in range(n):
        u = beta[:, :, c, :, None] * (Tv[:, :, c] - Tk[:, :, c] @ S.transpose(-1, -2))
        o.append(qe[:, :, c] @ S.transpose(-1, -2) + att[:, :, c] @ u)
        S = last[:, :, c] * S + u.transpose(-1, -2) @ ke[:, :, c]
    return torch.stack(o, 2).movedim(1, 3).flatten(1, 2)[:, :L], S


def _plain_fwd(s, case):
    H, t = case["H"], s["v"].dtype
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    q, k = (_heads(_unit(x, case["l2norm"]), H) for x in (q, k))
    S = s["init"]
    if S is None:
        S = v.new_zeros(case["nseq"] or case["b"], H, case["P"], case["N"])
    if not case["nseq"]:
        o, S = _chunked(q, k, v, g, beta, S, s["scale"])
        return o.to(t), S
    # packed sequences as the rows of a padded batch; what is padded neither decays nor writes
    cu = s["cu_seqlens"].long()
    most = int((cu[1:] - cu[:-1]).max())
    at = cu[:-1, None] + torch.arange(most, device=cu.device)
    there = at < cu[1:, None]
    at = at.clamp(max=case["L"] - 1)
    rows = [x[0][at] * there.view(there.shape + (1,) * (x.dim() - 2)) for x in (q, k, v, g, beta)]
    o, S = _chunked(*rows, S, s["scale"])
    return o[there][None].to(t), S


def _plain_bwd(s, case):
    H, t = case["H"], s["v"].dtype
    leaves = [s[n].float().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    init = s["init"] if s["init"] is not None else s["dfinal"] * 0
    leaves.append(init.detach().requires_grad_())
    with torch.enable_grad():
        q, k = (_heads(_unit(x, case["l2norm"]), H) for x in leaves[:2])
        o, S = _chunked(q, k, *leaves[2:], s["scale"])
        grads = torch.autograd.grad([o, S], leaves, [s["do"].float(), s["dfinal"]])
    dq, dk, dv, dg, dbeta, dinit = grads
    return dict(dq=dq.to(t), dk=dk.to(t), dv=dv.to(t), dg=dg, dbeta=dbeta, dinit=dinit)


def _plain_step(s, case):
    H, t = case["H"], s["v"].dtype
    q, k, v, g, beta = (s[n].float() for n in ("q", "k", "v", "g", "beta"))
    q, k = (_heads(_unit(x, case["l2norm"]), H) for x in (q, k))
    S = s["init"]
    S.mul_(torch.exp(g)[..., None, None])
    u = beta[..., None] * (v - (S * k[..., None, :]).sum(-1))
    S.add_(u[..., None] * k[..., None, :])
    return ((S * q[..., None, :]).sum(-1) * s["scale"]).to(t), S


# ---------------------------------------------------------------- plain forms: the norm
def _plain_norm(s, case):
    x, t = s["x"].float(), s["x"].dtype
    out = []
    if case["residual"]:
        stored = (x + s["residual"].float()).to(t)
        x = stored.float()
        out.append(stored)
    if case["gate"] == "pre":
        z = s["z"].float()
        x = x * (z * torch.sigmoid(z))
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    if case["gate"] == "post":
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    if not case["quant"]:
        return [y.to(t)] + out if out else y.to(t)
    y = y.unflatten(-1, (-1, case["quant"]))
    scales = (y.abs().amax(-1) / E4M3_MAX).clamp(min=1e-30)
    y8 = (y / scales[..., None]).to(torch.float8_e4m3fn).flatten(1)
    return [y8, scales] + out


def _plain_norm_bwd(s, case):
    x, w, dy, t = s["x"].float(), s["weight"], s["dy"].float(), s["x"].dtype
    if case["gate"] != "none":
        z = s["z"].float()
        sig = torch.sigmoid(z)
        silu, dsilu = z * sig, sig * (1 + z * (1 - sig))
    h = x * silu if case["gate"] == "pre" else x
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    dn = dy * silu if case["gate"] == "post" else dy
    dh = r * (dn * w - n * (n * dn * w).mean(-1, keepdim=True))
    out = dict(dweight=(dn * n).sum(0))
    if case["gate"] == "pre":
        out |= dict(dx=(dh * silu).to(t), dz=(dh * x * dsilu).to(t))
    elif case["gate"] == "post":
        out |= dict(dx=dh.to(t), dz=(dy * n * w * dsilu).to(t))
    elif case["residual"]:
        out["dx"] = (dh + s["residual"].float()).to(t)
    else:
        out["dx"] = dh.to(t)
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        n, gated = rows * dim, case["gate"] != "none"
        if case["op"] == "norm":
            if case["quant"]:
                written = n + 4 * rows * (dim // case["quant"])
            else:
                written = n * e
            read = n * e * (1 + case["residual"] + gated)
            return dict(bytes=read + written + n * e * case["residual"] + 4 * dim,
                        flops=n * (4 + 5 * gated))
        return dict(bytes=n * e * (3 + case["residual"] + 2 * gated) + 8 * dim,
                    flops=n * (9 + 9 * gated))
    b, L, H, G, P, N = (case[k] for k in "bLHGPN")
    tokens, state = b * L, (case["nseq"] or b) * H * P * N * 4
    read = tokens * (e * (2 * G * N + H * P) + 8 * H) + state * case["init"]
    if case["op"] == "delta_step":
        return dict(bytes=read + tokens * e * H * P + state, flops=tokens * H * P * N * 7)
    # in chunks of 64: K S^T, Q S^T, U^T K, and the products with the two triangles
    chunk = 2 * (3 * P * N + 64 * (P + N)) * H
    if case["op"] == "delta_fwd":
        return dict(bytes=read + tokens * e * H * P + state, flops=tokens * chunk)
    return dict(bytes=read + tokens * e * H * P + state * 2
                + tokens * (e * (2 * G * N + H * P) + 8 * H), flops=tokens * chunk * 3)


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s, case)
    H, P, N = case["H"], case["P"], case["N"]
    d = {n: s[n].double() for n in ("q", "k", "v", "g", "beta")}
    if case["op"] == "delta_step":
        d = {n: x[:, None] for n, x in d.items()}
    raw = {n: d[n] for n in "qk"}
    if case["l2norm"]:
        for n in "qk":
            d[n] = d[n] / torch.sqrt((d[n] ** 2).sum(-1, keepdim=True) + L2_EPS)
    group = torch.arange(H, device="cuda") // (H // case["G"])
    nb = case["nseq"] or case["b"]
    S = torch.zeros(nb, H, P, N, dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        S += s["init"].double()
    if case["op"] == "delta_bwd":
        return _exact_bwd(s, case, d, raw, group, S)
    o = torch.empty(case["b"], case["L"], H, P, dtype=torch.float64, device="cuda")
    ends = _cuts(case, seed) if case["nseq"] else None
    longest = max(y - x for x, y in zip(ends, ends[1:])) if ends else case["L"]
    if longest * nb * H * P * N > 2e11:
        return None   # minutes of token steps
    for t in range(longest):
        if ends:   # the sequences that still run, and their tokens
            live = [i for i in range(nb) if ends[i] + t < ends[i + 1]]
            row = (0, torch.tensor([ends[i] + t for i in live], device="cuda"))
            live = torch.tensor(live, device="cuda")
        else:
            row, live = (slice(None), t), slice(None)
        S[live], o[row] = _token(S[live], *(d[n][row] for n in ("q", "k", "v", "g", "beta")),
                                 group, s["scale"])
    return (o[:, 0] if case["op"] == "delta_step" else o), S


def _token(S, q, k, v, g, beta, group, scale):
    kt, qt = k[:, group], q[:, group]
    S = torch.exp(g)[..., None, None] * S
    u = beta[..., None] * (v - torch.einsum("bhpn,bhn->bhp", S, kt))
    S = S + torch.einsum("bhp,bhn->bhpn", u, kt)
    return S, scale * torch.einsum("bhpn,bhn->bhp", S, qt)


def _exact_bwd(s, case, d, raw, group, S):
    """The adjoint recurrence token by token, the states kept in spans."""
    b, L, H, G, P, N = (case[k] for k in "bLHGPN")
    if L * b * H * P * N > 4e10:
        return None
    span, starts = 128, []
    for t in range(L):
        if t % span == 0:
            starts.append(S)
        S, _ = _token(S, *(d[n][:, t] for n in ("q", "k", "v", "g", "beta")), group, s["scale"])
    do, D = s["do"].double() * s["scale"], s["dfinal"].double().clone()
    out = {n: torch.zeros_like(d[n]) for n in ("q", "k", "v", "g", "beta")}
    for t in range(L - 1, -1, -1):
        if t % span == span - 1 or t == L - 1:
            before = [starts[t // span]]
            for i in range(t // span * span, t):
                before.append(_token(before[-1], *(d[n][:, i] for n in ("q", "k", "v", "g", "beta")),
                                     group, s["scale"])[0])
        q, k = d["q"][:, t][:, group], d["k"][:, t][:, group]
        v, beta = d["v"][:, t], d["beta"][:, t]
        kept = torch.exp(d["g"][:, t])[..., None, None] * before.pop()
        w = v - torch.einsum("bhpn,bhn->bhp", kept, k)
        new = kept + torch.einsum("bhp,bhn->bhpn", beta[..., None] * w, k)
        dq = torch.einsum("bhpn,bhp->bhn", new, do[:, t])
        D = D + torch.einsum("bhp,bhn->bhpn", do[:, t], q)
        du = torch.einsum("bhpn,bhn->bhp", D, k)
        dw = beta[..., None] * du
        dk = torch.einsum("bhpn,bhp->bhn", D, beta[..., None] * w) \
            - torch.einsum("bhpn,bhp->bhn", kept, dw)
        out["v"][:, t], out["beta"][:, t] = dw, (du * w).sum(-1)
        D = D - torch.einsum("bhp,bhn->bhpn", dw, k)
        out["g"][:, t] = (D * kept).sum((-1, -2))
        D = D * torch.exp(d["g"][:, t])[..., None, None]
        out["q"][:, t] = dq.unflatten(1, (G, -1)).sum(2)
        out["k"][:, t] = dk.unflatten(1, (G, -1)).sum(2)
    if case["l2norm"]:
        for n in "qk":
            size = torch.sqrt((raw[n] ** 2).sum(-1, keepdim=True) + L2_EPS)
            out[n] = (out[n] - d[n] * (d[n] * out[n]).sum(-1, keepdim=True)) / size
    return dict(dq=out["q"], dk=out["k"], dv=out["v"], dg=out["g"], dbeta=out["beta"], dinit=D)


def _exact_norm(s, case):
    h, out = s["x"].double(), []
    if case["residual"]:
        # the stream's sum is kept in its own type; the norm is that of what is kept
        out = [h + s["residual"].double()]
        h = out[0].to(torch.float32).to(s["x"].dtype).double()
    z = s["z"].double() if case["gate"] != "none" else None
    if case["gate"] == "pre":
        h = h * z / (1 + torch.exp(-z))
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
    if case["gate"] == "post":
        y = y * z / (1 + torch.exp(-z))
    if not case["quant"]:
        return [y] + out if out else y
    groups = y.view(case["rows"], -1, case["quant"])
    scales = torch.clamp(groups.abs().max(-1).values / E4M3_MAX, min=1e-30)
    return [(groups / scales[..., None]).view_as(y), scales] + out


def _exact_norm_bwd(s, case):
    x, w, dy = s["x"].double(), s["weight"].double(), s["dy"].double()
    h, dn = x, dy
    if case["gate"] != "none":
        z = s["z"].double()
        e = torch.exp(-z)
        silu = z / (1 + e)
        slope = 1 / (1 + e) + z * e / (1 + e) ** 2
        h, dn = (x * silu, dy) if case["gate"] == "pre" else (x, dy * silu)
    size = torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    # y = w h / size and size^2 = mean(h^2) + eps: dh = w dy / size - h (dy . y) / (dim size^2)
    inner = (dn * w * h).sum(-1, keepdim=True) / case["dim"]
    dh = dn * w / size - h * inner / size ** 3
    out = dict(dweight=(dn * h / size).sum(0))
    if case["gate"] == "pre":
        return out | dict(dx=dh * silu, dz=dh * x * slope)
    if case["gate"] == "post":
        return out | dict(dx=dh, dz=dy * w * h / size * slope)
    return out | dict(dx=dh + s["residual"].double() if case["residual"] else dh)
