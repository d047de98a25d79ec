"""A mixer block of the operators together, as a model runs them: the pre-norm with the residual's sum,
the gated delta rule with its values from the normalised rows, the gated norm over each head's output,
the 8-bit output for the next product; prefill, decode and the backward pass.

Tolerances.  Forward stages are compared one by one on the values that the stage before really left, with
the tolerances of the operators' own tests.  The whole backward pass is compared with float64 autograd of
the block (2-norm): the forward values that it takes are off by 2^-8 (the norm's output) and 4 * 2^-8 (the
rule's), each of its three steps rounds its result, 2^-8, and takes operands off by the sum so far, and
the norms' gradients are differences of terms up to twice their size: 2 * 12 * 2^-8.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = 2.0 ** -8
EPS = 1e-5


def draw(L, H, G, P, N, seed):
    d = ref.draw(1, L, H, G, P, N, BF, seed=seed, unit=False)
    gen = torch.Generator().manual_seed(seed + 1)
    n = lambda *s: torch.randn(s, generator=gen)
    d |= dict(x=n(L, H * P).to(BF), residual=(2 * n(L, H * P)).to(BF), z=n(1, L, H, P).to(BF),
              w1=1 + 0.2 * n(H * P), w2=1 + 0.2 * n(P), dout=n(1, L, H, P).to(BF))
    return d


def block(d, dev):
    """The block's forward on the GPU: (y, h, o, final state, the gated norm's output)."""
    L, H, P = d["x"].shape[0], d["z"].shape[2], d["z"].shape[3]
    y, h = ssd.rms_norm(d["x"], d["w1"], eps=EPS, residual=d["residual"])
    o, s = ssd.delta_rule_fwd(d["q"], d["k"], y.view(1, L, H, P), d["g"], d["beta"],
                              init_state=d["init"], qk_l2norm=True)
    out = ssd.rms_norm(o, d["w2"], eps=EPS, z=d["z"], gate="post")
    return y, h, o, s, out


@pytest.mark.parametrize("L,H,G,P", [(150, 4, 2, 64), (130, 40, 1, 64), (40, 20, 4, 128)])
def test_forward_stages_and_decode(cuda_device, L, H, G, P):
    N = 128
    cpu = draw(L, H, G, P, N, seed=L)
    d = {k: v.to(cuda_device) for k, v in cpu.items()}
    y, h, o, s, out = block(d, cuda_device)
    y_ref, h_ref = ref.rms_norm(cpu["x"], cpu["w1"], EPS, residual=cpu["residual"])
    assert torch.equal(h.cpu(), h_ref) and ref.rel(y, y_ref) <= 1.1 * HALF
    o_ref, s_ref = ref.delta_rule(cpu["q"], cpu["k"], y.cpu().view(1, L, H, P), cpu["g"], cpu["beta"],
                                  cpu["init"], N ** -0.5, True)
    tol = 4 * (L + 32) * 2.0 ** -24 + 4 * 2.0 ** -16
    assert ref.rel(s, s_ref) <= tol and ref.rel(o, o_ref) <= tol + 3 * HALF
    out_ref, _ = ref.rms_norm(o.cpu(), cpu["w2"], EPS, z=cpu["z"], gate="post")
    assert ref.rel(out, out_ref) <= 1.1 * HALF
    # the same rows in 8 bits, a scale per head
    y8, scales = ssd.rms_norm(o, d["w2"], eps=EPS, z=d["z"], gate="post", quant_group=P)
    assert ref.rel(y8.float() * scales, out_ref) <= 2.0 ** -4
    # one more token from the state that prefill left = the last row of one more token of prefill
    more = draw(L + 1, H, G, P, N, seed=L + 7)
    for name in ("q", "k", "g", "beta", "z", "x", "residual"):
        dim = 0 if name in ("x", "residual") else 1
        more[name][(slice(None),) * dim + (slice(0, L),)] = cpu[name]
    for name in ("w1", "w2", "init"):
        more[name] = cpu[name]
    m = {k: v.to(cuda_device) for k, v in more.items()}
    *_, s2, out2 = block(m, cuda_device)
    y1, _ = ssd.rms_norm(m["x"][-1:], m["w1"], eps=EPS, residual=m["residual"][-1:])
    o1 = ssd.delta_rule_update(s, *(m[n][:, -1].contiguous() for n in ("q", "k")),
                               y1.view(1, H, P), m["g"][:, -1].contiguous(),
                               m["beta"][:, -1].contiguous(), qk_l2norm=True)
    out1 = ssd.rms_norm(o1, m["w2"], eps=EPS, z=m["z"][:, -1].contiguous(), gate="post")
    assert ref.rel(s, s2.cpu()) <= 2 * tol
    assert ref.rel(out1, out2[:, -1].cpu()) <= 2 * (tol + 4 * HALF)


@pytest.mark.parametrize("L,H,G,P", [(150, 4, 2, 64), (70, 40, 1, 64)])
def test_backward_of_the_block(cuda_device, L, H, G, P):
    N = 128
    cpu = draw(L, H, G, P, N, seed=L + 3)
    leaf = {n: cpu[n].double().requires_grad_()
            for n in ("x", "residual", "q", "k", "g", "beta", "z", "w1", "w2", "init")}
    hh = leaf["x"] + leaf["residual"]
    norm = lambda t, w: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * w
    y = norm(hh, leaf["w1"]).view(1, L, H, P)
    o, _ = ref.delta_rule(leaf["q"], leaf["k"], y, leaf["g"], leaf["beta"], leaf["init"], N ** -0.5,
                          True)
    (norm(o, leaf["w2"]) * ref.silu(leaf["z"]) * cpu["dout"].double()).sum().backward()

    d = {k: v.to(cuda_device) for k, v in cpu.items()}
    y, h, o, _, _ = block(d, cuda_device)
    last = ssd.rms_norm_bwd(o, d["w2"], d["dout"], eps=EPS, z=d["z"], gate="post")
    rule = ssd.delta_rule_bwd(d["q"], d["k"], y.view(1, L, H, P), d["g"], d["beta"], last["dx"],
                              init_state=d["init"], qk_l2norm=True)
    first = ssd.rms_norm_bwd(h, d["w1"], rule["dv"].view(L, H * P), eps=EPS)
    got = dict(x=first["dx"], residual=first["dx"], w1=first["dweight"], w2=last["dweight"],
               z=last["dz"], q=rule["dq"], k=rule["dk"], g=rule["dg"], beta=rule["dbeta"],
               init=rule["dinit"])
    for name, g in got.items():
        assert ref.rel(g, leaf[name].grad) <= 2 * 12 * HALF, name
