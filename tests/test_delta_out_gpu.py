"""The output of the gated delta rule's chunked kernels is off by its own rounding to bf16 and little else:
no operand of its products is rounded to bf16 as a whole.

A value m 2^e (1 <= m < 2) is rounded to a multiple of 2^(e-7): off by at most 2^-8 2^e, evenly spread, so
2^-8 / sqrt(3) 2^e or less of it in the mean of squares; of the 2-norm that is at most 2^-8 / sqrt(3), since m >= 1.
Over 75000 values and more the mean of squares is within 2 % of that.  The operands' two bf16 parts and
the float32 sums add the state's tolerance, 4 * 2^-16 + 4 (L + 32) * 2^-24.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def bound(L):
    return 1.02 * 2.0 ** -8 / 3 ** 0.5 + 4 * 2.0 ** -16 + 4 * (L + 32) * 2.0 ** -24


@pytest.mark.parametrize("b,L,H,G,P,N,l2norm,init", [
    (1, 300, 4, 2, 64, 128, True, True),        # warp-level form
    (2, 300, 6, 1, 48, 64, False, True),
    (1, 130, 10, 1, 112, 128, True, False),
    (20, 64, 20, 2, 64, 64, True, True),
    (1, 300, 40, 1, 64, 128, True, True),       # tcgen05 form
    (2, 129, 21, 7, 64, 64, False, False),
    (1, 200, 20, 2, 128, 128, True, True),
    (1, 511, 19, 1, 128, 64, True, False),
])
def test_output_is_off_by_its_rounding(cuda_device, b, L, H, G, P, N, l2norm, init):
    d = ref.draw(b, L, H, G, P, N, BF, seed=L + P + H, unit=not l2norm, init=init)
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    o_ref, _ = ref.delta_rule(*args, d["init"], N ** -0.5, l2norm)
    o, _ = ssd.delta_rule_fwd(*(x.to(cuda_device) for x in args), qk_l2norm=l2norm,
                              init_state=None if d["init"] is None else d["init"].to(cuda_device))
    assert o.numel() >= 75000
    assert ref.rel(o, o_ref) <= bound(L)


@pytest.mark.parametrize("P,H", [(64, 40), (128, 20), (48, 8)])
def test_packed(cuda_device, P, H):
    cu, G, N = [0, 70, 70, 264, 400], 2, 128
    d = ref.draw(1, cu[-1], H, G, P, N, BF, seed=P, unit=False, nseq=4)
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    parts = [ref.delta_rule(*(x[:, a:e] for x in args), d["init"][i:i + 1], N ** -0.5, True)[0]
             for i, (a, e) in enumerate(zip(cu, cu[1:])) if a < e]
    o, _ = ssd.delta_rule_varlen_fwd(
        *(x.to(cuda_device) for x in args), torch.tensor(cu, dtype=torch.int32, device=cuda_device),
        init_states=d["init"].to(cuda_device), qk_l2norm=True)
    assert o.numel() >= 75000
    assert ref.rel(o, torch.cat(parts, 1)) <= bound(cu[-1])


@pytest.mark.parametrize("b,L,H,G,P,N", [(8, 60, 6, 2, 64, 128), (8, 64, 4, 2, 128, 64),
                                         (12, 33, 4, 4, 48, 64), (6, 50, 9, 1, 128, 128)])
def test_gradients_of_keys_and_queries_are_off_by_their_rounding(cuda_device, b, L, H, G, P, N):
    """Within one span of 64 tokens from an empty state, with no gradient of the final one, dq is sum over
    j <= i of M1_ij k_j, M1_ij = scale exp(cs_i - cs_j) beta_j (dO_i . W_j): neither M1 nor W is rounded to
    bf16 as a whole, and dq is off by its own rounding.  dk is M1^T q less (M2 + M2^T) k, M2_ij = exp(cs_i -
    cs_j) beta_j (dV_i . W_j) below the diagonal, where M2 and dV are rounded: 2^-8 / sqrt(3) of that term
    each."""
    d = ref.draw(b, L, H, G, P, N, BF, seed=L + P, init=False)
    dout = torch.randn((b, L, H, P), generator=torch.Generator().manual_seed(3)).to(BF)
    leaf = {n: d[n].double().requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    o, _ = ref.delta_rule(*leaf.values(), None, N ** -0.5, False)
    o.backward(dout.double())
    # W by the recurrence, then the term of M2
    k, v, g, beta = (leaf[n].detach() for n in ("k", "v", "g", "beta"))
    k = ref.heads(k, H)
    S, W = torch.zeros(b, H, P, N, dtype=torch.float64), []
    for t in range(L):
        S = torch.exp(g[:, t])[..., None, None] * S
        W.append(v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + (beta[:, t, :, None] * W[-1])[..., None] * k[:, t, :, None, :]
    W = torch.stack(W, 1)
    cs = g.cumsum(1)
    M2 = torch.einsum("bihp,bjhp->bhij", leaf["v"].grad, W) * beta.transpose(1, 2)[:, :, None]
    M2 = (M2 * torch.exp((cs[:, :, None] - cs[:, None]).permute(0, 3, 1, 2).clamp(max=0))).tril(-1)
    term = torch.einsum("bhij,bjhn->bihn", M2 + M2.transpose(2, 3), k)
    term = term.unflatten(2, (G, -1)).sum(3)
    got = ssd.delta_rule_bwd(*(d[n].to(cuda_device) for n in ("q", "k", "v", "g", "beta")),
                             dout.to(cuda_device))
    u, more = 1.02 * 2.0 ** -8 / 3 ** 0.5, 8 * 2.0 ** -16 + 8 * (L + 32) * 2.0 ** -24
    dq, dk = leaf["q"].grad, leaf["k"].grad
    assert ref.rel(got["dq"], dq) <= u + more
    share = float(term.norm() / dk.norm())
    assert ref.rel(got["dk"], dk) <= u * (1 + 2 * share ** 2) ** 0.5 + more
