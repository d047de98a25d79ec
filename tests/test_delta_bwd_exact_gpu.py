"""Gradients of the gated delta rule whose value, or whose error, is known more closely than the
operands' roundings: where an input has no effect its gradient is 0 to the bit."""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def args(d):
    return [d[n] for n in ("q", "k", "v", "g", "beta")]


@pytest.mark.parametrize("L", [1, 2, 33, 65])
@pytest.mark.parametrize("P,N,l2norm", [(128, 64, True), (64, 128, False), (16, 64, True)])
def test_decay_before_any_token_has_no_gradient(cuda_device, L, P, N, l2norm):
    """dg_t = <dS, exp(g_t) S_{t-1}>, and without an initial state S is 0 before the first token: its
    decay changes nothing, and its gradient is exactly 0 -- not what is left of sums that cancel."""
    d = ref.draw(2, L, 4, 2, P, N, BF, seed=L, unit=not l2norm, init=False)
    c = {k: None if x is None else x.to(cuda_device) for k, x in d.items()}
    gen = torch.Generator().manual_seed(5)
    dout = torch.randn(d["v"].shape, generator=gen).to(BF).to(cuda_device)
    dfinal = torch.randn((2, 4, P, N), generator=gen).to(cuda_device)
    got = ssd.delta_rule_bwd(*args(c), dout, dfinal=dfinal, qk_l2norm=l2norm)
    assert (got["dg"][:, 0] == 0).all()
    assert L == 1 or (got["dg"][:, 1:] != 0).any()


@pytest.mark.parametrize("P,N", [(64, 128), (128, 64), (48, 128)])
def test_decay_gradient_of_two_tokens(cuda_device, P, N):
    """dg of the second token with the final state's gradient D alone: exp(g_1) <D (I - beta_1 k_1 k_1^T),
    u_0 k_0^T>, of which the kernel takes <D, S'> - <dV_1, V_1>, sums over P N and P terms.  D, as operand,
    and the values written are held in three bf16 parts (2^-24) and leave no error beside float32's: over
    64 heads, in the mean of squares, a sum of n random terms loses about sqrt(n) / 2 * 2^-25 of itself to
    its lanes' additions (64 at most one after the other: 2e-7), three such sums 2^-21 at most, and D k in
    products of 128 as much again.  The triangle's inverse and what it multiplies enter as two parts each:
    three errors of 2^-18 of exp(g_1) beta_0 (k_1 . k_0) dV_1 . W_0.  (In two parts D and the values
    written cost 2.7e-6.)"""
    H = 64
    d = ref.draw(1, 2, H, H, P, N, BF, seed=P + N, unit=True, init=False)
    gen = torch.Generator().manual_seed(8)
    dfinal = torch.randn((1, H, P, N), generator=gen)
    c = {k: None if x is None else x.to(cuda_device) for k, x in d.items()}
    got = ssd.delta_rule_bwd(*args(c), torch.zeros_like(c["v"]), dfinal=dfinal.to(cuda_device))
    k, v, g, beta = (d[n][0].double() for n in ("k", "v", "g", "beta"))
    D = dfinal[0].double()
    D0, D1 = ((D * k[t][:, None, :]).sum(-1) for t in (0, 1))              # D k_t: (H, P)
    dv1 = beta[1][:, None] * D1
    kk = (k[0] * k[1]).sum(-1)
    through_k = torch.exp(g[1]) * beta[0] * kk * (dv1 * v[0]).sum(-1)
    want = torch.exp(g[1]) * beta[0] * (D0 * v[0]).sum(-1) - through_k
    err = (got["dg"][0, 1].double().cpu() - want).norm()
    assert err <= 2.0 ** -20 * want.norm() + 3 * 2.0 ** -18 * through_k.norm()
