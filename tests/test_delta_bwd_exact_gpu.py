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


@pytest.mark.parametrize("P,N", [(64, 128), (128, 128), (64, 64)])
def test_decays_behind_tokens_that_wipe_the_state_out(cuda_device, P, N):
    """Sixty tokens of g = -200, then fractions of 2^-10: the running sum of g is near -12000, where a
    float32 keeps steps of 2^-10 only, but the decay between the last tokens is a difference of such
    sums and has float32's accuracy.  One token (61) writes; dk there is beta exp(g_62 + g_63) D^T v,
    D the final state's gradient, in exact operands: all that is rounded is dk itself, each value by
    at most 2^-8 of it, which over the n = H N values' projection on the true ones has a deviation of
    at most 2^-8 / sqrt(n) (|x|^4 of a normal x is 3); six of them are allowed.  (The sum in one float32
    is off by 1.27e-3 here.)"""
    H, L = 64, 64
    gen = torch.Generator().manual_seed(P + N)
    n = lambda *s: torch.randn(s, generator=gen)
    k = n(1, L, H, N)
    k = (k / k.norm(dim=-1, keepdim=True)).to(BF)
    v, dfinal = n(1, L, H, P).to(BF), n(1, H, P, N).to(BF).float()
    g = torch.full((1, L, H), -200.0)
    g[:, 60], g[:, 61], g[:, 62], g[:, 63] = -0.65 * 2.0 ** -10, 0, -0.7 * 2.0 ** -10, 0
    beta = torch.zeros(1, L, H)
    beta[:, 61] = 0.5
    c = [x.to(cuda_device) for x in (k, k, v, g, beta)]
    got = ssd.delta_rule_bwd(*c, torch.zeros_like(c[2]), dfinal=dfinal.to(cuda_device))
    decay = torch.exp(g[0, 62:].double().sum(0))[:, None]
    want = 0.5 * decay * (dfinal[0].double() * v[0, 61].double()[..., None]).sum(1)   # (H, N)
    dk = got["dk"][0, 61].double().cpu()
    along = float((dk * want).sum() / (want * want).sum()) - 1
    assert abs(along) <= 6 * 2.0 ** -8 * (H * N) ** -0.5
    # a beta of 0 is taken as 1e-20: |dk| <= |dv| |S|, |dv| <= 1e-20 |D| |k| and |S| <= 0.5 |v|, with values
    # of D and v below 6: 1e-20 * 6 * 128 * 0.5 * 6 * sqrt(128) < 1e-15
    assert (got["dk"][0, 62:].abs() <= 1e-15).all()
