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
