"""The scalars of the gated delta rule's and the RMS norm's calls are taken at the call: what the binding
keeps from call to call goes by their values (no GPU needed)."""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import build, ssd


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def options(scale, l2norm=False):
    return ssd._delta_options(scale, 64, l2norm)._obj


def desc(eps, quant_group=0):
    x, w = torch.zeros(4, 64), torch.zeros(64)
    return ssd._norm_inputs(x, w, eps, None, "none", quant_group, ()).desc


def test_scale_that_changes_in_place():
    scale = torch.tensor(2.0)
    assert options(scale).scale == 2.0
    scale.mul_(3)
    assert options(scale).scale == 6.0
    on = torch.tensor(False)
    assert options(2.0, on).qk_l2norm == 0
    on.fill_(True)
    assert options(2.0, on).qk_l2norm == 1
    assert options(None).scale == 0.125


def test_eps_and_groups_that_change_in_place():
    eps = torch.tensor(0.5)
    assert desc(eps).eps == 0.5
    eps.fill_(0.25)
    assert desc(eps).eps == 0.25
    group = torch.tensor(32)
    assert desc(0.5, group).quant_group == 32
    group.fill_(64)
    assert desc(0.5, group).quant_group == 64
    with pytest.raises(TypeError):
        desc(0.5, 32.5)


def test_equal_values_share_what_is_kept():
    assert options(0.5) is options(0.5) and options(0.5) is not options(0.25)
    assert desc(0.5) is desc(torch.tensor(0.5))
