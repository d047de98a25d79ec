"""Delta rule and norm calls on another stream than the current one: where their memory comes from."""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _norm(dev):
    x, w = torch.randn(1024, 2048, device=dev, dtype=BF), torch.ones(2048, device=dev)
    return x, lambda **kw: ssd.rms_norm(x, w, **kw)


def _norm_bwd(dev):
    x, w = torch.randn(1024, 2048, device=dev, dtype=BF), torch.ones(2048, device=dev)
    return x, lambda **kw: ssd.rms_norm_bwd(x, w, x, **kw)["dx"]


def _delta(call):
    def make(dev):
        d = {k: x.to(dev) for k, x in ref.draw(1, 2048, 16, 1, 64, 64, BF).items()}
        args = [d[n] for n in ("q", "k", "v", "g", "beta")]
        return d["v"], lambda **kw: call(*args, **kw)
    return make


def _varlen(dev):
    cut = torch.tensor([0, 1000, 2048], dtype=torch.int32, device=dev)
    return _delta(lambda *a, **kw: ssd.delta_rule_varlen_fwd(*a, cut, **kw)[0])(dev)


def _update(dev):
    d = {k: x.to(dev) for k, x in ref.draw(256, 1, 128, 1, 64, 64, BF).items()}
    step = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    return step[2], lambda **kw: ssd.delta_rule_update(d["init"], *step, **kw)


CALLS = dict(norm=_norm, norm_bwd=_norm_bwd, update=_update, varlen=_varlen,
             forward=_delta(lambda *a, **kw: ssd.delta_rule_fwd(*a, **kw)[0]),
             backward=_delta(lambda q, k, v, g, beta, **kw: ssd.delta_rule_bwd(
                 q, k, v, g, beta, v, **kw)["dv"]))


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(cuda_device, name):
    """The call may not write what the current stream still has to read, though the tensor is gone and
    its memory free for the current stream's next one; and its output, gone too, may not be handed to
    the other stream while the current one still has to read it."""
    like, call = CALLS[name](cuda_device)   # 4 MB: a tensor and the output are blocks of one size
    want = call().clone()
    current, side = torch.cuda.current_stream(), torch.cuda.Stream()
    got_here = torch.empty_like(like)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.full_like(like, 3.0)
    kept, where = torch.empty_like(held), held.data_ptr()
    side.wait_stream(current)
    torch.cuda._sleep(100_000_000)          # some 50 ms
    kept.copy_(held)
    del held
    got = call(stream=side)
    assert got.data_ptr() != where
    side.synchronize()
    torch.cuda.synchronize()
    assert (kept == 3).all()
    if name != "update":                    # (its state has moved on)
        assert torch.equal(got, want)
    before, at = got.clone(), got.data_ptr()
    torch.cuda._sleep(100_000_000)
    got_here.copy_(got)
    del got
    with torch.cuda.stream(side):
        other = torch.full_like(like, 5.0)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got_here, before)
