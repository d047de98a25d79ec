"""The gated delta rule where launches are large enough that a CTA takes many heads, a warp a second
one and the gradients' kernel sums several heads in its registers: against the float64 recurrence, run
on the GPU, head by head, group by group and span by span, so that no part hides behind the others.

Forward tolerances are the chunked kernels': the state's factors in two bf16 parts, 4 * 2^-16, and float32
sums over the tokens it remembers, 4 (L + 32) * 2^-24; the output's rounding and the bf16 parts that it
alone takes, 3 * 2^-8; four times these for one head of one sequence.

Gradients.  A value rounded to bf16 is off by at most 2^-8 of it, 2^-8 / sqrt(3) or less in the mean of
squares (u).  dv is rounded once.  dq and dk are rounded once and are sums of products of which a state
or triangle on one side and W or dV on the other are rounded, independently: sqrt(2) u of each term; the
terms may cancel to half their joint size: sqrt(1 + 2 * 4) u = 3 u < 2 * 2^-8.  dinit and dbeta: operands in
two or three bf16 parts, 8 * 2^-16 and the recurrence's float32 sums 8 (L + 32) * 2^-24 as for small calls.
dg weighs two sums of up to 64 tokens' <dO, O> and <dV, V>, whose operands leave up to eight independent
errors of 2^-18 each: 8 / sqrt(3) * sqrt(64) / 2 * 2^-18 < 32 * 2^-18 of a token's terms.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


def on(d, device):
    return {k: None if v is None else v.to(device) for k, v in d.items()}


def args(d):
    return [d[n] for n in NAMES]


def rel(got, want, dims):
    """2-norm of the difference over the 2-norm, per slice over `dims`; the largest."""
    d = (got.double() - want).square().sum(dims).sqrt()
    return float((d / want.square().sum(dims).sqrt()).max())


def check_forward(o, s, o_ref, s_ref, L):
    state = 4 * (L + 32) * 2.0 ** -24 + 4 * 2.0 ** -16
    assert rel(s, s_ref, (2, 3)) <= 4 * state
    assert rel(o, o_ref, (1, 3)) <= 4 * (state + 3 * 2.0 ** -8)


@pytest.mark.parametrize("case", [
    # (b, L, H, G, P, N, l2norm): 16 heads to a CTA of the tcgen05 form's triangles, the last one with 14 ...
    (89, 128, 78, 1, 64, 64, True),
    # ... 8, of 18 heads of a group ...
    (60, 190, 36, 2, 128, 64, False),
    (47, 130, 50, 1, 64, 128, True),
    # ... and of the warp-level form's, where a warp takes up to four of the heads
    (100, 64, 48, 1, 64, 128, True),
    (150, 33, 44, 2, 48, 64, False),
], ids=lambda c: "-".join(str(x) for x in c))
def test_many_heads_to_a_cta(cuda_device, case):
    b, L, H, G, P, N, l2norm = case
    d = on(ref.draw(b, L, H, G, P, N, BF, seed=L + H, unit=not l2norm), cuda_device)
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], N ** -0.5, l2norm)
    o, s = ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=l2norm)
    check_forward(o, s, o_ref, s_ref, L)
    again = ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=l2norm)
    assert torch.equal(o, again[0]) and torch.equal(s, again[1])


def test_many_heads_to_a_cta_packed(cuda_device):
    n, H, G, P, N = 70, 70, 1, 64, 128
    gen = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 320, (n,), generator=gen).tolist()
    lens[5], lens[17], lens[-1] = 0, 1, 65
    cut = [0]
    for x in lens:
        cut.append(cut[-1] + x)
    L, most = cut[-1], max(lens)
    d = on(ref.draw(1, L, H, G, P, N, BF, seed=n, unit=False, nseq=n), cuda_device)
    o, s = ssd.delta_rule_varlen_fwd(
        *args(d), torch.tensor(cut, dtype=torch.int32, device=cuda_device), init_states=d["init"],
        qk_l2norm=True)
    # the sequences as rows of a batch; what is behind their ends writes nothing and decays nothing
    at = torch.tensor(cut[:-1])[:, None] + torch.arange(most)
    there = (at < torch.tensor(cut[1:])[:, None]).to(cuda_device)
    at = at.clamp(max=L - 1).to(cuda_device)
    rows = [x[0][at] * there.view(there.shape + (1,) * (x.dim() - 2)) for x in args(d)]
    o_ref, s_ref = ref.delta_rule(*rows, d["init"], N ** -0.5, True)
    state = 4 * (most + 32) * 2.0 ** -24 + 4 * 2.0 ** -16
    assert rel(s, s_ref, (2, 3)) <= 4 * state
    for i, (a, e) in enumerate(zip(cut, cut[1:])):
        if a < e:
            assert rel(o[:, a:e], o_ref[i:i + 1, :e - a], (1, 3)) <= 4 * (state + 3 * 2.0 ** -8), i
        else:
            assert torch.equal(s[i], d["init"][i])


@pytest.mark.parametrize("P,H", [(64, 40), (128, 20), (48, 6)])
@pytest.mark.parametrize("beta", [1.0, 1.5])
def test_keys_that_repeat(cuda_device, P, H, beta):
    """One key for every token and no decay: the triangular system at its worst, on the tcgen05 form's
    blocks (P 64 and 128) and the warp-level form's.  Its inverse has rows -beta (1 - beta)^j, whose
    sum, at most 1 + beta / (2 - beta), multiplies the error of what it is applied to."""
    L, N = 200, 64
    d = on(ref.draw(1, L, H, 1, P, N, BF, seed=4, unit=False, decay=None), cuda_device)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = beta
    d["beta"][:, ::7] *= 0.9
    o_ref, s_ref = ref.delta_rule(*args(d)[:3], torch.zeros_like(d["beta"]), d["beta"], d["init"],
                                  N ** -0.5, True)
    o, s = ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=True)
    grow = 1 + beta / (2 - beta)
    state = (4 * (L + 32) * 2.0 ** -24 + 4 * 2.0 ** -16) * grow
    assert rel(s, s_ref, (2, 3)) <= 4 * state
    assert rel(o, o_ref, (1, 3)) <= 4 * (state + grow * 3 * 2.0 ** -8)


BACKWARD = [
    # (b, L, H, G, P, N, l2norm): heads summed in registers: 3 to a CTA, the last one with 1 ...
    (4, 130, 64, 1, 16, 64, True),
    (8, 130, 80, 1, 16, 64, False),     # ... 7, the last one with 3 ...
    (2, 100, 41, 1, 128, 128, True),    # ... 2 of 128 rows, the last one with 1 ...
    (6, 200, 24, 2, 64, 128, True),
    (20, 70, 80, 1, 48, 64, True),      # ... and a second head to a warp of the triangles
]


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(str(x) for x in c))
def test_backward_of_many_heads(cuda_device, case):
    b, L, H, G, P, N, l2norm = case
    d = on(ref.draw(b, L, H, G, P, N, BF, seed=L + H, unit=not l2norm), cuda_device)
    gen = torch.Generator().manual_seed(7)
    dout = torch.randn((b, L, H, P), generator=gen).to(BF).to(cuda_device)
    dfinal = torch.randn((b, H, P, N), generator=gen).to(cuda_device)
    leaf = {n: d[n].double().requires_grad_() for n in NAMES + ("init",)}
    o, S = ref.delta_rule(*(leaf[n] for n in NAMES + ("init",)), N ** -0.5, l2norm)
    torch.autograd.backward([o, S], [dout.double(), dfinal.double()])
    want = {"d" + n: leaf[n].grad for n in leaf}
    terms = ((o.detach() * dout).sum(-1).square() + (want["dv"] * d["v"]).sum(-1).square())
    del o, S
    run = lambda: ssd.delta_rule_bwd(*args(d), dout, init_state=d["init"], dfinal=dfinal,
                                     qk_l2norm=l2norm)
    got = run()
    f32 = 8 * 2.0 ** -16 + 8 * (L + 32) * 2.0 ** -24
    last = (L - 1) // 64 * 64                       # the last span's first token
    for part in (slice(0, L), slice(last, L)):
        at = lambda name: (got[name][:, part], want[name][:, part])
        for name in ("dq", "dk"):                   # a group of a sequence
            assert rel(*at(name), (1, 3)) <= 2 * 2.0 ** -8, name
        assert rel(*at("dv"), (1, 3)) <= 2.0 ** -8 + f32
        assert rel(*at("dbeta"), (1,)) <= 2 * f32
        dg, dg_ref = at("dg")
        size = dg_ref.square().sum(1).sqrt() + terms[:, part].sum(1).sqrt()
        assert ((dg.double() - dg_ref).square().sum(1).sqrt() <= 32 * 2.0 ** -18 * size).all()
    assert rel(got["dinit"], want["dinit"], (2, 3)) <= f32
    again = run()
    assert all(torch.equal(got[n], again[n]) for n in got)
