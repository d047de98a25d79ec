"""The gated delta rule's gradients on the GPU against autograd of the float64 recurrence, and that
against differences.

Tolerances (2-norm of the difference over the 2-norm of the reference, per gradient).  dinit, dg and
dbeta are float32: their factors are held as two bf16 parts (2^-16 each), the state, its gradient,
the residuals, W, dV and the two triangles: 8 * 2^-16, plus the float32 sums of the recurrence,
8 (L + 32) * 2^-24.  dg is a difference of sums over up to 64 tokens: its error is measured against
the terms, 8 * 2^-16 * sqrt(64) of one token's <dO, O> and <dV, V>.  dq, dk and dv are bf16: their own
rounding (2^-8) and, for dq and dk, those of the operands of the last products -- the states or
triangles on one side, W or dV on the other (2 * 2^-8 per product of which up to four are summed, the
terms of dk partly cancelling, which doubles them against their sum).
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

BF = torch.bfloat16
HALF = 2.0 ** -8


def grads(d, dout, dfinal, scale, l2norm):
    """float64 gradients of <dout, o> + <dfinal, S>, and <dO, O> and <dV, V> per token and head."""
    names = [n for n in ("q", "k", "v", "g", "beta", "init") if d[n] is not None]
    leaf = {n: d[n].double().requires_grad_() for n in names}
    get = lambda n: leaf.get(n)
    o, S = ref.delta_rule(*(get(n) for n in ("q", "k", "v", "g", "beta", "init")), scale, l2norm)
    loss = (o * dout.double()).sum()
    if dfinal is not None:
        loss = loss + (S * dfinal.double()).sum()
    loss.backward()
    out = {"d" + n: leaf[n].grad for n in names}
    terms = ((o.detach() * dout.double()).sum(-1) ** 2
             + (out["dv"] * d["v"].double()).sum(-1) ** 2).sum() ** 0.5
    return out, float(terms)


def check(got, want, terms, L):
    f32 = 8 * 2.0 ** -16 + 8 * (L + 32) * 2.0 ** -24
    for name, w in want.items():
        if w is None:
            continue
        name = "dinit" if name == "dinit" else name
        err = float((got[name].double().cpu() - w).norm())
        size = float(w.norm())
        if name == "dg":
            bound = f32 * (size + 8 * terms)
        elif name in ("dbeta", "dinit"):
            bound = f32 * size
        elif name == "dv":
            bound = (HALF + f32) * size
        else:
            bound = (HALF + 2 * 2 * 2 * HALF) * size
        assert err <= bound + 1e-12, f"{name}: {err / max(size, 1e-30):.3g} of it off, {bound / max(size, 1e-30):.3g} allowed"


CASES = [
    # (b, L, H, G, P, N, l2norm, init, dfinal, decay)
    (1, 1, 1, 1, 64, 128, False, True, True, "mixed"),
    (2, 3, 4, 2, 64, 128, True, False, True, "mixed"),
    (1, 32, 2, 1, 64, 128, False, True, False, "mixed"),
    (1, 33, 4, 1, 64, 128, True, True, True, "mixed"),
    (2, 64, 4, 4, 128, 128, True, True, True, "mixed"),
    (1, 65, 6, 2, 64, 64, True, True, True, "strong"),
    (1, 97, 5, 1, 48, 128, True, True, True, None),
    (1, 160, 3, 1, 16, 64, False, True, True, "mixed"),
    (2, 200, 10, 1, 64, 128, True, True, True, "mixed"),     # runs of heads, the last one shorter
    (1, 130, 9, 1, 128, 64, False, False, False, "mixed"),
    (1, 500, 4, 2, 64, 128, True, True, True, "mixed"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_backward(cuda_device, case):
    b, L, H, G, P, N, l2norm, init, with_final, decay = case
    d = ref.draw(b, L, H, G, P, N, BF, seed=L + P, unit=not l2norm, decay=decay, init=init)
    gen = torch.Generator().manual_seed(77)
    dout = torch.randn((b, L, H, P), generator=gen).to(BF)
    dfinal = torch.randn((b, H, P, N), generator=gen) if with_final else None
    want, terms = grads(d, dout, dfinal, N ** -0.5, l2norm)
    c = {k: None if x is None else x.to(cuda_device) for k, x in d.items()}
    call = lambda: ssd.delta_rule_bwd(
        *(c[n] for n in ("q", "k", "v", "g", "beta")), dout.to(cuda_device),
        init_state=c["init"], dfinal=None if dfinal is None else dfinal.to(cuda_device),
        qk_l2norm=l2norm)
    got = call()
    assert got["dq"].dtype == got["dk"].dtype == got["dv"].dtype == BF
    assert (got["dg"] is None) == (d["g"] is None)
    check(got, want, terms, L)
    again = call()
    assert all(torch.equal(got[k], again[k]) for k in got if got[k] is not None)


@pytest.mark.gpu
def test_beta_of_zero_and_rows_without_a_key(cuda_device):
    """Where beta is 0 dbeta is still the gradient (the token would have written something), dv is
    nothing; a key of zeros under the norm gets a gradient of at most that of its epsilon."""
    d = ref.draw(1, 80, 4, 2, 64, 128, BF, seed=2, unit=False)
    d["beta"][:, ::3] = 0.0
    d["beta"][:, 1::3] = 1.0
    d["q"][:, 7] = 0
    dout = torch.randn((1, 80, 4, 64), generator=torch.Generator().manual_seed(1)).to(BF)
    want, terms = grads(d, dout, None, 128 ** -0.5, True)
    c = {k: x.to(cuda_device) for k, x in d.items()}
    got = ssd.delta_rule_bwd(*(c[n] for n in ("q", "k", "v", "g", "beta")), dout.to(cuda_device),
                             init_state=c["init"], qk_l2norm=True)
    check(got, want, terms, 80)
    assert (got["dv"][:, ::3].abs() <= 1e-15).all()


@pytest.mark.gpu
def test_against_differences(cuda_device):
    """A few elements of every gradient against central differences of the float64 recurrence."""
    b, L, H, G, P, N = 1, 40, 2, 1, 16, 64
    d = ref.draw(b, L, H, G, P, N, BF, seed=6, unit=False)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn((b, L, H, P), generator=gen).to(BF)
    dfinal = torch.randn((b, H, P, N), generator=gen)
    c = {k: x.to(cuda_device) for k, x in d.items()}
    got = ssd.delta_rule_bwd(*(c[n] for n in ("q", "k", "v", "g", "beta")), dout.to(cuda_device),
                             init_state=c["init"], dfinal=dfinal.to(cuda_device), qk_l2norm=True)

    def loss(**kw):
        a = {k: x.double() for k, x in d.items()} | kw
        o, S = ref.delta_rule(*(a[n] for n in ("q", "k", "v", "g", "beta", "init")), N ** -0.5, True)
        return float((o * dout.double()).sum() + (S * dfinal.double()).sum())

    for name in ("q", "k", "v", "g", "beta", "init"):
        flat = d[name].double().flatten()
        size = float(got["d" + name].float().abs().max())
        for i in torch.randint(flat.numel(), (6,), generator=gen).tolist():
            step = torch.zeros_like(flat)
            step[i] = 1e-5
            up, down = (loss(**{name: (flat + s * step).view(d[name].shape)}) for s in (1, -1))
            diff = (up - down) / 2e-5
            assert abs(float(got["d" + name].flatten()[i]) - diff) <= 9 * HALF * size


@pytest.mark.gpu
def test_empty_calls_guard_bands_and_streams(cuda_device):
    dev = cuda_device
    d = {k: x.to(dev) for k, x in ref.draw(2, 0, 4, 2, 64, 128, BF).items()}
    args = lambda d: [d[n] for n in ("q", "k", "v", "g", "beta")]
    fin = torch.randn(2, 4, 64, 128, device=dev)
    got = ssd.delta_rule_bwd(*args(d), d["v"], init_state=d["init"], dfinal=fin)
    assert torch.equal(got["dinit"], fin) and got["dq"].shape == (2, 0, 2, 128)
    d = {k: x.to(dev) for k, x in ref.draw(2, 150, 4, 2, 64, 128, BF, unit=False).items()}
    dout = torch.randn(d["v"].shape, device=dev).to(BF)
    run = lambda **kw: ssd.delta_rule_bwd(*args(d), dout, init_state=d["init"], dfinal=fin,
                                          qk_l2norm=True, **kw)
    want = run()
    shape = ssd.make_shape(2, 150, 4, 64, 128, 2, ssd.SSD_BF16)
    import ctypes
    size = ssd.lib().ssd_delta_rule_bwd_workspace_size(ctypes.byref(shape))
    ws = torch.full((size + 512,), 9, dtype=torch.uint8, device=dev)
    got = run(workspace=ws[256:-256])
    torch.cuda.synchronize()
    assert (ws[:256] == 9).all() and (ws[-256:] == 9).all()
    assert all(torch.equal(want[k], got[k]) for k in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    # captured, then replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for k, x in ref.draw(2, 150, 4, 2, 64, 128, BF, seed=9, unit=False).items():
        d[k].copy_(x)
    graph.replay()
    want = run()
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)


def test_refusals():
    import ctypes
    from mamba_ssd_layer_scan_b200 import build
    build.build()
    L = ssd.lib()
    ok, mis = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
    o = ssd.DeltaOptions(0.1, 1)

    def call(sh, **kw):
        p = dict(q=ok, k=ok, v=ok, g=ok, beta=ok, init=None, dout=ok, dfinal=None, dq=ok, dk=ok,
                 dv=ok, dg=ok, dbeta=ok, dinit=None, ws=ok, n=1 << 40, o=o) | kw
        return L.ssd_delta_rule_bwd(
            ctypes.byref(sh), p["q"], p["k"], p["v"], p["g"], p["beta"],
            ctypes.byref(p["o"]) if p["o"] else None, p["init"], p["dout"], p["dfinal"], p["dq"],
            p["dk"], p["dv"], p["dg"], p["dbeta"], p["dinit"], p["ws"], p["n"], None)

    good = dict(batch=2, seqlen=50, nheads=4, headdim=64, dstate=128, ngroups=2,
                dtype=ssd.SSD_BF16)
    for kw in (dict(dtype=ssd.SSD_F32), dict(headdim=40), dict(dstate=256), dict(dstate=32)):
        sh = ssd.make_shape(**(good | kw))
        assert call(sh) == ssd.SSD_ERR_UNSUPPORTED
        assert L.ssd_delta_rule_bwd_workspace_size(ctypes.byref(sh)) == 0
    sh = ssd.make_shape(**good)
    for kw in ([{n: None} for n in ("q", "k", "v", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta",
                                    "ws", "o", "g")]
               + [{n: mis} for n in ("q", "k", "v", "init", "dout", "dfinal", "dq", "dk", "dv",
                                     "dinit", "ws")] + [dict(n=1000)]):
        assert call(sh, **kw) == ssd.SSD_ERR_INVALID_ARG and ssd.last_error(), kw
    t = lambda *s: torch.zeros(s, dtype=BF)
    f = lambda *s: torch.zeros(s)
    args = (t(1, 5, 1, 64), t(1, 5, 1, 64), t(1, 5, 2, 16), f(1, 5, 2), f(1, 5, 2))
    with pytest.raises(ValueError, match="dout"):
        ssd.delta_rule_bwd(*args, t(1, 5, 2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_bwd(*args, t(1, 5, 2, 16))
