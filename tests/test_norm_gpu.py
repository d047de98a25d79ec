"""GPU parity of the RMS norm, its e4m3 output and its gradients against float64.

Tolerances.  Forward in bf16: the result's rounding is at most 2^-8 of the value; the float32
arithmetic before it (a sum of at most 16384 squares in at most 32 + 16 + 5 sequential additions,
rsqrt, silu by fast exponential and division at about 4 ulp, products) stays below 128 * 2^-24 of
the value.  In float32 the second part alone remains.  e4m3: half a step is 2^-4 of the value, or
2^-10 (half the smallest step) times the scale below the normal range; a value that the float32
error moves over a border is covered by adding that error.  Gradients in float32 are differences
of two terms, so they are held to 256 * 2^-24 of the larger one, which is at most
(|dn w| + |n| |mean|) r; the 2-norm over the row takes that in.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

F32 = 128 * 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-5


def _draw(rows, dim, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)
    return dict(x=n(rows, dim).to(dtype), residual=(2 * n(rows, dim)).to(dtype),
                z=n(rows, dim).to(dtype), dy=n(rows, dim).to(dtype), w=1 + 0.3 * n(dim))


DIMS = [1, 7, 8, 33, 64, 72, 128, 130, 200, 256, 1000, 1024, 1025, 1536, 2560, 2561, 4096, 5120,
        8192, 16384]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("mode", ["plain", "residual", "pre", "post"])
def test_forward(cuda_device, dim, dtype, mode):
    d = _draw(37, dim, dtype, seed=dim)
    kw = {}
    if mode == "residual":
        kw = dict(residual=d["residual"])
    elif mode != "plain":
        kw = dict(z=d["z"], gate=mode)
    y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, **kw)
    dev = {k: v.to(cuda_device) if torch.is_tensor(v) else v for k, v in kw.items()}
    out = ssd.rms_norm(d["x"].to(cuda_device), d["w"].to(cuda_device), eps=EPS, **dev)
    y = out
    if mode == "residual":
        y, h = out
        assert torch.equal(h.cpu(), h_ref)
    assert y.dtype == dtype
    err = (y.cpu().double() - y_ref).abs()
    assert (err <= (STEP[dtype] + F32) * y_ref.abs() + 1e-30).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 32), (160, 32),
                                       (1280, 64), (2560, 128), (2560, 2560), (1537, 1537),
                                       (5, 5), (16384, 128), (16384, 16384)])
@pytest.mark.parametrize("mode", ["residual", "post"])
def test_forward_e4m3(cuda_device, dim, group, dtype, mode):
    d = _draw(19, dim, dtype, seed=dim + group)
    d["x"][3] = 0
    d["residual"][3] = 0        # a row of nothing: the smallest scale, zeros
    kw = dict(residual=d["residual"]) if mode == "residual" else dict(z=d["z"], gate=mode)
    y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, **kw)
    dev = {k: v.to(cuda_device) if torch.is_tensor(v) else v for k, v in kw.items()}
    out = ssd.rms_norm(d["x"].to(cuda_device), d["w"].to(cuda_device), eps=EPS, quant_group=group,
                       **dev)
    y8, scales = out[0].cpu(), out[1].cpu()
    assert y8.dtype == torch.float8_e4m3fn and scales.shape == (19, dim // group)
    groups = y_ref.view(19, -1, group)
    s_ref = (groups.abs().amax(-1) / 448).clamp_min(1e-30)
    assert ((scales.double() - s_ref).abs() <= F32 * s_ref).all()
    assert (scales[3] == torch.tensor(1e-30)).all() and (y8[3].float() == 0).all()
    got = y8.float().double().view_as(groups) * scales.double()[..., None]
    bound = (2.0 ** -4 + 4 * F32) * groups.abs() + (2.0 ** -10 + F32) * s_ref[..., None]
    assert ((got - groups).abs() <= bound).all()
    if mode == "residual":
        assert torch.equal(out[2].cpu(), h_ref)


@pytest.mark.parametrize("quant", [0, 64, 128])
def test_nan_and_infinite_rows_stay_in_their_rows(cuda_device, quant):
    d = _draw(6, 128, torch.bfloat16)
    d["x"][1, 5] = float("nan")
    d["x"][4, 9] = float("inf")
    out = ssd.rms_norm(d["x"].to(cuda_device), d["w"].to(cuda_device), eps=EPS, quant_group=quant)
    y = (out[0] if quant else out).float().cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[4, 9])
    assert torch.isfinite(y[[0, 2, 3, 5]]).all()
    if quant:
        assert torch.isnan(out[1][1]).all() and torch.isfinite(out[1][[0, 2, 3, 5]]).all()


def _grads(d, eps, gate, residual):
    """float64 gradients by autograd of the definition, at the stored sum."""
    x = d["x"].double().requires_grad_()
    z = d["z"].double().requires_grad_()
    w = d["w"].double().requires_grad_()
    n = x * ref.silu(z) if gate == "pre" else x
    y = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + eps) * w
    if gate == "post":
        y = y * ref.silu(z)
    y.backward(d["dy"].double())
    dx = x.grad + (d["residual"].double() if residual else 0)
    return dx, w.grad, z.grad if gate != "none" else None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("mode", ["plain", "residual", "pre", "post"])
def test_backward(cuda_device, dim, dtype, mode):
    rows = 70 if dim > 200 else 1500    # several rows per CTA, and rows past the last full CTA
    d = _draw(rows, dim, dtype, seed=dim)
    gate = mode if mode in ("pre", "post") else "none"
    dx, dw, dz = _grads(d, EPS, gate, mode == "residual")
    c = {k: v.to(cuda_device) for k, v in d.items()}
    got = ssd.rms_norm_bwd(c["x"], c["w"], c["dy"], eps=EPS, gate=gate,
                           z=c["z"] if gate != "none" else None,
                           dresidual=c["residual"] if mode == "residual" else None)
    tol = STEP[dtype] + 2 * F32
    # with one element per row dh is eps r^3 dy w, the difference of two terms of size r dy w:
    # held to float32's error in those
    size = (d["dy"].double() * d["w"].double()).norm() if dim == 1 else 0.0
    assert ref.rel(got["dx"], dx) <= tol + F32 * float(size / dx.norm()) * 400
    assert ref.rel(got["dweight"], dw) <= 2 * F32
    if gate != "none":
        assert ref.rel(got["dz"], dz) <= tol + F32 * float(size / dz.norm()) * 400
    again = ssd.rms_norm_bwd(c["x"], c["w"], c["dy"], eps=EPS, gate=gate,
                             z=c["z"] if gate != "none" else None,
                             dresidual=c["residual"] if mode == "residual" else None)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_backward_against_differences(cuda_device):
    """dx, dz and dweight in float32 against central differences of the float64 definition."""
    d = _draw(3, 40, torch.float32, seed=9)
    c = {k: v.to(cuda_device) for k, v in d.items()}
    for gate in ("pre", "post"):
        got = ssd.rms_norm_bwd(c["x"], c["w"], c["dy"], eps=EPS, z=c["z"], gate=gate)

        def loss(**kw):
            a = {k: d[k].double() for k in ("x", "z", "w")} | kw
            n = a["x"] * ref.silu(a["z"]) if gate == "pre" else a["x"]
            y = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * a["w"]
            return float(((y * ref.silu(a["z"]) if gate == "post" else y) * d["dy"].double()).sum())

        for key, name in (("x", "dx"), ("z", "dz"), ("w", "dweight")):
            flat = d[key].double().flatten()
            for i in range(0, flat.numel(), 13):
                step = torch.zeros_like(flat)
                step[i] = 1e-5
                up, down = ((flat + s * step).view_as(d[key]) for s in (1, -1))
                diff = (loss(**{key: up}) - loss(**{key: down})) / 2e-5
                assert abs(float(got[name].flatten()[i]) - diff) <= 1e-4 * max(1.0, abs(diff))


def test_in_place_and_guard_bands(cuda_device):
    """residual_out on the residual itself, y on x itself, dx on dy; nothing outside is written."""
    d = _draw(33, 2560, torch.bfloat16, seed=3)
    y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, residual=d["residual"])
    buf = torch.full((3, 35, 2560), 7.0, dtype=torch.bfloat16, device=cuda_device)
    x, r, dy = buf[0, 1:34], buf[1, 1:34], buf[2, 1:34]
    x.copy_(d["x"])
    r.copy_(d["residual"])
    dy.copy_(d["dy"])
    w = d["w"].to(cuda_device)
    y, h = ssd.rms_norm(x, w, eps=EPS, residual=r, y=x, residual_out=r)
    assert torch.equal(r.cpu(), h_ref)
    assert ((x.cpu().double() - y_ref).abs() <= (2.0 ** -8 + F32) * y_ref.abs() + 1e-30).all()
    fresh = ssd.rms_norm_bwd(h, w, dy.clone(), eps=EPS)
    got = ssd.rms_norm_bwd(h, w, dy, eps=EPS, dx=dy)
    assert torch.equal(fresh["dx"], dy) and torch.equal(fresh["dweight"], got["dweight"])
    assert (buf[:, 0] == 7).all() and (buf[:, 34] == 7).all()


def test_empty_rows_and_streams(cuda_device):
    w = torch.ones(64, device=cuda_device)
    empty = torch.empty(0, 64, device=cuda_device)
    assert ssd.rms_norm(empty, w).shape == (0, 64)
    assert (ssd.rms_norm_bwd(empty, w, empty)["dweight"] == 0).all()
    x = torch.randn(4096, 64, device=cuda_device)
    want = ssd.rms_norm(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ssd.rms_norm(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_captured_calls_see_new_inputs(cuda_device):
    d = {k: v.to(cuda_device) for k, v in _draw(50, 2560, torch.bfloat16).items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ssd.rms_norm(d["x"], d["w"], residual=d["residual"], quant_group=128)
        ssd.rms_norm_bwd(d["x"], d["w"], d["dy"])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = ssd.rms_norm(d["x"], d["w"], residual=d["residual"], quant_group=128)
        grads = ssd.rms_norm_bwd(d["x"], d["w"], d["dy"])
    for seed in (1, 2):
        for k, v in _draw(50, 2560, torch.bfloat16, seed).items():
            d[k].copy_(v)
        graph.replay()
        want = ssd.rms_norm(d["x"], d["w"], residual=d["residual"], quant_group=128)
        wgrads = ssd.rms_norm_bwd(d["x"], d["w"], d["dy"])
        torch.cuda.synchronize()
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(out, want))
        assert all(torch.equal(grads[k], wgrads[k]) for k in grads)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", [1, 2, 15, 17, 63, 65, 130, 257, 513, 1537, 2049, 4097, 8191, 16383])
@pytest.mark.parametrize("offset", [0, 1, 2])
def test_rows_of_any_width_at_any_start(cuda_device, dim, dtype, offset):
    """Rows that are not whole 16-byte vectors, starting at any element, next to others: the values, and
    nothing written beside them (also in place)."""
    rows = 45
    if dim % (8 if dtype == torch.bfloat16 else 4) == 0:
        pytest.skip("whole vectors")
    d = _draw(rows, dim, dtype, seed=dim + offset)

    def placed(t, fill=None):
        buf = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device=cuda_device)
        view = buf[offset:offset + t.numel()].view(t.shape)
        if fill is None:
            view.copy_(t)
        return buf, view

    def clean(buf, n):
        return bool((buf[:offset].float() == 7).all() and (buf[offset + n:].float() == 7).all())

    n = rows * dim
    c = {k: placed(d[k])[1] for k in ("x", "residual", "z", "dy")}
    w = d["w"].to(cuda_device)
    xb, x = placed(d["x"])
    rb, r = placed(d["residual"])
    y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, residual=d["residual"])
    ssd.rms_norm(x, w, eps=EPS, residual=r, y=x, residual_out=r)
    tol = STEP[dtype] + F32
    assert ((x.double().cpu() - y_ref).abs() <= tol * y_ref.abs() + F32 * y_ref.abs().max()).all()
    assert torch.equal(r.cpu(), h_ref) and clean(xb, n) and clean(rb, n)
    y8b, y8 = placed(torch.zeros(rows, dim).to(torch.float8_e4m3fn))
    y8, scales = ssd.rms_norm(c["x"], w, eps=EPS, z=c["z"], gate="pre", quant_group=dim, y=y8)
    y_ref, _ = ref.rms_norm(d["x"], d["w"], EPS, z=d["z"], gate="pre")
    got = y8.float().double().cpu() * scales.double().cpu()
    s_ref = (y_ref.abs().amax(-1, keepdim=True) / 448).clamp_min(1e-30)
    assert ((got - y_ref).abs() <= (2.0 ** -4 + 4 * F32) * y_ref.abs() + (2.0 ** -10 + F32) * s_ref).all()
    assert clean(y8b, n)
    dx, dw, dz = _grads(d, EPS, "post", False)
    gb, g = placed(d["dy"])
    zb, gz = placed(d["z"])
    out = ssd.rms_norm_bwd(c["x"], w, g, eps=EPS, z=c["z"], gate="post", dx=g, dz=gz)
    # dx is the difference of r dn w and h r^3 sum(dn w h) / dim, neither longer than r |dn w| (for the
    # second: |h|^2 r^2 / dim <= 1); dz is dy n w times silu's slope, itself a sum of two terms below 1.1.
    # Both are held to float32's error in the terms, and to the storage type's in the result.
    x64, w64, dy64, z64 = (d[k].double() for k in ("x", "w", "dy", "z"))
    r = torch.rsqrt((x64 * x64).mean(-1, keepdim=True) + EPS)
    terms = (r * (dy64 * ref.silu(z64) * w64).norm(dim=-1, keepdim=True),
             (dy64 * x64 * r * w64).norm(dim=-1, keepdim=True))
    for got, want, size in ((out["dx"], dx, terms[0]), (out["dz"], dz, terms[1])):
        err = (got.double().cpu() - want).norm(dim=-1, keepdim=True)
        assert (err <= (STEP[dtype] + 2 * F32) * want.norm(dim=-1, keepdim=True) + 4 * F32 * size).all()
    assert ref.rel(out["dweight"], dw) <= 256 * 2.0 ** -24 * 8
    assert clean(gb, n) and clean(zb, n)
