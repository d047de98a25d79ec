"""The RMS norm of so many rows that every CTA takes several steps: its ring of rows is used again and
again, or the next row's registers, whatever the width; against float64 on the GPU, row by row.

Tolerances per row as for few rows: the result's rounding (2^-8 or 2^-24 of the value) and 128 * 2^-24
of float32's arithmetic; e4m3 half a step, 2^-4 of the value, or 2^-10 of the scale below its normal
range.  dx and dz are held to twice that of the value and 512 * 2^-24 of the terms that they are the
difference of.  dweight: a column's sum over the rows takes at most steps + 64 additions one after the
other, each off by 2^-24 of the sum of the absolute values, and its terms 64 * 2^-24.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

F32 = 128 * 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-5
BF = torch.bfloat16

# (rows, dim, first element): rows for seven steps and more of 148 SMs full of CTAs.  Whole 16-byte
# vectors on 8, 16 and 32 lanes and on a CTA with 1, 2, 4 and (float32) 8 of them a thread; pairs with the
# next row in registers and without, of even and odd width; single elements, at an odd start
SIZES = [(300000, 64, 0), (150000, 128, 0), (70000, 256, 0), (16000, 2560, 0), (9000, 4096, 0),
         (5000, 8192, 0), (2500, 16384, 0),
         (300000, 13, 0), (70000, 57, 0), (70000, 130, 0), (70001, 255, 0), (16000, 1537, 0),
         (9000, 2050, 0), (4000, 8191, 0), (2000, 16383, 0),
         (70000, 130, 1), (9000, 1537, 1), (2500, 8191, 1)]


def draw(rows, dim, first, dtype, device):
    gen = torch.Generator(device=device).manual_seed(rows + dim)

    def n(scale=1.0):
        flat = torch.empty(rows * dim + 8, dtype=dtype, device=device)
        t = flat[first:first + rows * dim].view(rows, dim)
        return t.copy_(scale * torch.randn(rows, dim, generator=gen, device=device))

    return dict(x=n(), residual=n(2.0), z=n(), dy=n(),
                w=1 + 0.3 * torch.randn(dim, generator=gen, device=device))


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,dim,first", SIZES)
def test_forward(cuda_device, rows, dim, first, dtype):
    d = draw(rows, dim, first, dtype, cuda_device)
    for mode in ("residual", "pre", "post", "plain"):
        kw = {}
        if mode == "residual":
            kw = dict(residual=d["residual"])
        elif mode != "plain":
            kw = dict(z=d["z"], gate=mode)
        y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, **kw)
        out = ssd.rms_norm(d["x"], d["w"], eps=EPS, **kw)
        y = out
        if mode == "residual":
            y, h = out
            assert torch.equal(h, h_ref)
        assert ((y.double() - y_ref).abs() <= (STEP[dtype] + F32) * y_ref.abs() + 1e-30).all(), mode
    # in place, the sum on the residual: the next rows are on their way while these are written
    y_ref, h_ref = ref.rms_norm(d["x"], d["w"], EPS, residual=d["residual"])
    ssd.rms_norm(d["x"], d["w"], eps=EPS, residual=d["residual"], y=d["x"], residual_out=d["residual"])
    assert torch.equal(d["residual"], h_ref)
    assert ((d["x"].double() - y_ref).abs() <= (STEP[dtype] + F32) * y_ref.abs() + 1e-30).all()


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,dim,first,group", [
    (300000, 64, 0, 64), (150000, 128, 0, 32), (70000, 256, 0, 128), (16000, 2560, 0, 2560),
    (9000, 4096, 0, 128), (4000, 8192, 0, 8192), (70001, 255, 0, 255), (9000, 1537, 1, 1537)])
def test_forward_e4m3(cuda_device, rows, dim, first, group, dtype):
    d = draw(rows, dim, first, dtype, cuda_device)
    for kw in (dict(residual=d["residual"]), dict(z=d["z"], gate="pre")):
        y_ref, _ = ref.rms_norm(d["x"], d["w"], EPS, **kw)
        y8, scales = ssd.rms_norm(d["x"], d["w"], eps=EPS, quant_group=group, **kw)[:2]
        groups = y_ref.view(rows, -1, group)
        s_ref = (groups.abs().amax(-1) / 448).clamp_min(1e-30)
        assert ((scales.double() - s_ref).abs() <= F32 * s_ref).all()
        got = y8.float().double().view_as(groups) * scales.double()[..., None]
        bound = (2.0 ** -4 + 4 * F32) * groups.abs() + (2.0 ** -10 + F32) * s_ref[..., None]
        assert ((got - groups).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,dim,first", SIZES)
def test_backward(cuda_device, rows, dim, first, dtype):
    d = draw(rows, dim, first, dtype, cuda_device)
    x, z, w, dy = (d[k].double() for k in ("x", "z", "w", "dy"))
    steps = rows // 608 + 1
    for mode in ("residual", "pre", "post", "plain"):
        gated = mode in ("pre", "post")
        kw = dict(z=d["z"], gate=mode) if gated else {}
        if mode == "residual":
            kw["dresidual"] = d["residual"]
        got = ssd.rms_norm_bwd(d["x"], d["w"], d["dy"], eps=EPS, **kw)
        silu = ref.silu(z) if gated else None
        h = x * silu if mode == "pre" else x
        dn = dy * silu if mode == "post" else dy
        r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        n = h * r
        dh = r * (dn * w - n * (n * dn * w).mean(-1, keepdim=True))
        size = (r * dn * w).norm(dim=-1, keepdim=True)
        sig = torch.sigmoid(z)
        slope = sig * (1 + z * (1 - sig))
        want = {"dx": (dh * silu if mode == "pre" else dh + d["residual"].double()
                       if mode == "residual" else dh, size)}
        if mode == "post":
            want["dz"] = (dy * n * w * slope, (dy * n * w).norm(dim=-1, keepdim=True))
        if mode == "pre":   # silu and its slope stay below |z| + 1.1
            most = z.abs().amax(-1, keepdim=True) + 1.1
            want["dx"] = (want["dx"][0], size * most)
            want["dz"] = (dh * x * slope, 1.1 * size * x.abs().amax(-1, keepdim=True))
        for name, (v, terms) in want.items():
            err = (got[name].double() - v).norm(dim=-1, keepdim=True)
            bound = (STEP[dtype] + 2 * F32) * v.norm(dim=-1, keepdim=True) + 4 * F32 * terms
            assert (err <= bound).all(), (mode, name)
        err = (got["dweight"].double() - (dn * n).sum(0)).abs()
        assert (err <= (steps + 128) * 2.0 ** -24 * (dn * n).abs().sum(0)).all(), mode
