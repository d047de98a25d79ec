"""Refusals of the gated delta rule's and the RMS norm's entry points, before anything is launched
(no GPU needed)."""
import ctypes

import pytest
import torch

from mamba_ssd_layer_scan_b200 import build, ssd


@pytest.fixture(scope="module")
def L():
    build.build()
    return ssd.lib()


OK = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


def shape(**kw):
    d = dict(batch=2, seqlen=100, nheads=8, headdim=64, dstate=128, ngroups=2, dtype=ssd.SSD_BF16)
    return ssd.make_shape(**(d | kw))


def fwd(L, sh, options=ssd.DeltaOptions(0.1, 1), **kw):
    p = dict(q=OK, k=OK, v=OK, g=OK, beta=OK, init=None, o=OK, final=None, ws=OK, bytes=BIG) | kw
    return L.ssd_delta_rule_fwd(ctypes.byref(sh), p["q"], p["k"], p["v"], p["g"], p["beta"],
                                ctypes.byref(options) if options else None, p["init"], p["o"],
                                p["final"], p["ws"], p["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ngroups=3), ssd.SSD_ERR_INVALID_ARG),
    (dict(batch=-1), ssd.SSD_ERR_INVALID_ARG),
    (dict(seqlen=-1), ssd.SSD_ERR_INVALID_ARG),
    (dict(dtype=5), ssd.SSD_ERR_INVALID_ARG),
    (dict(headdim=129), ssd.SSD_ERR_UNSUPPORTED),
    (dict(headdim=0), ssd.SSD_ERR_UNSUPPORTED),
    (dict(dstate=96), ssd.SSD_ERR_UNSUPPORTED),
    (dict(dstate=256, headdim=128), ssd.SSD_ERR_UNSUPPORTED),
])
def test_delta_bad_shapes(L, kw, code):
    sh = shape(**kw)
    assert fwd(L, sh) == code and ssd.last_error()
    assert L.ssd_delta_rule_workspace_size(ctypes.byref(sh)) == 0
    if "seqlen" not in kw:
        assert L.ssd_delta_rule_update(ctypes.byref(sh), OK, OK, OK, OK, OK, OK,
                                       ctypes.byref(ssd.DeltaOptions(1.0, 0)), OK, None) == code


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(beta=None),
                                dict(o=None), dict(ws=None), dict(q=MIS), dict(k=MIS), dict(v=MIS),
                                dict(o=MIS), dict(init=MIS), dict(final=MIS),
                                dict(ws=ctypes.c_void_p((1 << 20) + 128)), dict(bytes=16),
                                dict(options=None), dict(options=ssd.DeltaOptions(0.1, 2))])
def test_delta_bad_pointers_and_options(L, kw):
    assert fwd(L, shape(), **kw) == ssd.SSD_ERR_INVALID_ARG and ssd.last_error()


def test_delta_empty_is_valid(L):
    none = dict(q=None, k=None, v=None, beta=None, o=None, ws=None, bytes=0)
    assert fwd(L, shape(batch=0), **none) == ssd.SSD_OK
    assert fwd(L, shape(seqlen=0), **none) == ssd.SSD_OK


@pytest.mark.parametrize("kw,nseq,code", [(dict(batch=2), 3, ssd.SSD_ERR_INVALID_ARG),
                                          (dict(batch=1), 0, ssd.SSD_ERR_INVALID_ARG),
                                          (dict(batch=1, dstate=96), 2, ssd.SSD_ERR_UNSUPPORTED)])
def test_delta_varlen_refusals(L, kw, nseq, code):
    sh = shape(**kw)
    assert L.ssd_delta_rule_varlen_workspace_size(ctypes.byref(sh), nseq) == 0
    o = ssd.DeltaOptions(0.1, 1)
    call = lambda s, n, cu=OK, size=BIG: L.ssd_delta_rule_varlen_fwd(
        ctypes.byref(s), OK, OK, OK, OK, OK, ctypes.byref(o), cu, n, None, OK, None, OK, size, None)
    assert call(sh, nseq) == code
    assert call(shape(batch=1), 2, cu=None) == ssd.SSD_ERR_INVALID_ARG
    assert call(shape(batch=1), 2, size=100) == ssd.SSD_ERR_INVALID_ARG


def test_delta_update_refusals(L):
    o = ssd.DeltaOptions(0.1, 1)
    sh = shape()
    for i in range(8):
        if i == 4:
            continue   # g may be NULL
        p = [OK] * 8
        p[i] = None
        state, q, k, v, g, beta, _, out = p
        rc = L.ssd_delta_rule_update(ctypes.byref(sh), state, q, k, v, g, beta,
                                     ctypes.byref(o) if p[6] else None, out, None)
        assert rc == ssd.SSD_ERR_INVALID_ARG and ssd.last_error()
    assert L.ssd_delta_rule_update(ctypes.byref(sh), MIS, OK, OK, OK, OK, OK, ctypes.byref(o), OK,
                                   None) == ssd.SSD_ERR_INVALID_ARG


def norm(L, desc, **kw):
    p = dict(x=OK, residual=None, z=None, w=OK, y=OK, scales=None, out=None) | kw
    return L.ssd_rms_norm(ctypes.byref(desc), p["x"], p["residual"], p["z"], p["w"], p["y"],
                          p["scales"], p["out"], None)


def desc(rows=10, dim=256, dtype=ssd.SSD_BF16, gate=0, quant=0, eps=1e-5):
    return ssd.NormDesc(rows, dim, dtype, gate, quant, eps)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), ssd.SSD_ERR_INVALID_ARG), (dict(dim=0), ssd.SSD_ERR_UNSUPPORTED),
    (dict(dim=16385), ssd.SSD_ERR_UNSUPPORTED), (dict(dtype=3), ssd.SSD_ERR_INVALID_ARG),
    (dict(gate=3), ssd.SSD_ERR_INVALID_ARG), (dict(eps=-1.0), ssd.SSD_ERR_INVALID_ARG),
    (dict(eps=float("nan")), ssd.SSD_ERR_INVALID_ARG), (dict(quant=48), ssd.SSD_ERR_UNSUPPORTED),
    (dict(quant=-128), ssd.SSD_ERR_UNSUPPORTED), (dict(dim=192, quant=128),
                                                  ssd.SSD_ERR_UNSUPPORTED),
])
def test_norm_bad_descriptions(L, kw, code):
    d = desc(**kw)
    assert norm(L, d, scales=OK, z=OK if d.gate else None) == code and ssd.last_error()
    assert L.ssd_rms_norm_bwd_workspace_size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("d,kw,code", [
    (desc(), dict(x=None), ssd.SSD_ERR_INVALID_ARG), (desc(), dict(w=None), ssd.SSD_ERR_INVALID_ARG),
    (desc(), dict(y=None), ssd.SSD_ERR_INVALID_ARG),
    (desc(quant=128), dict(), ssd.SSD_ERR_INVALID_ARG),            # no scales
    (desc(), dict(residual=OK), ssd.SSD_ERR_INVALID_ARG),          # no residual_out
    (desc(), dict(out=OK), ssd.SSD_ERR_INVALID_ARG),
    (desc(), dict(z=OK), ssd.SSD_ERR_INVALID_ARG),                 # z without a gate
    (desc(gate=1), dict(), ssd.SSD_ERR_INVALID_ARG),               # a gate without z
    (desc(gate=1), dict(z=OK, residual=OK, out=OK), ssd.SSD_ERR_UNSUPPORTED),
    (desc(), dict(x=MIS), ssd.SSD_ERR_INVALID_ARG), (desc(), dict(y=MIS), ssd.SSD_ERR_INVALID_ARG),
    (desc(), dict(w=MIS), ssd.SSD_ERR_INVALID_ARG),
    (desc(dim=255), dict(x=ctypes.c_void_p(3)), ssd.SSD_ERR_INVALID_ARG),
])
def test_norm_bad_pointers(L, d, kw, code):
    assert norm(L, d, **kw) == code and ssd.last_error()


def test_norm_bwd_refusals(L):
    def bwd(d, **kw):
        p = dict(x=OK, z=None, w=OK, dy=OK, dres=None, dx=OK, dz=None, dw=OK, ws=OK, n=BIG) | kw
        return L.ssd_rms_norm_bwd(ctypes.byref(d), p["x"], p["z"], p["w"], p["dy"], p["dres"],
                                  p["dx"], p["dz"], p["dw"], p["ws"], p["n"], None)
    for kw in (dict(x=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None),
               dict(ws=None), dict(n=100), dict(x=MIS), dict(dx=MIS), dict(z=OK), dict(dz=OK),
               dict(ws=ctypes.c_void_p((1 << 20) + 64))):
        assert bwd(desc(), **kw) == ssd.SSD_ERR_INVALID_ARG and ssd.last_error()
    assert bwd(desc(gate=1), z=OK) == ssd.SSD_ERR_INVALID_ARG
    assert bwd(desc(gate=1), z=OK, dz=OK, dres=OK) == ssd.SSD_ERR_UNSUPPORTED
    assert bwd(desc(quant=256)) == ssd.SSD_ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors_shapes_types_and_strides(L):
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    f = lambda *s: t(*s, dtype=torch.float32)
    good = dict(q=t(2, 5, 2, 64), k=t(2, 5, 2, 64), v=t(2, 5, 4, 32), g=f(2, 5, 4), beta=f(2, 5, 4))
    bad = [dict(q=t(2, 5, 2, 32)), dict(k=t(2, 4, 2, 64)), dict(q=f(2, 5, 2, 64)),
           dict(g=t(2, 5, 4)), dict(beta=f(2, 5, 3)), dict(v=t(2, 4, 5, 32).transpose(1, 2)),
           dict(v=t(2, 5, 128)), dict(init_state=f(2, 4, 32, 32)),
           dict(init_state=t(2, 4, 32, 64)), dict(o=t(2, 5, 4, 16))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            ssd.delta_rule_fwd(**(good | kw))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_fwd(**good)
    half = {k: v.half() if v.dtype == torch.bfloat16 else v for k, v in good.items()}
    with pytest.raises(TypeError):
        ssd.delta_rule_fwd(**half)
    step = {k: v[:, 0].contiguous() for k, v in good.items()}
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_update(f(2, 4, 32, 64), **step)
    with pytest.raises(ValueError, match="state"):
        ssd.delta_rule_update(f(2, 4, 64, 32), **step)
    packed = {k: v[:1] for k, v in good.items()}
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.delta_rule_varlen_fwd(**packed, cu_seqlens=cu)
    with pytest.raises(TypeError):
        ssd.delta_rule_varlen_fwd(**packed, cu_seqlens=cu.long())
    with pytest.raises(ValueError):
        ssd.delta_rule_varlen_fwd(**packed, cu_seqlens=cu, init_states=f(1, 4, 32, 64))
    x, w = t(4, 64), f(64)
    for kw in (dict(weight=t(64)), dict(weight=f(32)), dict(residual=t(4, 32)), dict(z=x),
               dict(gate="pre"), dict(gate="swish", z=x), dict(quant_group=48),
               dict(quant_group=-64), dict(residual_out=x), dict(residual=f(4, 64)),
               dict(x=t(64, 4).t())):
        with pytest.raises((ValueError, TypeError)):
            ssd.rms_norm(**(dict(x=x, weight=w) | kw))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.rms_norm_bwd(x, w, x)
    with pytest.raises(ValueError):
        ssd.rms_norm_bwd(x, w, x, dz=x)
