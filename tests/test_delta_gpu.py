"""GPU parity of the gated delta rule against the float64 token recurrence.

Tolerances (2-norm of the difference over the 2-norm of the reference, per output).  The float32
recurrence: every token adds a few roundings of 2^-24 to the state and a sum of N products
(at most 8 sequential additions and 5 folds); with keys of norm 1 and beta below 1 the state does
not grow, so the errors add up no worse than one by one over the tokens that it remembers:
(L + 32) * 2^-24 * 4.  The chunked kernels hold every factor that is not a bf16 input as two bf16
parts, which leaves 2^-16 of it, for the state, the residual and the triangular inverse: 2^-16 * 4
with the same memory.  A bf16 output adds its rounding, 2^-8, and in the chunked kernels the bf16
parts that the output alone takes: the state and the products with it, 2 * 2^-8.
"""
import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def state_tol(dtype, L):
    return 4 * (L + 32) * 2.0 ** -24 + (4 * 2.0 ** -16 if dtype == BF else 0.0)


def out_tol(dtype, L):
    return state_tol(dtype, L) + (3 * 2.0 ** -8 if dtype == BF else 0.0)


def to(d, device):
    return {k: None if v is None else v.to(device) for k, v in d.items()}


def args(d):
    return [d[n] for n in ("q", "k", "v", "g", "beta")]


CASES = [
    # (b, L, H, G, P, N, dtype, l2norm, init, decay)
    (1, 1, 1, 1, 64, 128, BF, False, True, "mixed"),
    (2, 2, 4, 2, 64, 128, BF, True, False, "mixed"),
    (1, 31, 4, 1, 64, 128, BF, False, True, "mixed"),
    (2, 32, 4, 1, 64, 128, BF, True, True, "mixed"),
    (1, 33, 6, 2, 64, 64, BF, False, True, "mixed"),
    (2, 64, 4, 4, 128, 128, BF, True, True, "mixed"),
    (1, 65, 3, 1, 128, 64, BF, True, True, "strong"),
    (1, 127, 5, 1, 64, 128, BF, True, True, None),
    (2, 300, 8, 2, 64, 128, BF, True, True, "mixed"),
    (1, 300, 4, 2, 48, 128, BF, True, True, "mixed"),       # rows of three tiles of 16
    (1, 300, 4, 2, 16, 64, BF, False, True, "mixed"),
    (1, 200, 4, 2, 112, 128, BF, True, True, "mixed"),
    (1, 300, 4, 2, 20, 128, BF, True, True, "mixed"),       # rows of no whole tile
    (1, 100, 2, 1, 64, 32, BF, True, True, "mixed"),
    (1, 100, 2, 1, 64, 256, BF, True, True, "mixed"),
    (3, 700, 2, 1, 64, 128, BF, False, True, "strong"),
    (1, 1500, 4, 1, 64, 128, BF, True, False, "mixed"),
    (2, 1, 3, 3, 5, 32, F32, True, True, "mixed"),
    (1, 90, 4, 2, 64, 128, F32, True, True, "mixed"),
    (1, 200, 6, 2, 128, 128, F32, False, True, "strong"),
    (2, 64, 2, 1, 33, 256, F32, True, True, None),
    (1, 64, 2, 2, 1, 64, F32, True, False, "mixed"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).split(".")[-1] for x in c))
def test_forward(cuda_device, case):
    b, L, H, G, P, N, dtype, l2norm, init, decay = case
    d = ref.draw(b, L, H, G, P, N, dtype, seed=L + P, unit=not l2norm, decay=decay, init=init)
    scale = N ** -0.5
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], scale, l2norm)
    c = to(d, cuda_device)
    o, s = ssd.delta_rule_fwd(*args(c), init_state=c["init"], qk_l2norm=l2norm)
    assert o.dtype == dtype and s.dtype == F32
    assert ref.rel(s, s_ref) <= state_tol(dtype, L)
    assert ref.rel(o, o_ref) <= out_tol(dtype, L)
    o2, s2 = ssd.delta_rule_fwd(*args(c), init_state=c["init"], qk_l2norm=l2norm)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    o3, none = ssd.delta_rule_fwd(*args(c), init_state=c["init"], qk_l2norm=l2norm,
                                  return_final_state=False)
    assert none is None and torch.equal(o, o3)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_split_resume_and_steps_continue_a_sequence(cuda_device, dtype):
    """The whole sequence = its first part, its second part from the kept state, then one token
    at a time."""
    b, L, H, G, P, N = 2, 230, 4, 2, 64, 128
    d = to(ref.draw(b, L, H, G, P, N, dtype, seed=5, unit=False), cuda_device)
    cut = lambda x, a, e: x[:, a:e].contiguous()
    whole, s_whole = ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=True)
    state = d["init"].clone()
    parts = []
    for a, e in ((0, 77), (77, 200)):
        o, state = ssd.delta_rule_fwd(*(cut(x, a, e) for x in args(d)), init_state=state,
                                      qk_l2norm=True, final_state=state)
        parts.append(o)
    for t in range(200, L):
        parts.append(ssd.delta_rule_update(state, *(x[:, t].contiguous() for x in args(d)),
                                           qk_l2norm=True)[:, None])
    assert ref.rel(torch.cat(parts, 1), whole.cpu()) <= 2 * out_tol(dtype, L)
    assert ref.rel(state, s_whole.cpu()) <= 2 * state_tol(dtype, L)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("b,H,G,P,N,l2norm", [(1, 24, 1, 64, 128, True), (3, 8, 8, 128, 128, False),
                                              (37, 6, 2, 64, 64, True), (2, 4, 2, 33, 32, True),
                                              (1, 2, 1, 64, 256, True), (5, 3, 1, 1, 128, True)])
def test_update(cuda_device, b, H, G, P, N, l2norm, dtype):
    """Several tokens, every output against float64, from a state larger than the values."""
    d = ref.draw(b, 5, H, G, P, N, dtype, seed=b + P, unit=not l2norm)
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], 0.5, l2norm)
    c = to(d, cuda_device)
    state = c["init"]
    o = [ssd.delta_rule_update(state, *(x[:, t].contiguous() for x in args(c)), scale=0.5,
                               qk_l2norm=l2norm) for t in range(5)]
    assert ref.rel(state, s_ref) <= 4 * 37 * 2.0 ** -24
    assert ref.rel(torch.stack(o, 1), o_ref) <= \
        4 * 37 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF else 0)


def test_beta_of_zero_and_one_and_rows_without_a_key(cuda_device):
    """beta 0: the token writes nothing; beta 1 with a key of norm 1: the state then gives back
    exactly v; a key of zeros (also under the norm) writes nothing."""
    for L, P in ((40, 64), (40, 20)):
        d = ref.draw(1, L, 2, 1, P, 128, BF, seed=2, unit=False)
        d["beta"][:, ::3] = 0.0
        d["beta"][:, 1::3] = 1.0
        d["k"][:, 5:9] = 0
        d["q"][:, 7] = 0
        c = to(d, cuda_device)
        o_ref, s_ref = ref.delta_rule(*args(d), d["init"], 128 ** -0.5, True)
        o, s = ssd.delta_rule_fwd(*args(c), init_state=c["init"], qk_l2norm=True)
        assert ref.rel(s, s_ref) <= state_tol(BF, L) and ref.rel(o, o_ref) <= out_tol(BF, L)
        assert (o[:, 7] == 0).all()


def test_keys_that_repeat(cuda_device):
    """One key for every token, beta near 1: the triangular system at its worst."""
    d = ref.draw(1, 200, 2, 1, 64, 128, BF, seed=4, unit=False, decay=None)
    d["k"][:] = d["k"][:, :1]
    d["beta"] = 0.9 + 0.1 * d["beta"]
    c = to(d, cuda_device)
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], 128 ** -0.5, True)
    o, s = ssd.delta_rule_fwd(*args(c), init_state=c["init"], qk_l2norm=True)
    assert ref.rel(s, s_ref) <= state_tol(BF, 200) and ref.rel(o, o_ref) <= out_tol(BF, 200)


PACKS = [
    [0, 1], [0, 40], [0, 32, 64], [0, 0, 5, 5, 70, 71, 200], [0, 31, 31, 64, 97, 300],
    [0, 500, 500], [0, 0],
]


@pytest.mark.parametrize("dtype,P", [(BF, 64), (BF, 48), (BF, 20), (F32, 64)])
@pytest.mark.parametrize("cu", PACKS, ids=lambda c: "-".join(map(str, c)))
def test_varlen(cuda_device, cu, dtype, P):
    """Each packed sequence against the recurrence on it alone; empty ones keep their state."""
    L, nseq, H, G, N = cu[-1], len(cu) - 1, 4, 2, 128
    d = ref.draw(1, L, H, G, P, N, dtype, seed=len(cu) + P, unit=False, nseq=nseq)
    c = to(d, cuda_device)
    cut = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    o, s = ssd.delta_rule_varlen_fwd(*args(c), cut, init_states=c["init"], qk_l2norm=True)
    o0, s0 = ssd.delta_rule_varlen_fwd(*args(c), cut, qk_l2norm=True)
    for i, (a, e) in enumerate(zip(cu, cu[1:])):
        part = [x[:, a:e] for x in args(d)]
        if a == e:
            assert torch.equal(s[i].cpu(), d["init"][i]) and (s0[i] == 0).all()
            continue
        o_ref, s_ref = ref.delta_rule(*part, d["init"][i:i + 1], N ** -0.5, True)
        assert ref.rel(s[i:i + 1], s_ref) <= state_tol(dtype, L)
        assert ref.rel(o[:, a:e], o_ref) <= out_tol(dtype, L)
        o_ref, s_ref = ref.delta_rule(*part, None, N ** -0.5, True)
        assert ref.rel(s0[i:i + 1], s_ref) <= state_tol(dtype, L)
        assert ref.rel(o0[:, a:e], o_ref) <= out_tol(dtype, L)


@pytest.mark.parametrize("P", [64, 20])
def test_varlen_inconsistent_offsets_compute_nothing(cuda_device, P):
    d = to(ref.draw(1, 100, 2, 1, P, 128, BF, nseq=2), cuda_device)
    shape = ssd.make_shape(1, 100, 2, P, 128, 1, ssd.SSD_BF16)
    import ctypes
    ws = torch.empty(ssd.lib().ssd_delta_rule_varlen_workspace_size(ctypes.byref(shape), 2),
                     dtype=torch.uint8, device=cuda_device)
    for cu in ([0, 60, 99], [1, 60, 100], [0, 101, 100], [0, -4, 100]):
        o = torch.full_like(d["v"], 3.0)
        s = torch.full_like(d["init"], 3.0)
        ssd.delta_rule_varlen_fwd(*args(d), torch.tensor(cu, dtype=torch.int32,
                                                         device=cuda_device),
                                  init_states=d["init"], o=o, final_states=s, workspace=ws)
        assert ssd.workspace_status(ws) == ssd.SSD_ERR_INVALID_ARG
        assert (o == 3).all() and (s == 3).all()


def test_empty_batch_and_empty_sequence(cuda_device):
    d = to(ref.draw(2, 0, 4, 2, 64, 128, BF), cuda_device)
    o, s = ssd.delta_rule_fwd(*args(d), init_state=d["init"])
    assert o.shape == (2, 0, 4, 64) and torch.equal(s, d["init"])
    _, s = ssd.delta_rule_fwd(*args(d))
    assert (s == 0).all()
    d = to(ref.draw(0, 5, 4, 2, 64, 128, BF, init=False), cuda_device)
    o, s = ssd.delta_rule_fwd(*args(d))
    assert o.shape == (0, 5, 4, 64) and s.shape == (0, 4, 64, 128)


@pytest.mark.parametrize("L,P", [(70, 64), (70, 20), (1, 64)])
def test_guard_bands_and_aliased_states(cuda_device, L, P):
    """o, the final state and the workspace are written where they are and nowhere else; the final
    state may be the initial one."""
    d = to(ref.draw(2, L, 4, 2, P, 128, BF, seed=8), cuda_device)
    want_o, want_s = ssd.delta_rule_fwd(*args(d), init_state=d["init"])
    n = d["v"].numel()
    ob = torch.full((n + 256,), 5.0, dtype=BF, device=cuda_device)
    sb = torch.full((d["init"].numel() + 256,), 5.0, device=cuda_device)
    o, s = ob[128:128 + n].view_as(d["v"]), sb[128:-128].view_as(d["init"])
    s.copy_(d["init"])
    size = ssd.delta_rule_workspace_size(ssd.make_shape(2, L, 4, P, 128, 2, ssd.SSD_BF16))
    wb = torch.full((size + 512,), 9, dtype=torch.uint8, device=cuda_device)
    ssd.delta_rule_fwd(*args(d), init_state=s, o=o, final_state=s, workspace=wb[256:-256])
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    assert (ob[:128] == 5).all() and (ob[128 + n:] == 5).all()
    assert (sb[:128] == 5).all() and (sb[-128:] == 5).all()
    assert (wb[:256] == 9).all() and (wb[-256:] == 9).all()


def test_streams_and_captured_calls(cuda_device):
    """Two streams at once with workspaces of their own, and a captured call that is replayed on
    new inputs."""
    a = to(ref.draw(2, 300, 8, 2, 64, 128, BF, seed=1, unit=False), cuda_device)
    b = to(ref.draw(2, 300, 8, 2, 64, 128, BF, seed=2, unit=False), cuda_device)
    run = lambda d, **kw: ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=True, **kw)
    want = [run(a), run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [run(d, stream=s) for d, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    graph = torch.cuda.CUDAGraph()
    state = a["init"][:, :, :, :].clone()
    step = [x[:, 0].contiguous() for x in args(a)]
    with torch.cuda.graph(graph, stream=streams[0]):
        o, s = run(a)
        y = ssd.delta_rule_update(state, *step, qk_l2norm=True)
    for k in ("q", "k", "v", "g", "beta", "init"):
        a[k].copy_(b[k])
    state.copy_(b["init"])
    for x, n in zip(step, args(b)):
        x.copy_(n[:, 0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[1][0]) and torch.equal(s, want[1][1])
    fresh = b["init"].clone()
    assert torch.equal(y, ssd.delta_rule_update(fresh, *step, qk_l2norm=True))
    assert torch.equal(state, fresh)
