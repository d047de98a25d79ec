"""GPU parity of the gated delta rule's tcgen05 kernels, which take over with many heads and more than
64 tokens a sequence, against the float64 token recurrence.

Tolerances as for the warp-level chunked kernels: every factor that is not a bf16 input is held as two
bf16 parts (2^-16 of it is left) for the state, the residual and the triangular inverse, 2^-16 * 4
over the tokens that the state remembers, plus the float32 sums, 4 (L + 32) * 2^-24.  The output adds
its rounding, 2^-8, and the bf16 parts that it alone takes -- the state, W, and the triangle they are
multiplied with -- 2 * 2^-8.
"""
import ctypes

import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

import _delta_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def state_tol(L):
    return 4 * (L + 32) * 2.0 ** -24 + 4 * 2.0 ** -16


def out_tol(L):
    return state_tol(L) + 3 * 2.0 ** -8


def to(d, device):
    return {k: None if v is None else v.to(device) for k, v in d.items()}


def args(d):
    return [d[n] for n in ("q", "k", "v", "g", "beta")]


CASES = [
    # (b, L, H, G, P, N, l2norm, init, decay)
    (1, 65, 40, 1, 64, 128, True, True, "mixed"),
    (1, 128, 40, 2, 64, 64, False, True, "mixed"),
    (2, 129, 21, 7, 64, 128, True, False, "mixed"),      # three heads to a group: one without a partner
    (3, 100, 13, 13, 64, 64, True, True, None),          # one head to a group
    (1, 200, 20, 2, 128, 128, True, True, "mixed"),
    (2, 257, 10, 5, 128, 64, False, True, "strong"),
    (1, 1000, 38, 1, 64, 128, True, True, "strong"),
    (1, 511, 19, 1, 128, 128, True, False, "mixed"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_forward(cuda_device, case):
    b, L, H, G, P, N, l2norm, init, decay = case
    d = ref.draw(b, L, H, G, P, N, BF, seed=L + P, unit=not l2norm, decay=decay, init=init)
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], 0.3, l2norm)
    c = to(d, cuda_device)
    kw = dict(scale=0.3, init_state=c["init"], qk_l2norm=l2norm)
    o, s = ssd.delta_rule_fwd(*args(c), **kw)
    assert ref.rel(s, s_ref) <= state_tol(L)
    assert ref.rel(o, o_ref) <= out_tol(L)
    for h in range(H):   # no head hides behind the others
        assert ref.rel(s[:, h], s_ref[:, h]) <= 4 * state_tol(L)
        assert ref.rel(o[:, :, h], o_ref[:, :, h]) <= 4 * out_tol(L)
    o2, s2 = ssd.delta_rule_fwd(*args(c), **kw)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    o3, none = ssd.delta_rule_fwd(*args(c), return_final_state=False, **kw)
    assert none is None and torch.equal(o, o3)


@pytest.mark.parametrize("P,H", [(64, 24), (128, 12)])
@pytest.mark.parametrize("cu", [[0, 70, 200], [0, 0, 64, 64, 193, 194, 500], [0, 300, 300, 363, 428]],
                         ids=lambda c: "-".join(map(str, c)))
def test_varlen(cuda_device, cu, P, H):
    """Each packed sequence against the recurrence on it alone; empty ones keep their state."""
    L, nseq, G, N = cu[-1], len(cu) - 1, 2, 128
    d = ref.draw(1, L, H, G, P, N, BF, seed=len(cu) + P, unit=False, nseq=nseq)
    c = to(d, cuda_device)
    cut = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    o, s = ssd.delta_rule_varlen_fwd(*args(c), cut, init_states=c["init"], qk_l2norm=True)
    o0, s0 = ssd.delta_rule_varlen_fwd(*args(c), cut, qk_l2norm=True)
    for i, (a, e) in enumerate(zip(cu, cu[1:])):
        if a == e:
            assert torch.equal(s[i].cpu(), d["init"][i]) and (s0[i] == 0).all()
            continue
        part = [x[:, a:e] for x in args(d)]
        for got_o, got_s, start in ((o, s, d["init"][i:i + 1]), (o0, s0, None)):
            o_ref, s_ref = ref.delta_rule(*part, start, N ** -0.5, True)
            assert ref.rel(got_s[i:i + 1], s_ref) <= state_tol(L)
            assert ref.rel(got_o[:, a:e], o_ref) <= out_tol(L)


def test_more_sequences_than_threads(cuda_device):
    """A CTA ranks the sequences by length up to its number of threads; past that they run in order."""
    n, L, H, G, P, N = 500, 67, 2, 1, 64, 64
    d = ref.draw(n, L, H, G, P, N, BF, seed=3, unit=False)
    o_ref, s_ref = ref.delta_rule(*args(d), d["init"], N ** -0.5, True)
    flat = [x.reshape((1, n * L) + tuple(x.shape[2:])).to(cuda_device) for x in args(d)]
    cut = torch.arange(0, n * L + 1, L, dtype=torch.int32, device=cuda_device)
    o, s = ssd.delta_rule_varlen_fwd(*flat, cut, init_states=d["init"].to(cuda_device),
                                     qk_l2norm=True)
    assert ref.rel(s, s_ref) <= state_tol(L)
    assert ref.rel(o.view(n, L, H, P), o_ref) <= out_tol(L)


def test_not_finite_stays_in_its_head_and_sequence(cuda_device):
    """Heads that share a CTA, and packed sequences that share a chunk's rows, keep to themselves.  In
    its own head and sequence it reaches every later token, and back to the start of its chunk of 64:
    there it is multiplied by the zeros above a triangle's diagonal."""
    L, H, G, P, N, cu = 300, 24, 2, 64, 128, [0, 100, 300]
    d = to(ref.draw(1, L, H, G, P, N, BF, seed=9, unit=False, nseq=2), cuda_device)
    cut = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    run = lambda: ssd.delta_rule_varlen_fwd(*args(d), cut, init_states=d["init"], qk_l2norm=True)
    o, s = run()
    d["beta"][0, 20, 3] = float("nan")        # head 3 of the first sequence, from token 20 on
    d["v"][0, 40, 6, 5] = float("inf")        # one row of the state of head 6
    d["g"][0, 130, 9] = float("nan")          # head 9 of the second sequence
    d["k"][0, 250, 1] = float("nan")          # a key: group 1 (heads 12 on) of the second sequence
    o2, s2 = run()
    head = torch.zeros(H, dtype=torch.bool, device=cuda_device)
    head[[3, 6, 9]] = True
    assert torch.equal(o[:, :100, ~head], o2[:, :100, ~head])
    assert torch.equal(s[0, ~head], s2[0, ~head])
    assert torch.isnan(o2[:, 20:100, 3]).all()
    assert torch.isnan(s2[0, 3]).all()
    rows = torch.arange(P, device=cuda_device) != 5
    assert torch.equal(s[0, 6, rows], s2[0, 6, rows]) and not torch.isfinite(s2[0, 6, 5]).any()
    assert torch.equal(s[1, :9], s2[1, :9]) and torch.equal(s[1, 10:12], s2[1, 10:12])
    assert torch.isnan(s2[1, 9]).all() and torch.isnan(s2[1, 12:]).all()
    assert torch.equal(o[:, 100:228, 12:], o2[:, 100:228, 12:])   # two chunks
    assert torch.isnan(o2[:, 250:, 12:]).all()


def test_guard_bands_status_and_aliased_states(cuda_device):
    b, L, H, G, P, N = 2, 135, 21, 7, 64, 128
    d = to(ref.draw(b, L, H, G, P, N, BF, seed=8, unit=False), cuda_device)
    want_o, want_s = ssd.delta_rule_fwd(*args(d), init_state=d["init"], qk_l2norm=True)
    n = d["v"].numel()
    ob = torch.full((n + 256,), 5.0, dtype=BF, device=cuda_device)
    sb = torch.full((d["init"].numel() + 256,), 5.0, device=cuda_device)
    o, s = ob[128:128 + n].view_as(d["v"]), sb[128:-128].view_as(d["init"])
    s.copy_(d["init"])
    size = ssd.delta_rule_workspace_size(ssd.make_shape(b, L, H, P, N, G, ssd.SSD_BF16))
    wb = torch.full((size + 512,), 9, dtype=torch.uint8, device=cuda_device)
    ws = wb[256:-256]
    ssd.delta_rule_fwd(*args(d), init_state=s, o=o, final_state=s, workspace=ws, qk_l2norm=True)
    assert ssd.workspace_status(ws) == ssd.SSD_OK
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
    assert (ob[:128] == 5).all() and (ob[128 + n:] == 5).all()
    assert (sb[:128] == 5).all() and (sb[-128:] == 5).all()
    assert (wb[:256] == 9).all() and (wb[-256:] == 9).all()


def test_inconsistent_offsets_compute_nothing(cuda_device):
    H = 24
    d = to(ref.draw(1, 300, H, 1, 64, 128, BF, nseq=2), cuda_device)
    shape = ssd.make_shape(1, 300, H, 64, 128, 1, ssd.SSD_BF16)
    ws = torch.empty(ssd.lib().ssd_delta_rule_varlen_workspace_size(ctypes.byref(shape), 2),
                     dtype=torch.uint8, device=cuda_device)
    for cu in ([0, 60, 299], [1, 60, 300], [0, 301, 300], [0, -4, 300], [0, 100, 300]):
        o, s = torch.full_like(d["v"], 3.0), torch.full_like(d["init"], 3.0)
        ssd.delta_rule_varlen_fwd(*args(d), torch.tensor(cu, dtype=torch.int32, device=cuda_device),
                                  init_states=d["init"], o=o, final_states=s, workspace=ws)
        good = cu == [0, 100, 300]   # the status is the last call's
        assert ssd.workspace_status(ws) == (ssd.SSD_OK if good else ssd.SSD_ERR_INVALID_ARG)
        assert bool((o == 3).all()) != good and bool((s == 3).all()) != good


def test_streams_and_captured_calls(cuda_device):
    """Two streams at once with workspaces of their own, and two captured calls that share one, one
    after the other, replayed on new inputs."""
    a = to(ref.draw(2, 300, 20, 2, 64, 128, BF, seed=1, unit=False), cuda_device)
    b = to(ref.draw(2, 300, 20, 2, 64, 128, BF, seed=2, unit=False), cuda_device)
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
    size = ssd.delta_rule_workspace_size(ssd.make_shape(2, 300, 20, 64, 128, 2, ssd.SSD_BF16))
    ws = torch.empty(size, dtype=torch.uint8, device=cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        first = run(a, workspace=ws)
        second = run(b, workspace=ws)
    for k in ("q", "k", "v", "g", "beta", "init"):
        x = a[k].clone()
        a[k].copy_(b[k])
        b[k].copy_(x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for w, g in zip(reversed(want), (first, second)):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("L,H,P", [(5, 2, 64), (70, 4, 64), (70, 4, 48), (100, 2, 20), (130, 40, 64)])
def test_status_word_is_left_clean(cuda_device, L, H, P):
    """By every forward kernel, whatever the workspace held; and by the backward."""
    d = to(ref.draw(1, L, H, 2, P, 128, BF), cuda_device)
    size = ssd.delta_rule_workspace_size(ssd.make_shape(1, L, H, P, 128, 2, ssd.SSD_BF16))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=cuda_device)
    ssd.delta_rule_fwd(*args(d), workspace=ws)
    assert ssd.workspace_status(ws) == ssd.SSD_OK
    if P % 16 == 0:
        shape = ssd.make_shape(1, L, H, P, 128, 2, ssd.SSD_BF16)
        size = ssd.lib().ssd_delta_rule_bwd_workspace_size(ctypes.byref(shape))
        ws = torch.full((size,), 255, dtype=torch.uint8, device=cuda_device)
        ssd.delta_rule_bwd(*args(d), d["v"], workspace=ws)
        assert ssd.workspace_status(ws) == ssd.SSD_OK
