"""RMS norm calls of several host threads at once, each on a stream of its own."""
import ctypes
import threading

import pytest
import torch

from mamba_ssd_layer_scan_b200 import ssd

pytestmark = pytest.mark.gpu


def test_threads_with_rows_of_different_widths(cuda_device):
    """The same kernel with rings of 46 KB and of 74 KB of shared memory (the backward, with a gradient
    added), called through the C ABI so that the threads spend their time inside it: no call may take
    back what another one has been given."""
    rows, count = 8, 4000
    lib, p = ssd.lib(), lambda t: ctypes.c_void_p(t.data_ptr())
    failed, gate = [], threading.Barrier(4)

    def work(dim, seed):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            gen = torch.Generator(device=cuda_device).manual_seed(seed)
            x, dy, dres = (torch.randn(rows, dim, device=cuda_device, generator=gen).bfloat16()
                           for _ in range(3))
            w = torch.ones(dim, device=cuda_device)
            want = ssd.rms_norm_bwd(x, w, dy, dresidual=dres)
            dx, dw = torch.empty_like(x), torch.empty_like(w)
            desc = ssd.NormDesc(rows, dim, ssd.SSD_BF16, 0, 0, 1e-5)
            size = lib.ssd_rms_norm_bwd_workspace_size(ctypes.byref(desc))
            ws = torch.empty(size, dtype=torch.uint8, device=cuda_device)
            args = (ctypes.byref(desc), p(x), None, p(w), p(dy), p(dres), p(dx), None, p(dw), p(ws),
                    ctypes.c_size_t(size), ctypes.c_void_p(stream.cuda_stream))
            gate.wait(timeout=60)
            refused = sum(lib.ssd_rms_norm_bwd(*args) != ssd.SSD_OK for _ in range(count))
            stream.synchronize()
            if refused:
                failed.append(f"dim {dim}: {refused} of {count} calls refused, {ssd.last_error()}")
            elif not (torch.equal(dx, want["dx"]) and torch.equal(dw, want["dweight"])):
                failed.append(f"dim {dim}: other values than a call alone")

    threads = [threading.Thread(target=work, args=(dim, i))
               for i, dim in enumerate((2560, 4096, 2560, 4096))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
