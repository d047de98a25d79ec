"""The one-token update takes no notice of the shape's seqlen, whatever a caller left there (no GPU
needed: an empty batch launches nothing)."""
import ctypes

import pytest

from mamba_ssd_layer_scan_b200 import build, ssd


@pytest.mark.parametrize("seqlen", [0, 1, -1, -(1 << 63), (1 << 34) + 1, (1 << 63) - 1])
def test_update_ignores_seqlen(seqlen):
    build.build()
    sh = ssd.make_shape(0, seqlen, 80, 64, 128, 1, ssd.SSD_BF16)
    o = ssd.DeltaOptions(0.1, 1)
    rc = ssd.lib().ssd_delta_rule_update(ctypes.byref(sh), None, None, None, None, None, None,
                                         ctypes.byref(o), None, None)
    assert rc == ssd.SSD_OK, ssd.last_error()
