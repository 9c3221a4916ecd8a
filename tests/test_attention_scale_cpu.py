"""Softmax scales that attention over the FP8 cache takes and refuses, on the
host (the addresses are never followed)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


def call(iqp, scale):
    need = iqp.attention_fp8_kv_workspace_bytes(128)
    return iqp._lib.attention_fp8_kv(P(16), 512, 3, 4, 2, 128, P(16), P(16), P(16), P(16), 5, 64, P(16), 4, 4, P(16), P(16), 2, scale, 0,
                                     P(16), 512, P(256), need, None)


@pytest.mark.parametrize("scale", [3e38, 2.4e38, 1.9e19, 5e-20, 1e-39, 1e-45, 0.0, -0.125])
def test_scales_that_leave_float32_are_refused(scale):
    import fp4_quantized_prep_amd as iqp
    assert call(iqp, scale) == iqp.IQP_ERR_INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run")
@pytest.mark.parametrize("scale", [2.0 ** 64, 2.0 ** -64, 1.0, 0.125])
def test_scales_that_are_taken(scale):
    """Past the checks of the arguments, up to that of the device."""
    import fp4_quantized_prep_amd as iqp
    assert call(iqp, scale) == iqp.IQP_ERR_HIP
