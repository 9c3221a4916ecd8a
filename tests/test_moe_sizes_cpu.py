"""Sizes that the entry points of experts and adapters refuse, on the host."""
import ctypes

import pytest

P = ctypes.c_void_p
LAST = (1 << 63) - 1


@pytest.fixture(scope="module")
def iqp():
    import fp4_quantized_prep_amd as m
    return m


def test_lora_workspace_of_refused_sizes(iqp):
    """No bytes for what lora_add refuses: a rank or K that is no multiple of 8, a K
    beyond 2^22; and then the call says unsupported, with a workspace or without."""
    sizes = ((5, 3, 12, 256), (5, 3, 9, 256), (5, 3, 16, 250), (5, 3, 16, 255), (5, 3, 16, (1 << 22) + 8), (5, 3, 16, LAST - 63),
             (5, 3, 136, 256), (5, 1025, 16, 256), (1 << 31, 3, 16, 256))
    for M, G, rank, K in sizes:
        assert iqp.lora_add_workspace_bytes(M, G, rank, K) == 0, (M, G, rank, K)
        ldx = (K + 7) // 8 * 8
        for w, wb in ((None, 0), (P(256), 1 << 40)):
            assert iqp._lib.lora_add(P(16), ldx, M, K, P(16), P(16), None, rank, P(16), P(16), G, 100, P(16), 100, w, wb, None) \
                == iqp.IQP_ERR_UNSUPPORTED, (M, G, rank, K, wb)
    assert iqp.lora_add_workspace_bytes(5, 3, 16, 1 << 22) > 0 and iqp.lora_add_workspace_bytes(5, 3, 128, 8) > 0
    # a workspace that is missing or too small, where the sizes are right
    need = iqp.lora_add_workspace_bytes(5, 3, 16, 256)
    for w, wb in ((None, 0), (None, need), (P(256), need - 1)):
        assert iqp._lib.lora_add(P(16), 256, 5, 256, P(16), P(16), None, 16, P(16), P(16), 3, 100, P(16), 100, w, wb, None) == iqp.IQP_ERR_INVALID
