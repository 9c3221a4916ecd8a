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


def test_sizes_at_the_end_of_64_bits(iqp):
    """No size check is done with numbers that pass 2^63 (the sanitized run of this
    test ends at one)."""
    L, p, uns = iqp._lib, P(256), iqp.IQP_ERR_UNSUPPORTED
    for M in (LAST, LAST - 1, LAST - 2, LAST - 3, 1 << 62, (1 << 26) - 3):
        assert L.moe_route(p, 8, 0, None, M, 8, 2, 0, 1, 1.0, p, p, None) == uns, M
        assert L.moe_combine(p, 8, 4, p, p, M, 2, 8, None, 0, p, 8, None) == uns, M
    assert L.moe_combine(p, LAST - 7, 4, p, p, 1, 2, LAST - 7, None, 0, p, LAST - 7, None) == uns
    assert iqp.group_rows_workspace_bytes(LAST, 8) == 0 and iqp.lora_add_workspace_bytes(LAST, 8, 16, LAST) == 0
    assert L.group_rows(p, LAST, 8, p, p, p, p, LAST, None) == uns
    for M in (LAST, (1 << 31) - 1):
        assert L.lora_add(p, LAST - 7, M, 8, p, p, None, 8, p, p, 2, 8, p, 8, p, LAST, None) == uns
        assert L.lora_add(p, 8, M, 8, p, p, None, 8, p, p, 2, LAST, p, LAST, p, LAST, None) == uns
    far = (1 << 31) - 16
    for M, lda, sm, sw in ((LAST, 128, 1, LAST), (LAST, LAST - 15, LAST, 1), ((1 << 31) - 1, far, far, 1), ((1 << 31) - 1, 128, 1, 1 << 31),
                           (1, LAST - 15, 1, 1)):
        for N in (1, (1 << 31) - 1, LAST // 2):
            assert L.fp8_grouped_gemm_1x128_128x128(p, lda, p, sm, sw, M, p, LAST - 15, 128, p, LAST, LAST, p, p, M, 3, 0, N, 128, p, LAST,
                                                    None) == uns, (M, lda, N)
            assert L.fp8_grouped_swiglu_1x128(p, lda, p, sm, sw, M, p, LAST - 15, 128, p, LAST, LAST, p, p, M, 3, 0, N, 128, p, LAST - 15, p,
                                              LAST, 1, None) == uns, (M, lda, N)
