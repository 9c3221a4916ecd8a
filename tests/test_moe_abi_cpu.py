"""Refusals of the entry points whose weights depend on the token, on the host:
the C calls return before anything touches a device (the addresses are never
followed), and the binding rejects wrong tensors before it calls them."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def iqp():
    import fp4_quantized_prep_amd as m
    return m


def test_route_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(z=16, ld=64, half=0, b=16, M=3, E=64, top=8, scoring=0, renorm=1, scale=1.0, w=16, e=16):
        return iqp._lib.moe_route(P(z), ld, half, P(b), M, E, top, scoring, renorm, scale, P(w), P(e), None)
    for bad in (dict(M=-1), dict(E=-1), dict(top=-1), dict(scoring=-1), dict(scoring=3), dict(z=0), dict(w=0), dict(e=0),
                dict(E=0), dict(top=0), dict(top=65), dict(ld=63)):
        assert call(**bad) == inv, bad
    for bad in (dict(E=1025, ld=1025), dict(E=100, ld=100, top=65), dict(z=18), dict(z=17, half=1), dict(b=18), dict(w=18),
                dict(e=18), dict(M=1 << 31)):
        assert call(**bad) == uns, bad
    assert call(M=0) == iqp.IQP_OK


def test_group_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(i=16, R=100, G=8, o=16, r=16, s=16, w=0, wb=0):
        return iqp._lib.group_rows(P(i), R, G, P(o), P(r), P(s), P(w), wb, None)
    need = iqp.group_rows_workspace_bytes(10000, 8)
    assert need > 0 and iqp.group_rows_workspace_bytes(100, 8) == 0
    for rows, groups in ((-1, 8), (1 << 31, 8), (10000, 0), (10000, 1025), (10000, -1)):
        assert iqp.group_rows_workspace_bytes(rows, groups) == 0
    for bad in (dict(R=-1), dict(G=-1), dict(wb=-1), dict(G=0), dict(o=0), dict(i=0), dict(r=0), dict(s=0), dict(R=10000),
                dict(R=10000, w=16, wb=need - 1)):
        assert call(**bad) == inv, bad
    for bad in (dict(G=1025), dict(R=1 << 31), dict(i=18), dict(o=18), dict(r=18), dict(s=18), dict(R=10000, w=18, wb=need)):
        assert call(**bad) == uns, bad


def grouped(a=16, lda=256, s=16, sm=1, sw=1, M=2, w=16, ldwg=65536, ldw=256, ws=16, wsg=4, lws=2, off=16, rows=16, R=4, G=3, top=2,
            N=256, K=256):
    return P(a), lda, P(s), sm, sw, M, P(w), ldwg, ldw, P(ws), wsg, lws, P(off), P(rows), R, G, top, N, K


GROUPED_INVALID = (dict(M=-1), dict(R=-1), dict(G=-1), dict(top=-1), dict(N=-1), dict(K=-1), dict(a=0), dict(s=0), dict(w=0),
                   dict(ws=0), dict(off=0), dict(rows=0), dict(G=0), dict(K=0), dict(lda=128), dict(ldw=128), dict(M=3), dict(M=4),
                   dict(R=5), dict(top=3), dict(top=0), dict(M=1 << 62, R=1 << 62), dict(sm=3, sw=3), dict(lws=1), dict(ldwg=-16), dict(wsg=-1))
GROUPED_UNSUPPORTED = (dict(K=200), dict(a=8), dict(lda=264), dict(w=8), dict(ldw=264), dict(ldwg=65544), dict(s=18), dict(off=18),
                       dict(rows=18), dict(G=1025), dict(ldw=(1 << 22) + 16), dict(lda=1 << 31), dict(lda=(1 << 31) - 256),
                       dict(K=257 * 128, lda=257 * 128, ldw=257 * 128, lws=257, sm=65), dict(M=1 << 31, R=1 << 32), dict(sm=1 << 31),
                       dict(sm=(1 << 29) - 1), dict(ldwg=1 << 53), dict(wsg=1 << 53), dict(lws=1 << 32))


def test_grouped_gemm_refusals(iqp):
    def call(o=16, ldo=256, **more):
        return iqp._lib.fp8_grouped_gemm_1x128_128x128(*grouped(**more), P(o), ldo, None)
    for bad in GROUPED_INVALID + (dict(o=0), dict(ldo=255)):
        assert call(**bad) == iqp.IQP_ERR_INVALID, bad
    for bad in GROUPED_UNSUPPORTED + (dict(o=17), dict(N=1 << 31, ldo=1 << 31)):
        assert call(**bad) == iqp.IQP_ERR_UNSUPPORTED, bad
    assert call(R=0, M=0) == iqp.IQP_OK and call(N=0) == iqp.IQP_OK


def test_grouped_swiglu_refusals(iqp):
    def call(q=16, ldq=256, qs=16, qm=1, qw=1, **more):
        return iqp._lib.fp8_grouped_swiglu_1x128(*grouped(**more), P(q), ldq, P(qs), qm, qw, None)
    for bad in GROUPED_INVALID + (dict(q=0), dict(qs=0), dict(ldq=240), dict(qm=3, qw=3), dict(qm=1, qw=3, N=640, ldq=640)):
        assert call(**bad) == iqp.IQP_ERR_INVALID, bad
    for bad in GROUPED_UNSUPPORTED + (dict(N=200), dict(q=8), dict(ldq=264), dict(qs=18), dict(N=1 << 30, ldq=1 << 30)):
        assert call(**bad) == iqp.IQP_ERR_UNSUPPORTED, bad
    assert call(R=0, M=0) == iqp.IQP_OK and call(N=0) == iqp.IQP_OK


def test_combine_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(y=16, ldy=64, R=6, s=16, w=16, M=3, top=2, d=64, sh=16, lds=64, o=16, ldo=64):
        return iqp._lib.moe_combine(P(y), ldy, R, P(s), P(w), M, top, d, P(sh), lds, P(o), ldo, None)
    for bad in (dict(R=-1), dict(M=-1), dict(top=-1), dict(d=-1), dict(y=0), dict(s=0), dict(w=0), dict(o=0), dict(top=0), dict(ldy=56),
                dict(ldo=56), dict(lds=56)):
        assert call(**bad) == inv, bad
    for bad in (dict(d=60), dict(y=8), dict(ldy=68), dict(o=8), dict(ldo=68), dict(sh=8), dict(lds=68), dict(s=18), dict(w=18),
                dict(R=1 << 31), dict(M=1 << 31), dict(d=1 << 31, ldy=1 << 31, ldo=1 << 31, lds=1 << 31)):
        assert call(**bad) == uns, bad
    assert call(M=0) == iqp.IQP_OK and call(d=0) == iqp.IQP_OK


def test_lora_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED
    need = iqp.lora_add_workspace_bytes(5, 3, 16, 256)
    assert need > 0
    for bad in ((0, 3, 16, 256), (1 << 31, 3, 16, 256), (5, 0, 16, 256), (5, 1025, 16, 256), (5, 3, 0, 256), (5, 3, 136, 256), (5, 3, 16, 0)):
        assert iqp.lora_add_workspace_bytes(*bad) == 0, bad

    def call(x=16, ldx=256, M=5, K=256, a=16, b=16, sc=16, rank=16, off=16, rows=16, G=3, N=100, o=16, ldo=100, w=256, wb=need):
        return iqp._lib.lora_add(P(x), ldx, M, K, P(a), P(b), P(sc), rank, P(off), P(rows), G, N, P(o), ldo, P(w), wb, None)
    for bad in (dict(M=-1), dict(K=-1), dict(rank=-1), dict(G=-1), dict(N=-1), dict(wb=-1), dict(x=0), dict(a=0), dict(b=0), dict(off=0),
                dict(rows=0), dict(o=0), dict(w=0), dict(K=0), dict(rank=0), dict(ldx=248), dict(ldo=99), dict(wb=need - 1)):
        assert call(**bad) == inv, bad
    for bad in (dict(rank=12), dict(rank=136), dict(K=252), dict(K=(1 << 22) + 8, ldx=1 << 23, wb=1 << 40), dict(x=8), dict(ldx=260), dict(a=8), dict(b=8), dict(sc=18), dict(off=18), dict(ldx=1 << 30), dict(M=(1 << 20) + 1, ldx=1024, wb=1 << 40),
                dict(rows=18), dict(o=17), dict(M=1 << 31), dict(N=1 << 31, ldo=1 << 31), dict(G=1025), dict(w=128)):
        assert call(**bad) == uns, bad
    assert call(M=0) == iqp.IQP_OK and call(N=0) == iqp.IQP_OK and call(G=0) == iqp.IQP_OK


def test_python_refusals(iqp):
    """Tensors that are not on a GPU, and names that are none."""
    z = torch.zeros(2, 8)
    i = torch.zeros(2, dtype=torch.int32)
    gr = iqp.RowGroups(i, i, i)
    b = torch.zeros(2, 8, dtype=torch.bfloat16)
    c = torch.zeros(2, 128, dtype=torch.uint8)
    for call in (lambda: iqp.moe_route(z, 2), lambda: iqp.group_rows(i, 2), lambda: iqp.fp8_grouped_gemm_1x128_128x128(c, i, c, c, gr),
                 lambda: iqp.fp8_grouped_swiglu_1x128(c, i, c, c, gr), lambda: iqp.moe_combine(b, gr, z), lambda: iqp.lora_add(b, b, b, b, gr)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(ValueError, match="scoring"):
        iqp.moe_route(z, 2, scoring="relu")


def test_launches_of_too_many_workgroups_are_refused(iqp):
    """2^24 workgroups of 256 threads or more are beyond a launch: every call says so
    before it looks for a device."""
    uns = iqp.IQP_ERR_UNSUPPORTED
    L, p = iqp._lib, P(256)
    for M in ((1 << 26) - 3, 1 << 26, (1 << 31) - 1):
        assert L.moe_route(p, 8, 0, None, M, 8, 2, 0, 1, 1.0, p, p, None) == uns, M
    for M, d in ((1 << 24, 8), (1 << 23, 2056), ((1 << 31) - 1, 8), ((1 << 31) - 1, (1 << 31) - 8)):
        assert L.moe_combine(p, d, 4, p, p, M, 2, d, None, 0, p, d, None) == uns, (M, d)
    for G, R, N in ((1024, 1024, 1 << 22), (1024, 1 << 20, 1 << 20), (2, 4, (1 << 31) - 256)):
        assert L.fp8_grouped_gemm_1x128_128x128(p, 128, p, 1, R, R, p, 128 * N, 128, p, (N + 127) // 128, 1, p, p, R, G, 0, N, 128, p, N,
                                                None) == uns, (G, R, N)
        I = N // 2
        assert L.fp8_grouped_swiglu_1x128(p, 128, p, 1, R, R, p, 128 * N, 128, p, N // 128, 1, p, p, R, G, 0, I, 128, p, I, p,
                                          1, R, None) == uns, (G, R, I)
    for M, G, N in ((1024, 1024, 1 << 22), (4, 4, (1 << 31) - 1), (1 << 20, 8, 1 << 18)):
        need = iqp.lora_add_workspace_bytes(M, G, 16, 64)
        assert L.lora_add(p, 64, M, 64, p, p, None, 16, p, p, G, N, p, N, p, need, None) == uns, (M, G, N)
