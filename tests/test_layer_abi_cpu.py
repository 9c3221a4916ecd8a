"""Refusals of the attention layer's entry points, on the host: the C calls
return before anything touches a device (the addresses are never followed),
and the binding rejects wrong tensors before it calls them."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def iqp():
    import fp4_quantized_prep_amd as m
    return m


def test_gemm_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(a=16, lda=256, s=16, sm=1, sw=1, w=16, ldw=256, ws=16, ldws=2, M=1, N=130, K=256, o=16, ldo=136, wk=0, wkb=0):
        return iqp._lib.fp8_gemm_1x128_128x128(P(a), lda, P(s), sm, sw, P(w), ldw, P(ws), ldws, M, N, K, P(o), ldo, P(wk), wkb, None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(a=0), dict(s=0), dict(w=0), dict(ws=0), dict(o=0), dict(K=0),
                dict(lda=128), dict(ldw=128), dict(ldo=129), dict(ldws=1), dict(sm=3, sw=3), dict(M=4, sm=1, sw=2)):
        assert call(**bad) == inv, bad
    for bad in (dict(K=200), dict(a=8), dict(w=8), dict(lda=264), dict(ldw=264), dict(s=18), dict(o=17),
                dict(K=257 * 128, lda=257 * 128, ldw=257 * 128, ldws=257, sm=65), dict(lda=1 << 23), dict(ldw=1 << 23),
                dict(lda=(1 << 22) + 16), dict(ldw=(1 << 22) + 16), dict(sm=1 << 20), dict(sm=1 << 19),
                dict(M=2, sm=1, sw=1 << 27), dict(M=1 << 31, sm=1, sw=1 << 31, ldo=136)):
        assert call(**bad) == uns, bad
    # a product that is split: the workspace's size and alignment count
    need = iqp.fp8_gemm_workspace_bytes(128, 256, 7168)
    assert need > 0 and iqp.fp8_gemm_workspace_bytes(16, 256, 7168) == 0 and iqp.fp8_gemm_workspace_bytes(0, 256, 7168) == 0
    big = dict(M=128, N=256, K=7168, lda=7168, ldw=7168, ldws=56, sm=14, ldo=256)
    assert call(**big, wk=256, wkb=need - 1) == inv
    assert call(**big, wk=128, wkb=need) == uns
    assert call(wkb=-1) == inv
    assert call(M=0) == iqp.IQP_OK and call(N=0) == iqp.IQP_OK


def test_norm_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(q=16, ldq=512, k=16, ldk=128, M=2, Hq=4, Hk=1, D=128, rd=64, qw=16, kw=16, eps=1e-6, pos=16, cs=16, mp=9,
             qo=16, ldqo=512, ko=16, ldko=128, flags=0):
        return iqp._lib.qk_norm_rope(P(q), ldq, P(k), ldk, M, Hq, Hk, D, rd, P(qw), P(kw), eps, P(pos), P(cs), mp, P(qo),
                                     ldqo, P(ko), ldko, flags, None)
    for bad in (dict(M=-1), dict(Hq=0), dict(Hk=0), dict(q=0), dict(k=0), dict(qw=0), dict(kw=0), dict(pos=0), dict(cs=0),
                dict(qo=0), dict(ko=0), dict(mp=0), dict(eps=-1.0), dict(eps=float("nan")), dict(ldq=504), dict(ldk=120),
                dict(ldqo=504), dict(ldko=120), dict(rd=144), dict(flags=2), dict(flags=4), dict(flags=-1)):
        assert call(**bad) == inv, bad
    for bad in (dict(D=96, ldq=512, rd=32), dict(rd=0), dict(rd=24), dict(q=8), dict(ldq=516), dict(k=8), dict(ldk=132),
                dict(qo=8), dict(ldqo=516), dict(ko=8), dict(ldko=132), dict(qw=8), dict(kw=8), dict(pos=4), dict(cs=8)):
        assert call(**bad) == uns, bad
    assert call(M=0) == iqp.IQP_OK


def batch(n=5, b=64, table=16, ldt=4, mb=4, lens=16, cu=16, S=2):
    return n, b, P(table), ldt, mb, P(lens), P(cu), S


BATCH_INVALID = (dict(n=-1), dict(b=-16), dict(mb=-1), dict(S=-1), dict(table=0), dict(lens=0), dict(cu=0), dict(mb=0),
                 dict(n=0), dict(ldt=3))
BATCH_UNSUPPORTED = (dict(b=48), dict(b=8), dict(b=256), dict(table=18), dict(lens=18), dict(cu=18), dict(n=1 << 31),
                     dict(mb=(1 << 24) + 1, ldt=1 << 25))


def test_append_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(k=16, ldk=256, v=16, ldv=256, T=3, Hk=2, D=128, kc=16, vc=16, ks=16, vs=16, **more):
        return iqp._lib.kv_cache_append_fp8(P(k), ldk, P(v), ldv, T, Hk, D, P(kc), P(vc), P(ks), P(vs), *batch(**more), None)
    for bad in BATCH_INVALID + (dict(T=-1), dict(Hk=0), dict(k=0), dict(v=0), dict(kc=0), dict(vc=0), dict(ks=0),
                                dict(vs=0), dict(ldk=248), dict(ldv=248)):
        assert call(**bad) == inv, bad
    for bad in BATCH_UNSUPPORTED + (dict(D=96), dict(D=256), dict(k=8), dict(ldk=260), dict(v=8), dict(ldv=260),
                                    dict(kc=8), dict(vc=8), dict(T=1 << 31), dict(Hk=65536, ldk=65536 * 128)):
        assert call(**bad) == uns, bad
    assert call(T=0) == iqp.IQP_OK and call(S=0) == iqp.IQP_OK


def test_read_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED

    def call(kc=16, vc=16, ks=16, vs=16, Hk=2, D=128, ko=16, ldk=256, vo=16, ldv=256, T=3, **more):
        n, b, table, ldt, mb, lens, cu, S = batch(**more)
        return iqp._lib.kv_cache_read_fp8(P(kc), P(vc), P(ks), P(vs), n, b, Hk, D, table, ldt, mb, lens, cu, S, P(ko), ldk,
                                          P(vo), ldv, T, None)
    for bad in BATCH_INVALID + (dict(T=-1), dict(Hk=0), dict(ko=0), dict(vo=0), dict(kc=0), dict(vc=0), dict(ks=0),
                                dict(vs=0), dict(ldk=248), dict(ldv=248)):
        assert call(**bad) == inv, bad
    for bad in BATCH_UNSUPPORTED + (dict(D=96), dict(ko=8), dict(ldk=260), dict(vo=8), dict(ldv=260), dict(kc=8), dict(vc=8)):
        assert call(**bad) == uns, bad
    assert call(T=0) == iqp.IQP_OK and call(S=0) == iqp.IQP_OK


def test_attention_refusals(iqp):
    inv, uns = iqp.IQP_ERR_INVALID, iqp.IQP_ERR_UNSUPPORTED
    need = iqp.attention_fp8_kv_workspace_bytes(128)
    assert need > iqp.attention_fp8_kv_workspace_bytes(64) > 0 and iqp.attention_fp8_kv_workspace_bytes(96) == 0

    def call(q=16, ldq=512, T=3, Hq=4, Hk=2, D=128, kc=16, vc=16, ks=16, vs=16, scale=0.1, window=0, o=16, ldo=512, ws=256,
             wsb=need, **more):
        return iqp._lib.attention_fp8_kv(P(q), ldq, T, Hq, Hk, D, P(kc), P(vc), P(ks), P(vs), *batch(**more), scale, window,
                                         P(o), ldo, P(ws), wsb, None)
    for bad in BATCH_INVALID + (dict(T=-1), dict(Hk=0), dict(Hq=0), dict(Hq=-4), dict(Hq=3), dict(q=0), dict(kc=0),
                                dict(vc=0), dict(ks=0), dict(vs=0), dict(o=0), dict(ws=0), dict(wsb=need - 1), dict(ldq=504),
                                dict(ldo=504), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(window=-1)):
        assert call(**bad) == inv, bad
    for bad in BATCH_UNSUPPORTED + (dict(D=96), dict(D=256), dict(q=8), dict(ldq=516), dict(o=8), dict(ldo=516), dict(kc=8),
                                    dict(vc=8), dict(ws=128)):
        assert call(**bad) == uns, bad
    assert call(T=0) == iqp.IQP_OK and call(S=0) == iqp.IQP_OK


def test_binding_takes_gpu_tensors_only(iqp):
    t = torch.zeros(2, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        iqp.fp8_gemm_1x128_128x128(t, t, t, t)
    with pytest.raises(TypeError):
        iqp.fp8_gemm_1x128_128x128(None, t, t, t)
    with pytest.raises(ValueError):
        iqp.fp8_kv_cache(4, 2, head_dim=96, device="cpu")
    c = iqp.fp8_kv_cache(4, 2, head_dim=64, block_size=16, device="cpu")
    assert tuple(c.k.shape) == (4, 2, 16, 64) and tuple(c.v.shape) == (4, 2, 64, 16) and tuple(c.k_scales.shape) == (4, 2)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        iqp.kv_cache_append_fp8(x, x, c, i[None], i, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        iqp.attention_fp8_kv(x, c, i[None], i, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        iqp.kv_cache_read_fp8(c, i[None], i, torch.zeros(2, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        iqp.qk_norm_rope(x, x, x[0, 0], x[0, 0], i.long(), torch.zeros(1, 64), head_dim=64)
