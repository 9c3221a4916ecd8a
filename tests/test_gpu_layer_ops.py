"""GPU: the attention layer's operators against plain float64 implementations
(layer_ref), at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import mfma_error_bound

pytestmark = pytest.mark.gpu


def gen(*key):
    return np.random.default_rng([77, *key])


def bf16(g, *shape, scale=1.0):
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


# ------------------------------------------------------------------ product

def exact_operands(g, M, N, K):
    """Codes of small whole numbers and scales whose sums stay whole numbers
    below 2^11 times one power of two: every order of summation is exact."""
    val = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8)      # 0, 1, -1, 2, -2
    a = val[torch.from_numpy(g.integers(0, 5, (M, K)))]
    w = val[torch.from_numpy(g.integers(0, 5, (N, K)))]
    # sparse, so that a row's sum stays small
    a[torch.from_numpy(g.random((M, K)) > 64 / K)] = 0
    sb = torch.from_numpy(g.integers(126, 129, (M, K // 128)).astype(np.uint8))
    words = torch.zeros(M, -(-K // 512) * 4, dtype=torch.uint8)
    words[:, : K // 128] = sb
    ws = torch.from_numpy(g.integers(126, 129, (-(-N // 128), K // 128)).astype(np.uint8))
    return a, words.view(torch.int32), w, ws


GEMM_SIZES = [(96, 140, 3200), (70, 64, 7168), (130, 515, 7168), (1, 128, 128), (1, 1536, 7168), (3, 131, 256), (16, 257, 640), (17, 384, 1536), (31, 96, 2048), (33, 1, 128),
              (64, 512, 896), (65, 130, 1536), (100, 2115, 512), (128, 128, 1024), (129, 256, 384), (200, 1000, 768),
              (257, 640, 1536), (513, 264, 128), (777, 515, 1280), (1100, 1536, 256)]


@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
def test_gemm_exact_sums(gpu_lib, M, N, K):
    print("gemm exact", M, N, K, flush=True)
    a, words, w, ws = exact_operands(gen(1, M, N, K), M, N, K)
    ref = (R.dequant_rows(a, words) @ R.dequant_tiles(w, ws).T).to(torch.bfloat16)
    out = gpu_lib.fp8_gemm_1x128_128x128(a.cuda(), words.cuda(), w.cuda(), ws.cuda())
    assert out.shape == (M, N) and torch.equal(out.cpu(), ref)


@pytest.mark.parametrize("M,N,K", [(1, 1536, 1536), (19, 300, 7168), (300, 520, 1536)])
def test_gemm_of_quantised_operands(gpu_lib, M, N, K):
    print("gemm", M, N, K, flush=True)
    g = gen(2, M, N, K)
    x, w = bf16(g, M, K), bf16(g, -(-N // 128) * 128, K, scale=0.02)
    a, words = gpu_lib.fp8_quant_1x128_ue8m0(x.cuda(), scale_layout="mn")
    wq, ws = gpu_lib.fp8_quant_weight_128x128_ue8m0(w.cuda())
    out = gpu_lib.fp8_gemm_1x128_128x128(a, words, wq[:N], ws).cpu().double()
    ac, wc = a.cpu(), wq[:N].cpu()
    ref = R.dequant_rows(ac, words.cpu().contiguous()) @ R.dequant_tiles(wc, ws.cpu()).T
    sb = words.cpu().contiguous().view(torch.uint8)[:, : K // 128].numpy()
    rows = np.repeat(ws.cpu().numpy(), 128, 0)[:N]
    # the matrix cores' own bound, per row of W (gpu_util), then the rounding
    A, W = R.dequant_rows(ac, words.cpu().contiguous()).abs(), R.dequant_tiles(wc, ws.cpu()).abs()
    mf = 2.0 ** -9 * (A.view(M, K // 64, 64).amax(2) @ W.view(N, K // 64, 64).amax(2).T)
    assert sb.shape == (M, K // 128) and rows.shape[0] == N
    tol = mf + 2.0 ** -8 * (ref.abs() + mf)
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())


def test_gemm_bound_matches_the_fused_kernels():
    """The bound above is gpu_util's for whole 128-row tiles."""
    g = gen(3)
    a = torch.from_numpy(g.integers(0, 120, (5, 256)).astype(np.uint8))
    w = torch.from_numpy(g.integers(0, 120, (256, 256)).astype(np.uint8))
    sb = g.integers(120, 130, (5, 2)).astype(np.uint8)
    ws = g.integers(120, 130, (2, 2)).astype(np.uint8)
    words = torch.zeros(5, 4, dtype=torch.uint8)
    words[:, :2] = torch.from_numpy(sb)
    A = R.dequant_rows(a, words.view(torch.int32)).abs()
    W = R.dequant_tiles(w, torch.from_numpy(ws)).abs()
    mine = 2.0 ** -9 * (A.view(5, 4, 64).amax(2) @ W.view(256, 4, 64).amax(2).T).numpy()
    assert np.allclose(mine, mfma_error_bound(a.numpy(), sb, w.numpy(), ws), rtol=1e-12)


@pytest.mark.parametrize("M,N", [(5, 200), (150, 387), (300, 256)])
def test_gemm_strides_and_outputs(gpu_lib, M, N):
    """Padded rows of every operand, an out whose rows allow no wide stores, and
    nothing written outside out."""
    print("gemm strides", M, N, flush=True)
    K = 640
    a, words, w, ws = exact_operands(gen(4, M, N), M, N, K)
    ref = (R.dequant_rows(a, words) @ R.dequant_tiles(w, ws).T).to(torch.bfloat16)
    ap = torch.full((M, K + 48), 0x7F, dtype=torch.uint8)
    ap[:, :K] = a
    wp = torch.full((N, K + 16), 0x7F, dtype=torch.uint8)
    wp[:, :K] = w
    wsp = torch.full((ws.shape[0], ws.shape[1] + 3), 255, dtype=torch.uint8)
    wsp[:, : ws.shape[1]] = ws
    mn = torch.zeros((words.shape[1], M + 3), dtype=torch.int32)
    mn[:, :M] = words.T
    ap, wp, wsp, mn = ap.cuda()[:, :K], wp.cuda()[:, :K], wsp.cuda()[:, : ws.shape[1]], mn.cuda().T[:M]
    for pad, first in ((0, 0), (7, 1), (8, 8), (5, 0)):
        buf = torch.full((M + 2, N + first + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1:M + 1, first:first + N]
        gpu_lib.fp8_gemm_1x128_128x128(ap, mn, wp, wsp, out=out)
        want = torch.full_like(buf, 7.0)
        want[1:M + 1, first:first + N] = ref.cuda()
        assert torch.equal(buf, want), (pad, first)


def test_gemm_split_with_and_without_a_workspace(gpu_lib):
    """A product split over K: the caller's workspace holding anything, one too
    small, and the same product without one through the C call."""
    M, N, K = 100, 200, 4096
    a, words, w, ws = exact_operands(gen(20), M, N, K)
    ref = (R.dequant_rows(a, words) @ R.dequant_tiles(w, ws).T).to(torch.bfloat16)
    need = gpu_lib.fp8_gemm_workspace_bytes(M, N, K)
    assert need > 0
    a, words, w, ws = a.cuda(), words.cuda(), w.cuda(), ws.cuda()
    space = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(gpu_lib.fp8_gemm_1x128_128x128(a, words, w, ws, workspace=space).cpu(), ref)
    with pytest.raises(gpu_lib.IqpError) as e:
        gpu_lib.fp8_gemm_1x128_128x128(a, words, w, ws, workspace=space[:-256])
    assert e.value.status == gpu_lib.IQP_ERR_INVALID
    out = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    st = gpu_lib._lib.fp8_gemm_1x128_128x128(a.data_ptr(), K, words.data_ptr(), words.stride(0), 1, w.data_ptr(), K, ws.data_ptr(),
                                             K // 128, M, N, K, out.data_ptr(), N, None, 0,
                                             torch.cuda.current_stream().cuda_stream)
    assert st == gpu_lib.IQP_OK and torch.equal(out.cpu(), ref)


def test_gemm_is_deterministic_and_empty(gpu_lib):
    a, words, w, ws = (t.cuda() for t in exact_operands(gen(5), 70, 300, 512))
    w = torch.randint(0, 126, w.shape, dtype=torch.uint8, device="cuda")
    r = [gpu_lib.fp8_gemm_1x128_128x128(a, words, w, ws) for _ in range(3)]
    assert torch.equal(r[0], r[1]) and torch.equal(r[0], r[2])
    assert gpu_lib.fp8_gemm_1x128_128x128(a[:0], words[:0], w, ws).shape == (0, 300)


# --------------------------------------------------------------- norm, RoPE

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,hq,hk,d,rope", [(1, 1, 1, 64, 16), (1, 64, 8, 128, 64), (3, 6, 2, 64, 64), (17, 5, 1, 128, 32),
                                            (5, 4, 4, 256, 128), (2, 3, 3, 256, 256), (700, 24, 8, 128, 128),
                                            (1500, 64, 8, 128, 64), (900, 64, 1, 64, 48)])
def test_norm_rope(gpu_lib, M, hq, hk, d, rope, interleaved):
    print("norm", M, hq, hk, d, rope, interleaved, flush=True)
    g = gen(6, M, hq, d, rope)
    x = bf16(g, M, (hq + hk) * d + 24)
    x *= torch.from_numpy((2.0 ** g.integers(-6, 7, (M, 1))).astype(np.float32)).to(torch.bfloat16)
    if M > 2:
        x[1] = 0                                             # a head of zeros: eps alone
    q, k = x[:, :hq * d], x[:, hq * d + 8:(hq + hk) * d + 8]
    qw, kw = bf16(g, d) + 1, bf16(g, d) + 1
    max_pos = 300
    pos = torch.from_numpy(g.integers(-3, max_pos + 4, M))   # some outside the table: clamped
    cs = gpu_lib.rope_cos_sin_table(10000.0, max_pos, rope)
    xd = x.cuda()
    qd, kd = xd[:, :hq * d], xd[:, hq * d + 8:(hq + hk) * d + 8]
    kwargs = dict(eps=1e-6, head_dim=d, rope_layout="interleaved" if interleaved else "half_split")
    qo, ko = gpu_lib.qk_norm_rope(qd, kd, qw.cuda(), kw.cuda(), pos.cuda(), cs, **kwargs)
    for got, src, w, h in ((qo, q, qw, hq), (ko, k, kw, hk)):
        ref, tol = R.norm_rope(src.reshape(M, h, d), w, pos, cs.cpu(), 1e-6, interleaved)
        off = (got.cpu().double().view(M, h, d) - ref).abs()
        assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())
    # in place, on the projection's rows, touching nothing else
    keep = xd.clone()
    gpu_lib.qk_norm_rope(qd, kd, qw.cuda(), kw.cuda(), pos.cuda(), cs, q_out=qd, k_out=kd, **kwargs)
    keep[:, :hq * d], keep[:, hq * d + 8:(hq + hk) * d + 8] = qo, ko
    assert torch.equal(xd, keep)


# -------------------------------------------------------------------- cache

def make_batch(g, lens, new, block, width_extra=0, n_extra=3):
    """Block table (every used block its own, shuffled), cu and lens."""
    used = [-(-max(n, 0) // block) for n in lens]
    total = sum(used) + n_extra
    order = g.permutation(total)
    table = np.full((len(lens), max(used + [1]) + width_extra), -1, dtype=np.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return torch.from_numpy(table), [int(x) for x in cu], total


def random_cache(g, n, h, block, d, nan_codes=False):
    """A cache with any codes (NaN ones too if asked) and scales near 1."""
    def codes(*shape):
        c = g.integers(0, 256, shape).astype(np.uint8)
        if not nan_codes:
            c[c & 127 == 127] = 0x30
        return torch.from_numpy(c)
    return {"k": codes(n, h, block, d), "v": codes(n, h, d, block),
            "ks": torch.from_numpy(g.integers(117, 122, (n, h)).astype(np.uint8)),
            "vs": torch.from_numpy(g.integers(117, 122, (n, h)).astype(np.uint8))}


def to_gpu(lib, c):
    return lib.Fp8KvCache(*(c[x].cuda() for x in ("k", "v", "ks", "vs")))


def same_cache(dev, ref):
    for t, x in zip(dev, ("k", "v", "ks", "vs")):
        assert torch.equal(t.cpu(), ref[x]), (x, int((t.cpu() != ref[x]).sum()))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


CACHE_BATCHES = [([1], [1]), ([5, 64, 65], [1, 1, 1]), ([7, 0, 200, 16], [7, 0, 130, 0]), ([128, 129, 40], [128, 3, 39]),
                 ([300], [300]), ([31, 33, 1, 2], [16, 17, 1, 2])]


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d,h", [(64, 3), (128, 2)])
@pytest.mark.parametrize("lens,new", CACHE_BATCHES)
def test_append_and_read(gpu_lib, lens, new, d, h, block):
    print("cache", lens, new, d, h, block, flush=True)
    g = gen(7, d, block, len(lens), lens[0])
    table, cu, n = make_batch(g, lens, new, block)
    ref = random_cache(g, n, h, block, d)
    T = cu[-1] + 2                                           # two rows behind the last sequence
    size = torch.from_numpy((2.0 ** g.integers(-12, 6, (T, h, 1))).astype(np.float32))
    k = (bf16(g, T, h, d).float() * size).to(torch.bfloat16)
    v = (bf16(g, T, h, d).float() * size).to(torch.bfloat16)
    dev = to_gpu(gpu_lib, ref)
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    R.append(ref, k, v, table, lens, cu)
    same_cache(dev, ref)
    # again with the same rows: the exponents have grown already
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    R.append(ref, k, v, table, lens, cu)
    same_cache(dev, ref)
    # read whole sequences back
    cu_all = [0] + [int(x) for x in np.cumsum(lens)]
    buf = torch.full((2, cu_all[-1] + 1, h * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.kv_cache_read_fp8(dev, table.cuda(), ints(lens), ints(cu_all), cu_all[-1] + 1, k_out=buf[0, :, :h * d],
                              v_out=buf[1, :, :h * d])
    want = torch.full(buf.shape, 7.0, dtype=torch.bfloat16)
    for s, n_s in enumerate(lens):
        kk, vv, held = R.held_values(ref, table, s, n_s)
        assert bool(held.all())
        want[0, cu_all[s]:cu_all[s + 1], :h * d] = kk.reshape(n_s, h * d).to(torch.bfloat16)
        want[1, cu_all[s]:cu_all[s + 1], :h * d] = vv.reshape(n_s, h * d).to(torch.bfloat16)
    assert torch.equal(buf.cpu(), want)


def test_append_token_by_token(gpu_lib):
    """A sequence grown one token at a time, with sizes that make the exponent
    grow at some and not at others; values of every bf16 exponent."""
    g = gen(8)
    h, d, block, total = 2, 64, 16, 40
    table, _, n = make_batch(g, [total], [total], block)
    ref = random_cache(g, n, h, block, d, nan_codes=True)
    dev = to_gpu(gpu_lib, ref)
    for i in range(total):
        k = (bf16(g, 1, h, d).float() * 2.0 ** int(g.integers(-40, 40))).to(torch.bfloat16)
        v = (bf16(g, 1, h, d).float() * 2.0 ** int(g.integers(-4, 4))).to(torch.bfloat16)
        if i == 7:
            k.zero_()
        gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints([i + 1]), ints([0, 1]))
        R.append(ref, k, v, table, [i + 1], [0, 1])
        same_cache(dev, ref)


@pytest.mark.parametrize("S", [64, 65, 129, 300, 4200])
def test_append_to_many_sequences(gpu_lib, S):
    """Sequences found among more than a wave has lanes, some without rows."""
    print("append many", S, flush=True)
    g = gen(27, S)
    h, d, block = 1, 64, 16
    lens = [int(x) for x in g.integers(0, 40, S)]
    new = [min(n, int(x)) for n, x in zip(lens, g.integers(0, 3, S))]
    table, cu, n = make_batch(g, lens, new, block)
    ref = random_cache(g, n, h, block, d)
    k, v = bf16(g, cu[-1], h, d), bf16(g, cu[-1], h, d)
    dev = to_gpu(gpu_lib, ref)
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    R.append(ref, k, v, table, lens, cu)
    same_cache(dev, ref)


def test_append_leaves_out_what_is_not_held(gpu_lib):
    """Table entries outside the cache, positions past the table and below
    zero: their rows are left out, and nothing else is touched."""
    g = gen(9)
    h, d, block = 2, 128, 32
    lens, new = [100, 90, 5, 40], [70, 90, 9, 40]
    table, cu, n = make_batch(g, lens, new, block)
    table = table[:, :3].contiguous()                        # positions 96 .. of the first: past the table
    table[1, 1], table[3, 0] = n, -7
    ref = random_cache(g, n, h, block, d)
    k, v = bf16(g, cu[-1], h, d), bf16(g, cu[-1], h, d)
    dev = to_gpu(gpu_lib, ref)
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    R.append(ref, k, v, table, lens, cu)
    same_cache(dev, ref)
    # malformed row offsets stay inside the batch's rows (which rows are then
    # written is not defined; that nothing outside the cache is touched shows in
    # the canaries around it)
    big = torch.full((dev.k.numel() + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    inner = big[256:-256].view(dev.k.shape)
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev._replace(k=inner), table.cuda(), ints(lens),
                                ints([-5, 300, 20, 1 << 30, 7]))
    assert bool((big[:256] == 0xA5).all()) and bool((big[-256:] == 0xA5).all())


# ---------------------------------------------------------------- attention

def attend(lib, g, lens, new, hq, h, d, block, window=0, scale=None, table=None, nan_codes=False, tail=0, extra=1):
    auto, cu, n = make_batch(g, lens, new, block, width_extra=extra)
    table = auto if table is None else table(auto, n)
    ref = random_cache(g, n, h, block, d, nan_codes=nan_codes)
    if nan_codes:
        # finite where a sequence holds a token, NaN codes elsewhere
        ok = {x: torch.zeros_like(ref[x], dtype=torch.bool) for x in "kv"}
        for s, length in enumerate(lens):
            for i in range(-(-length // block)):
                b = int(table[s, i]) if i < table.shape[1] else -1
                if 0 <= b < n:
                    ok["k"][b, :, :length - i * block] = True
                    ok["v"][b, :, :, :length - i * block] = True
        for x in "kv":
            bad = ref[x] & 127 == 127
            ref[x][bad & ok[x]] = 0x30
            ref[x][~ok[x]] = 0x7F
    T = cu[-1] + tail
    q = bf16(g, T, hq, d)
    sc = d ** -0.5 if scale is None else scale
    want, tol = R.attention(q, ref, table, lens, cu, sc, window)
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dev = to_gpu(lib, ref)
    args = (q.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    got = lib.attention_fp8_kv(*args, scale=scale, window=window, out=out).cpu().double()
    if tail:
        assert bool((got[cu[-1]:] == 7.0).all())
        got, want, tol = got[:cu[-1]], want[:cu[-1]], tol[:cu[-1]]
    off = (got - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).nan_to_num(1e9).max())
    return args, out


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,h,d", [(8, 1, 128), (6, 2, 64), (3, 3, 128), (16, 2, 64), (20, 1, 128)])
@pytest.mark.parametrize("window", [0, 50])
def test_attention_single_tokens(gpu_lib, hq, h, d, block, window):
    print("attend", hq, h, d, block, window, flush=True)
    for width in (1, 2100):                                  # a table that keeps them in one launch, and one that does not
        attend(gpu_lib, gen(10, hq, d, block, window), [1, 2, 63, 64, 65, 130, 517, 16], [1] * 8, hq, h, d, block, window,
               nan_codes=True, extra=-(-width // block))


@pytest.mark.parametrize("lens,new", [([70, 33, 5], [2, 3, 5]), ([200, 17, 0, 1, 129], [4, 0, 0, 1, 100]),
                                      ([130], [130]), ([400, 40, 300], [33, 40, 1]), ([257, 90], [200, 64])])
@pytest.mark.parametrize("hq,h,d,block", [(8, 2, 128, 64), (4, 4, 64, 16), (6, 2, 128, 32)])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_rows(gpu_lib, lens, new, hq, h, d, block, window):
    print("attend rows", lens, new, hq, h, d, block, window, flush=True)
    for width in (1, 2100):
        attend(gpu_lib, gen(11, len(lens), lens[0], hq, d, window), lens, new, hq, h, d, block, window, nan_codes=True, tail=3,
               extra=-(-width // block))


@pytest.mark.parametrize("lens,new", [([1500, 40, 1100], [200, 1, 90]), ([1300, 1200], [150, 130]), ([1030, 1, 5], [1, 1, 0]),
                                      ([1100, 1080, 1], [70, 66, 1])])
@pytest.mark.parametrize("hq,h,d,block", [(4, 2, 128, 64), (8, 1, 64, 32)])
@pytest.mark.parametrize("width", [1, 9000])
def test_attention_prompts_over_a_long_table(gpu_lib, lens, new, hq, h, d, block, width):
    """Batches whose sequences go to two kernels (a wide table), or to one of them alone."""
    print("attend long table", lens, new, hq, h, d, block, width, flush=True)
    attend(gpu_lib, gen(18, len(lens), lens[0], new[0], hq), lens, new, hq, h, d, block, 0, tail=1, extra=-(-width // block),
           nan_codes=width > 1)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_prompts_that_fill_the_chip(gpu_lib, d):
    """So many row tiles that a workgroup has one set of waves and no split."""
    print("attend many tiles", d, flush=True)
    g = gen(23, d)
    lens = [int(x) for x in g.integers(66, 200, 18)]
    attend(gpu_lib, g, lens, [min(n, 66 + i) for i, n in enumerate(lens)], 32, 32, d, 32, tail=1, nan_codes=True)


@pytest.mark.parametrize("width", [1, 9000])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_short_tiles_beside_prompts(gpu_lib, d, width):
    """Tiles of 1 to 33 rows, also the last of a prompt, in batches whose tiles are
    split over the tokens and in ones that are not; a hole in one of them."""
    print("attend short tiles", d, width, flush=True)
    def hole(t, n):
        t = t.clone()
        t[2, 1] = -1
        return t
    attend(gpu_lib, gen(24, d, width), [900, 333, 700, 65, 1, 130], [129, 1, 16, 2, 1, 130], 1, 1, d, 64, tail=1, nan_codes=True, table=hole,
           extra=-(-width // 64))
    lens = [900, 333, 700, 65, 1, 130, 600, 600, 20, 640, 70, 200]
    attend(gpu_lib, gen(25, d, width), lens, [69, 1, 4, 2, 1, 130, 8, 9, 3, 70, 70, 65], 16, 4, d, 16, nan_codes=True, table=hole, window=250,
           extra=-(-width // 16))


@pytest.mark.parametrize("window", [100, 700])
@pytest.mark.parametrize("hq,h,d", [(4, 2, 128), (8, 1, 64)])
def test_attention_short_window_in_a_long_table(gpu_lib, hq, h, d, window):
    """A window that keeps a batch with short sequences in one kernel, and a
    single sequence whose rows see too little to be split far."""
    print("attend window", hq, d, window, flush=True)
    attend(gpu_lib, gen(21, hq, window), [1500, 1203, 1100, 40], [200, 1, 90, 3], hq, h, d, 64, window, tail=2, nan_codes=True)
    attend(gpu_lib, gen(22, hq, window), [2000], [70], hq, h, d, 16, window)


def test_attention_many_sequences(gpu_lib):
    """More sequences than a wave has lanes, some without rows."""
    g = gen(19)
    lens = [int(x) for x in g.integers(1, 90, 150)]
    new = [int(x) for x in g.integers(0, 2, 150)]
    attend(gpu_lib, g, lens, new, 4, 2, 64, 16, tail=2)
    attend(gpu_lib, g, lens, new, 4, 2, 64, 16, tail=2, extra=130)
    lens = [int(x) for x in g.integers(1, 40, 300)]
    new = [int(x) for x in g.integers(0, 2, 300)]
    attend(gpu_lib, g, lens, new, 2, 1, 64, 16, tail=1, nan_codes=True, extra=200)   # one launch
    attend(gpu_lib, g, lens, new, 2, 1, 64, 16, tail=1, extra=300)                   # the decode kernel
    lens = [int(x) for x in g.integers(20, 60, 70)]
    attend(gpu_lib, g, lens, [int(x) for x in g.integers(0, 20, 70)], 8, 2, 128, 16, window=30)


def test_attention_long_sequence(gpu_lib):
    attend(gpu_lib, gen(12), [9000], [1], 8, 2, 128, 64)
    attend(gpu_lib, gen(13), [6001, 3], [2, 3], 4, 1, 64, 16, window=5000)


def test_attention_rows_that_see_nothing(gpu_lib):
    """Blocks that are not held (evicted or never given), more rows than tokens,
    a sequence of no length: zeros, and no NaN from what lies there."""
    def holes(t, n):
        t = t.clone()
        t[0, :] = -1                        # nothing held at all
        t[1, 1] = n + 5                     # a hole in the middle
        t[2, 0] = -1                        # the first rows of it see nothing
        return t
    for extra in (1, 140):
        attend(gpu_lib, gen(14), [40, 100, 60, 0, 3], [3, 2, 60, 2, 6], 4, 2, 128, 32, table=holes, nan_codes=True, extra=extra)
        attend(gpu_lib, gen(15), [40, 100, 60, 0, 3], [3, 2, 60, 2, 6], 4, 2, 64, 16, table=holes, nan_codes=True, window=20, extra=extra)
        attend(gpu_lib, gen(26), [40, 100, 60, 0, 3], [3, 2, 1, 2, 6], 4, 2, 64, 16, table=holes, nan_codes=True, extra=extra)


@pytest.mark.parametrize("lens,new", [([200], [1]), ([200, 200], [1, 1]), ([200, 180], [120, 100]), ([1300, 1200], [100, 120])])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_value_scales_far_apart(gpu_lib, lens, new, d):
    """Neighbouring blocks whose value and key exponents differ by many powers
    of two, and a block of zeros at the smallest exponent: a token's share of
    the sum must not depend on its value exponent."""
    print("attend scales", lens, new, d, flush=True)
    g = gen(16, d)
    h, block = 2, 32
    table, cu, n = make_batch(g, lens, new, block, width_extra=70 if lens == [200] else 0)
    ref = random_cache(g, n, h, block, d)
    for s in range(len(lens)):
        for i in range(-(-lens[s] // block)):
            ref["vs"][int(table[s, i])] = [105, 140, 100, 127, 90, 150, 120][i % 7]
            ref["ks"][int(table[s, i])] = [120, 119, 110, 118, 120, 121, 117][i % 7]
        ref["v"][int(table[s, 0])] = 0
    q = bf16(g, cu[-1], 4, d)
    want, tol = R.attention(q, ref, table, lens, cu, d ** -0.5, 0)
    got = gpu_lib.attention_fp8_kv(q.cuda(), to_gpu(gpu_lib, ref), table.cuda(), ints(lens), ints(cu)).cpu().double()
    off = (got - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).nan_to_num(1e9).max())


@pytest.mark.parametrize("lens,new", [([40, 70, 300], [1, 1, 1]), ([300, 70], [40, 1]), ([200, 300], [130, 200])])
@pytest.mark.parametrize("width", [1, 2100, 9000])
def test_rows_before_the_first_sequence(gpu_lib, lens, new, width):
    """Row offsets that do not begin at 0: the rows before belong to nobody."""
    print("rows before", lens, new, width, flush=True)
    g = gen(28, lens[0], width)
    h, d, block, skip = 2, 64, 16, 37
    table, cu, n = make_batch(g, lens, new, block, width_extra=-(-width // block))
    cu = [c + skip for c in cu]
    ref = random_cache(g, n, h, block, d)
    k, v, q = bf16(g, cu[-1] + 1, h, d), bf16(g, cu[-1] + 1, h, d), bf16(g, cu[-1] + 1, 8, d)
    dev = to_gpu(gpu_lib, ref)
    gpu_lib.kv_cache_append_fp8(k.cuda(), v.cuda(), dev, table.cuda(), ints(lens), ints(cu))
    R.append(ref, k, v, table, lens, cu)
    same_cache(dev, ref)
    want, tol = R.attention(q, ref, table, lens, cu, d ** -0.5, 0)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = gpu_lib.attention_fp8_kv(q.cuda(), dev, table.cuda(), ints(lens), ints(cu), out=out).cpu().double()
    assert bool((got[:skip] == 7.0).all()) and bool((got[cu[-1]:] == 7.0).all())
    assert bool(((got - want).abs() <= tol)[skip:cu[-1]].all())
    back = torch.full((2, cu[-1] + 1, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.kv_cache_read_fp8(dev, table.cuda(), ints(lens), ints(cu), cu[-1] + 1, k_out=back[0], v_out=back[1])
    assert bool((back[:, :skip] == 7.0).all()) and bool((back[:, cu[-1]:] == 7.0).all()) and not bool((back[:, skip:cu[-1]] == 7.0).all())


def test_attention_scale_and_deterministic(gpu_lib):
    args, out = attend(gpu_lib, gen(17), [700, 300, 90], [1, 1, 1], 16, 2, 128, 64, scale=0.3)
    again = [gpu_lib.attention_fp8_kv(*args, scale=0.3) for _ in range(3)]
    assert all(torch.equal(out, x) for x in again)
