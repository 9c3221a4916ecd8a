"""GPU: the attention layer's operators run together as a layer runs them, in
captured graphs, on other streams, with strided tensors, and their refusals of
tensors. Every stage is compared with its float64 form (layer_ref) on the
inputs it was given."""
import numpy as np
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HK, D, BLOCK, ROPE, MAX_POS = 512, 4, 2, 128, 32, 64, 400


def gen(*key):
    return np.random.default_rng([78, *key])


def bf16(g, *shape, scale=1.0):
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    """One attention layer and its cache, of the package's calls."""

    def __init__(self, lib, g, blocks):
        self.lib = lib
        n = (HQ + 2 * HK) * D
        self.wqkv, self.wqkv_s = lib.fp8_quant_weight_128x128_ue8m0(bf16(g, n, HIDDEN, scale=0.05).cuda())
        self.wo, self.wo_s = lib.fp8_quant_weight_128x128_ue8m0(bf16(g, HIDDEN, HQ * D, scale=0.05).cuda())
        self.qw, self.kw = (bf16(g, D) + 1).cuda(), (bf16(g, D) + 1).cuda()
        self.cs = lib.rope_cos_sin_table(10000.0, MAX_POS, ROPE)
        self.cache = lib.fp8_kv_cache(blocks, HK, D, BLOCK)

    def __call__(self, x, pos, table, lens, cu, window=0):
        """The layer's output, and what each stage was given and gave."""
        lib = self.lib
        a, s = lib.fp8_quant_1x128_ue8m0(x)
        qkv = lib.fp8_gemm_1x128_128x128(a, s, self.wqkv, self.wqkv_s)
        q, k, v = qkv.split((HQ * D, HK * D, HK * D), 1)
        qr, kr = lib.qk_norm_rope(q, k, self.qw, self.kw, pos, self.cs)
        lib.kv_cache_append_fp8(kr, v, self.cache, table, lens, cu)
        o = lib.attention_fp8_kv(qr, self.cache, table, lens, cu, window=window)
        oa, os = lib.fp8_quant_1x128_ue8m0(o)
        y = lib.fp8_gemm_1x128_128x128(oa, os, self.wo, self.wo_s)
        return y, (a, s, qkv, qr, kr, o, oa, os)


def check_gemm(out, a, words, w, ws):
    """Against the product of the operands' values: the matrix cores' own bound
    (2^-9 of the largest product of every 64 columns), then the rounding."""
    A, W = R.dequant_rows(a.cpu(), words.cpu().contiguous()), R.dequant_tiles(w.cpu(), ws.cpu())
    M, K = A.shape
    ref = A @ W.T
    mf = 2.0 ** -9 * (A.abs().view(M, K // 64, 64).amax(2) @ W.abs().view(-1, K // 64, 64).amax(2).T)
    assert bool(((out.cpu().double() - ref).abs() <= mf + 2.0 ** -8 * (ref.abs() + mf)).all())


def check_codes(a, words, x):
    """Quantised rows: off by half a step of E4M3, 2^-4 of the value, or half of
    the smallest step, 2^-10 of the block's scale."""
    got, x = R.dequant_rows(a.cpu(), words.cpu().contiguous()), x.cpu().double()
    b = torch.stack([(words.cpu().contiguous().long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, : x.shape[1] // 128]
    step = (2.0 ** (b.double() - 127 - 10)).repeat_interleave(128, 1)
    assert bool(((got - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), step)).all())


def check_step(layer, ref, x, pos, table, lens, cu, y, st, window=0):
    """Every stage of one step; ref, the cache on the CPU, follows."""
    a, s, qkv, qr, kr, o, oa, os = st
    M = x.shape[0]
    check_codes(a, s, x)
    check_gemm(qkv, a, s, layer.wqkv, layer.wqkv_s)
    q, k, v = qkv.cpu().split((HQ * D, HK * D, HK * D), 1)
    for got, src, w, h in ((qr, q, layer.qw, HQ), (kr, k, layer.kw, HK)):
        want, tol = R.norm_rope(src.reshape(M, h, D), w.cpu(), pos.cpu(), layer.cs.cpu(), 1e-6, False)
        assert bool(((got.cpu().double().view(M, h, D) - want).abs() <= tol).all())
    R.append(ref, kr.cpu().view(M, HK, D), v.reshape(M, HK, D), table, lens, cu)
    for t, n in zip(layer.cache, ("k", "v", "ks", "vs")):
        assert torch.equal(t.cpu(), ref[n]), n
    want, tol = R.attention(qr.cpu().view(M, HQ, D), ref, table, lens, cu, D ** -0.5, window)
    assert bool(((o.cpu().double().view(M, HQ, D) - want).abs() <= tol).all())
    check_codes(oa, os, o)
    check_gemm(y, oa, os, layer.wo, layer.wo_s)


def positions(lens, cu):
    return torch.tensor([lens[s] - (cu[s + 1] - cu[s]) + i for s in range(len(lens)) for i in range(cu[s + 1] - cu[s])])


@pytest.mark.parametrize("window", [0, 37])
def test_layer_prompt_then_decode(gpu_lib, window):
    """Three ragged prompts, then single tokens, then a drafted pair for one
    sequence beside a sequence that rests, all over one cache."""
    print("layer", window, flush=True)
    g = gen(1, window)
    layer = Layer(gpu_lib, g, 14)
    table = torch.from_numpy(g.permutation(14)[:12].reshape(3, 4).astype(np.int32))
    ref = {n: t.cpu().clone() for n, t in zip(("k", "v", "ks", "vs"), layer.cache)}
    lens = [0, 0, 0]
    for new in ([70, 5, 33], [1, 1, 1], [1, 1, 1], [2, 0, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        cu = [0] + [int(c) for c in np.cumsum(new)]
        x, pos = bf16(g, cu[-1], HIDDEN).cuda(), positions(lens, cu).cuda()
        y, st = layer(x, pos, table.cuda(), ints(lens), ints(cu), window)
        check_step(layer, ref, x, pos, table, lens, cu, y, st, window)


def test_layer_in_graphs(gpu_lib):
    """A decode step and a padded mixed step captured once each and replayed with
    other tokens, lengths and row offsets, eager work between the replays; every
    replay against the eager layer on a cache of its own."""
    g = gen(2)
    eager, captured = Layer(gpu_lib, gen(3), 14), Layer(gpu_lib, gen(3), 14)
    table = torch.from_numpy(gen(4).permutation(14)[:12].reshape(3, 4).astype(np.int32)).cuda()
    start = [60, 5, 31]
    cu0 = [0] + [int(c) for c in np.cumsum(start)]
    x = bf16(g, cu0[-1], HIDDEN).cuda()
    for layer in (eager, captured):
        layer(x, positions(start, cu0).cuda(), table, ints(start), ints(cu0))
    steps = {}
    for name, rows in (("decode", 3), ("mixed", 40)):
        buf = dict(x=bf16(g, rows, HIDDEN).cuda(), pos=torch.zeros(rows, dtype=torch.int64, device="cuda"), lens=ints([0, 0, 0]),
                   cu=ints([0, 0, 0, 0]))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            captured(buf["x"], buf["pos"], table, buf["lens"], buf["cu"])      # no rows: the cache stays as it is
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, st = captured(buf["x"], buf["pos"], table, buf["lens"], buf["cu"])
        steps[name] = (graph, buf, y, st)
    lens = list(start)
    for name, new in (("decode", [1, 1, 1]), ("mixed", [20, 0, 17]), ("decode", [1, 0, 1]), ("mixed", [1, 39, 0]), ("mixed", [3, 1, 1]),
                      ("decode", [1, 1, 1]), ("decode", [1, 1, 1])):
        graph, buf, y, st = steps[name]
        lens = [a + b for a, b in zip(lens, new)]
        cu = [0] + [int(c) for c in np.cumsum(new)]
        n = cu[-1]
        x = bf16(g, n, HIDDEN).cuda()
        pos = positions(lens, cu).cuda()
        want, ws = eager(x, pos, table, ints(lens), ints(cu))
        torch.cuda.synchronize()
        buf["x"][:n].copy_(x)
        buf["pos"][:n].copy_(pos)
        buf["lens"].copy_(ints(lens))
        buf["cu"].copy_(ints(cu))
        graph.replay()
        torch.cuda.synchronize()
        # (the attention of a padded step may take other kernels: the same to rounding)
        assert torch.equal(st[2][:n], ws[2]) and torch.equal(st[3][:n], ws[3]) and torch.equal(st[4][:n], ws[4]), name
        for t, r in zip(captured.cache, eager.cache):
            assert torch.equal(t, r)
        ref = {k: t.cpu() for k, t in zip(("k", "v", "ks", "vs"), captured.cache)}
        exp, tol = R.attention(st[3][:n].cpu().view(n, HQ, D), ref, table.cpu(), lens, cu, D ** -0.5, 0)
        assert bool(((st[5][:n].cpu().double().view(n, HQ, D) - exp).abs() <= tol).all()), name
        check_gemm(y[:n], st[6][:n], st[7][:n], captured.wo, captured.wo_s)
        assert want.shape == (n, HIDDEN)


def test_two_graphs_share_a_workspace(gpu_lib):
    """Attention and split products of two graphs over one workspace each,
    replayed in turn."""
    g = gen(5)
    cache = gpu_lib.fp8_kv_cache(40, 2, 128, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    lens, cu = ints([1200, 900]), ints([0, 1200, 2100])
    gpu_lib.kv_cache_append_fp8(bf16(g, 2100, 2, 128).cuda(), bf16(g, 2100, 2, 128).cuda(), cache, table, lens, cu)
    a, s = gpu_lib.fp8_quant_1x128_ue8m0(bf16(g, 100, 4096).cuda())
    w, ws = gpu_lib.fp8_quant_weight_128x128_ue8m0(bf16(g, 256, 4096).cuda())
    space = gpu_lib.attention_fp8_kv_workspace(128)
    gspace = torch.empty(gpu_lib.fp8_gemm_workspace_bytes(100, 256, 4096), dtype=torch.uint8, device="cuda")
    assert gspace.numel() > 0
    runs = []
    for rows in ([0, 1, 2], [0, 80, 100]):
        q = bf16(g, rows[-1], 8, 128).cuda()
        m = max(65, rows[-1])

        def call(q=q, rows=ints(rows), m=m):
            return (gpu_lib.attention_fp8_kv(q, cache, table, lens, rows, workspace=space),
                    gpu_lib.fp8_gemm_1x128_128x128(a[:m], s[:m], w, ws, workspace=gspace))
        want = [t.clone() for t in call()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        runs.append((graph, got, want, call))                # (call holds the inputs that the graph reads)
    for turn in range(3):
        for graph, got, want, _ in runs:
            for t in got:
                t.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            for t, r in zip(got, want):
                assert torch.equal(t, r), turn


def test_stream_argument(gpu_lib):
    """stream=: the launch and the outputs are that stream's, whatever is
    current; calls on two streams at once."""
    g = gen(6)
    layer = Layer(gpu_lib, g, 14)
    table = ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    lens, cu = ints([100, 40]), ints([0, 100, 140])
    x = bf16(g, 140, HIDDEN).cuda()
    pos = positions([100, 40], [0, 100, 140]).cuda()
    y, (a, s, qkv, qr, kr, o, oa, os) = layer(x, pos, table, lens, cu)
    k2, v2 = gpu_lib.kv_cache_read_fp8(layer.cache, table, lens, cu, 140)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        other = gpu_lib.fp8_kv_cache(14, HK, D, BLOCK)
        st.wait_stream(torch.cuda.current_stream())
        p = gpu_lib.fp8_gemm_1x128_128x128(a, s, layer.wqkv, layer.wqkv_s, stream=st)
        q, k, v = p.split((HQ * D, HK * D, HK * D), 1)
        r = gpu_lib.qk_norm_rope(q, k, layer.qw, layer.kw, pos, layer.cs, stream=st)
        assert gpu_lib.kv_cache_append_fp8(r[1], v, other, table, lens, cu, stream=st) is other
        e = gpu_lib.attention_fp8_kv(r[0], other, table, lens, cu, stream=st)
        outs.append((p, *r, e, *gpu_lib.kv_cache_read_fp8(other, table, lens, cu, 140, stream=st)))
    torch.cuda.synchronize()
    for got in outs:
        for t, ref in zip(got, (qkv, qr, kr, o, k2, v2)):
            assert torch.equal(t, ref)


def test_strided_rows(gpu_lib):
    """k, v, q and out as column ranges of wider rows; a block table with padded
    rows; nothing outside out is touched."""
    g = gen(7)
    h, hq, d = 2, 6, 64
    lens, cu = [90, 33, 70], [0, 20, 21, 60]
    table = torch.full((3, 9), 99, dtype=torch.int32)
    table[:, 2:8] = torch.from_numpy(g.permutation(18).reshape(3, 6).astype(np.int32))
    inner = table.cuda()[:, 2:8]
    ref = {"k": torch.full((18, h, 16, d), 0x20, dtype=torch.uint8), "v": torch.full((18, h, d, 16), 0x20, dtype=torch.uint8),
           "ks": torch.full((18, h), 120, dtype=torch.uint8), "vs": torch.full((18, h), 120, dtype=torch.uint8)}
    dev = gpu_lib.Fp8KvCache(*(ref[n].cuda() for n in ("k", "v", "ks", "vs")))
    wide = bf16(g, 60, (hq + 2 * h) * d + 40)
    at = (8, 8 + hq * d + 8, 8 + hq * d + 8 + h * d + 16)
    wd = wide.cuda()
    q, k, v = wd[:, at[0]:at[0] + hq * d], wd[:, at[1]:at[1] + h * d], wd[:, at[2]:at[2] + h * d]
    gpu_lib.kv_cache_append_fp8(k, v, dev, inner, ints(lens), ints(cu))
    R.append(ref, k.cpu().reshape(60, h, d), v.cpu().reshape(60, h, d), table[:, 2:8], lens, cu)
    for t, n in zip(dev, ("k", "v", "ks", "vs")):
        assert torch.equal(t.cpu(), ref[n]), n
    want, tol = R.attention(q.cpu().reshape(60, hq, d), ref, table[:, 2:8], lens, cu, d ** -0.5, 0)
    buf = torch.full((62, hq * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:61, 8:8 + hq * d]
    assert gpu_lib.attention_fp8_kv(q, dev, inner, ints(lens), ints(cu), out=out) is out
    off = (out.cpu().double().view(60, hq, d) - want).abs()
    assert bool((off <= tol).all())
    out.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_offsets_past_32_bits(gpu_lib):
    """Blocks whose codes lie beyond 2^32 bytes: as in a small cache."""
    g = gen(8)
    h, d, block, n = 8, 128, 128, 36000                       # 4.7 GB of keys, as much of values
    far = [n - 1, 33001, 32768, n - 7, 34000, 17]             # from 32768 on: past 2^32 bytes
    big = gpu_lib.Fp8KvCache(torch.empty((n, h, block, d), dtype=torch.uint8, device="cuda"),
                             torch.empty((n, h, d, block), dtype=torch.uint8, device="cuda"),
                             torch.zeros((n, h), dtype=torch.uint8, device="cuda"), torch.zeros((n, h), dtype=torch.uint8, device="cuda"))
    small = gpu_lib.fp8_kv_cache(6, h, d, block)
    for t, s in zip(big, small):
        t[far] = s
    tables = ints([far[:3], far[3:]]), ints([[0, 1, 2], [3, 4, 5]])
    for lens, new in (([300, 250], [300, 250]), ([301, 251], [1, 1]), ([380, 255], [79, 4])):
        cu = [0, new[0], new[0] + new[1]]
        k, v, q = bf16(g, cu[-1], h, d).cuda(), bf16(g, cu[-1], h, d).cuda(), bf16(g, cu[-1], h, d).cuda()
        outs = []
        for cache, table in zip((big, small), tables):
            gpu_lib.kv_cache_append_fp8(k, v, cache, table, ints(lens), ints(cu))
            outs.append((gpu_lib.attention_fp8_kv(q, cache, table, ints(lens), ints(cu)),
                         *gpu_lib.kv_cache_read_fp8(cache, table, ints(lens), ints(cu), cu[-1])))
        for a, b in zip(*outs):
            assert torch.equal(a, b)
    for t, s in zip(big, small):
        assert torch.equal(t[far], s)


def test_attention_ignores_other_rows(gpu_lib):
    """A query row of NaN or infinities makes its own output NaN and no other,
    in both kernels."""
    g = gen(9)
    cache = gpu_lib.fp8_kv_cache(40, 1, 64, 16)
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    lens, cu = ints([300, 200]), ints([0, 300, 500])
    gpu_lib.kv_cache_append_fp8(bf16(g, 500, 1, 64).cuda(), bf16(g, 500, 1, 64).cuda(), cache, table, lens, cu)
    for rows in ([0, 1, 2], [0, 150, 270]):
        q = bf16(g, rows[-1], 4, 64).cuda()
        clean = gpu_lib.attention_fp8_kv(q, cache, table, lens, ints(rows))
        q[1, 2] = float("nan")
        q[0, 1, 5] = float("inf")
        got = gpu_lib.attention_fp8_kv(q, cache, table, lens, ints(rows))
        bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        bad[1, 2] = bad[0, 1] = True
        assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], clean[~bad])


def test_single_token_contexts_and_empty_calls(gpu_lib):
    """Lengths of one and zero, no rows, no sequences."""
    g = gen(10)
    cache = gpu_lib.fp8_kv_cache(2, 1, 64, 16)
    k, v = bf16(g, 1, 1, 64).cuda(), bf16(g, 1, 1, 64).cuda()
    gpu_lib.kv_cache_append_fp8(k, v, cache, ints([[1]]), ints([1]), ints([0, 1]))
    rk, rv = gpu_lib.kv_cache_read_fp8(cache, ints([[1]]), ints([1]), ints([0, 1]), 1)
    out = gpu_lib.attention_fp8_kv(bf16(g, 1, 2, 64).cuda(), cache, ints([[1]]), ints([1]), ints([0, 1]))
    assert torch.equal(out[:, 0], rv[:, 0]) and torch.equal(out[:, 1], rv[:, 0])      # one token: its value
    none = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    before = [t.clone() for t in cache]
    gpu_lib.kv_cache_append_fp8(k[:0], v[:0], cache, ints([[1]]), ints([1]), ints([0, 0]))
    gpu_lib.kv_cache_append_fp8(k, v, cache, none, ints([]), ints([0]))
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
    assert gpu_lib.attention_fp8_kv(k[:0], cache, ints([[1]]), ints([1]), ints([0, 0])).shape == (0, 1, 64)
    assert gpu_lib.kv_cache_read_fp8(cache, ints([[1]]), ints([1]), ints([0, 0]), 0)[0].shape == (0, 1, 64)


def test_refusals_of_tensors(gpu_lib):
    lib = gpu_lib
    g = gen(11)
    a, s = lib.fp8_quant_1x128_ue8m0(bf16(g, 70, 256).cuda())
    w, ws = lib.fp8_quant_weight_128x128_ue8m0(bf16(g, 256, 256).cuda())
    out = torch.zeros((70, 256), dtype=torch.bfloat16, device="cuda")
    gemm = dict(a=a, a_scales=s, w=w, w_scales=ws)
    cache = lib.fp8_kv_cache(4, 2, 64, 16)
    x, table, lens, cu = bf16(g, 3, 2, 64).cuda(), ints([[0, 1], [2, 3]]), ints([5, 9]), ints([0, 1, 3])
    att = dict(q=x, cache=cache, block_table=table, seq_lens=lens, cu_rows=cu)
    app = dict(k=x, v=x, cache=cache, block_table=table, seq_lens=lens, cu_rows=cu)
    rd = dict(cache=cache, block_table=table, seq_lens=lens, cu_rows=cu, rows=3)
    wt, pos, cs = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), \
        lib.rope_cos_sin_table(10000.0, 8, 32)
    norm = dict(q=x, k=x, q_weight=wt, k_weight=wt, positions=pos, cos_sin=cs, head_dim=64)
    odd = torch.zeros((4, 2, 16, 72), dtype=torch.uint8, device="cuda")[..., :64]
    cases = [
        (lib.fp8_gemm_1x128_128x128, gemm, TypeError, [dict(a=a.float()), dict(w=w.int()), dict(a_scales=s.long()), dict(w_scales=ws.int()),
                                                      dict(out=out.float()), dict(workspace=out)]),
        (lib.fp8_gemm_1x128_128x128, gemm, ValueError, [dict(a=a.cpu()), dict(w=w.cpu()), dict(w=w[:, :128]), dict(w=w[:128]), dict(a=a[:5]),
                                                       dict(a_scales=s[:, :0]), dict(out=out[:3]), dict(out=out.t()[:70]), dict(a=a[0]),
                                                       dict(out=torch.zeros((256, 70), dtype=torch.bfloat16, device="cuda").t()),
                                                       dict(w=w.t().contiguous().t())]),
        (lib.attention_fp8_kv, att, TypeError, [dict(q=x.float()), dict(block_table=table.long()), dict(seq_lens=lens.long()),
                                                dict(cu_rows=cu.long()), dict(out=x.half()), dict(cache=cache._replace(k=cache.k.view(torch.int8))),
                                                dict(workspace=x)]),
        (lib.attention_fp8_kv, att, ValueError, [dict(q=x.cpu()), dict(q=x[:, :, :32]), dict(seq_lens=lens[:1]), dict(cu_rows=cu[:2]),
                                                 dict(out=x[:2]), dict(window=-1), dict(window=1 << 31), dict(q=bf16(g, 3, 3, 64).cuda()),
                                                 dict(cache=cache._replace(k=odd)), dict(cache=cache._replace(v=cache.k)),
                                                 dict(cache=cache._replace(k_scales=cache.k_scales[:3])),
                                                 dict(cache=cache._replace(v_scales=cache.v_scales.cpu())), dict(q=x.transpose(0, 1)),
                                                 dict(block_table=table.t()), dict(block_table=table.cpu()), dict(block_table=table[0])]),
        (lib.attention_fp8_kv, att, lib.IqpError, [dict(scale=0.0), dict(scale=-1.0), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                                                   dict(scale=float("nan"))]),
        (lib.kv_cache_append_fp8, app, TypeError, [dict(k=x.float()), dict(v=x.half())]),
        (lib.kv_cache_append_fp8, app, ValueError, [dict(k=x[:2]), dict(v=x[:, :1]), dict(v=x.cpu()), dict(cu_rows=cu[:1])]),
        (lib.kv_cache_append_fp8, app, lib.IqpError, [dict(k=torch.zeros(3 * 132, dtype=torch.bfloat16, device="cuda").as_strided((3, 128), (132, 1)))]),
        (lib.kv_cache_read_fp8, rd, ValueError, [dict(rows=-1), dict(k_out=x[:2]), dict(v_out=x.cpu()), dict(cache=cache._replace(v=cache.v.cpu()))]),
        (lib.kv_cache_read_fp8, rd, TypeError, [dict(k_out=x.float()), dict(rows="3")]),
        (lib.qk_norm_rope, norm, TypeError, [dict(q=x.float()), dict(positions=pos.int()), dict(cos_sin=cs.double()), dict(q_weight=wt.float())]),
        (lib.qk_norm_rope, norm, ValueError, [dict(k=x[:2]), dict(positions=pos[:2]), dict(k_weight=wt[:32]), dict(head_dim=128),
                                              dict(rope_layout="pairs"), dict(q_out=x[:1]), dict(cos_sin=cs.t()), dict(q=x.cpu())]),
        (lib.qk_norm_rope, norm, lib.IqpError, [dict(eps=-1.0), dict(head_dim=32, q=x.view(3, 4, 32), k=x.view(3, 4, 32), q_weight=wt[:32].clone(),
                                                                     k_weight=wt[:32].clone())]),
    ]
    for fn, good, error, bads in cases:
        fn(**good)
        for bad in bads:
            with pytest.raises(error):
                fn(**{**good, **bad})
                pytest.fail(f"{fn.__name__} took {list(bad)} it should refuse")
    with pytest.raises((ValueError, AttributeError, TypeError)):
        lib.attention_fp8_kv(**att, stream=torch.device("cpu"))
