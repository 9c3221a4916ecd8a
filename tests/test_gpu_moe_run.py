"""GPU: the operators whose weights depend on the token run together as a layer
runs them (router, products by expert, sum; a projection with adapters), in
captured graphs, on other streams, over shares of the experts, with empty
batches and with offsets past 32 bits. Every stage is compared with its float64
form (moe_ref) on the inputs it was given."""
import numpy as np
import pytest
import torch

import moe_ref as X

pytestmark = pytest.mark.gpu

HIDDEN, INTER, EXPERTS, TOP = 512, 256, 12, 3


def gen(*key):
    return np.random.default_rng([93, *key])


def experts_of(lib, g, n, rows, cols):
    pairs = [lib.fp8_quant_weight_128x128_ue8m0(X.bf16(g, rows, cols, scale=0.05).cuda()) for _ in range(n)]
    return torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])


class Moe:
    """A mixture of experts with a shared one, of the package's calls."""

    def __init__(self, lib, g, first=0, held=EXPERTS):
        self.lib, self.first, self.held = lib, first, held
        self.router = torch.from_numpy(g.standard_normal((HIDDEN, EXPERTS)).astype(np.float32) * HIDDEN ** -0.5).cuda()
        self.bias = torch.from_numpy(g.standard_normal(EXPERTS).astype(np.float32) * 0.1).cuda()
        part = slice(first, first + held)
        self.w13, self.w13_s = (t[part].contiguous() for t in experts_of(lib, g, EXPERTS, 2 * INTER, HIDDEN))
        self.w2, self.w2_s = (t[part].contiguous() for t in experts_of(lib, g, EXPERTS, HIDDEN, INTER))
        self.ws, self.ws_s = lib.fp8_quant_weight_128x128_ue8m0(X.bf16(g, HIDDEN, HIDDEN, scale=0.05).cuda())

    def __call__(self, x, shared=True):
        lib = self.lib
        logits = (x.float() @ self.router).contiguous()
        weights, experts = lib.moe_route(logits, TOP, bias=self.bias, scoring="sigmoid", scale=1.5)
        groups = lib.group_rows(experts - self.first, self.held)
        a, s = lib.fp8_quant_1x128_ue8m0(x)
        q, qs = lib.fp8_grouped_swiglu_1x128(a, s, self.w13, self.w13_s, groups, gather=True)
        y = lib.fp8_grouped_gemm_1x128_128x128(q, qs, self.w2, self.w2_s, groups)
        sh = lib.fp8_gemm_1x128_128x128(a, s, self.ws, self.ws_s) if shared else None
        return lib.moe_combine(y, groups, weights, shared=sh), (logits, weights, experts, groups, a, s, q, qs, y, sh)


def scale_bytes(words, n):
    return torch.stack([(words.cpu().contiguous().long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, :n]


def check_step(moe, out, st):
    logits, weights, experts, groups, a, s, q, qs, y, sh = st
    want, ids = X.route(logits.cpu(), TOP, moe.bias.cpu(), "sigmoid", True, 1.5)
    assert torch.equal(experts.cpu(), ids)
    assert bool(((weights.cpu().double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want).all())
    plan = X.plan(ids - moe.first, moe.held)
    for got, ref in zip(groups, plan):
        assert torch.equal(got.cpu(), ref)
    src = plan[1].long().clamp_min(0) // TOP
    v, bound = X.product(a.cpu(), scale_bytes(s, HIDDEN // 128), moe.w13.cpu(), moe.w13_s.cpu(), plan[0], src)
    X.check_swiglu(q.cpu(), qs.cpu(), v, bound)
    v, bound = X.product(q.cpu(), scale_bytes(qs, INTER // 128), moe.w2.cpu(), moe.w2_s.cpu(), plan[0], torch.arange(len(src)))
    X.check_product(y.cpu(), v, bound)
    want, tol = X.combine(y.cpu(), plan[2], weights.cpu(), None if sh is None else sh.cpu())
    assert bool(((out.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tokens", [1, 2, 9, 64, 333])
def test_layer(gpu_lib, tokens):
    print("moe layer", tokens, flush=True)
    moe = Moe(gpu_lib, gen(1))
    out, st = moe(X.bf16(gen(2, tokens), tokens, HIDDEN).cuda())
    check_step(moe, out, st)


def test_shares_of_experts(gpu_lib):
    """Two ranks with half of the experts each: what neither holds is left out, and
    the two sums are the layer's."""
    x = X.bf16(gen(3), 150, HIDDEN).cuda()
    parts = []
    for first in (0, EXPERTS // 2):
        moe = Moe(gpu_lib, gen(1), first, EXPERTS // 2)
        out, st = moe(x, shared=False)
        check_step(moe, out, st)
        parts.append(out.double())
    whole, st = Moe(gpu_lib, gen(1))(x, shared=False)
    mag = parts[0].abs() + parts[1].abs()       # three roundings to bf16, and float32 sums
    assert bool(((parts[0] + parts[1] - whole.double()).abs() <= 2.0 ** -7 * mag + 2.0 ** -8 * whole.double().abs()).all())


def test_empty_batches(gpu_lib):
    moe = Moe(gpu_lib, gen(1))
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    w, ids = gpu_lib.moe_route(e(0, EXPERTS, t=torch.float32), TOP)
    groups = gpu_lib.group_rows(ids, EXPERTS)
    assert groups.offsets.tolist() == [0] * (EXPERTS + 1) and groups.slots.shape == (0, TOP)
    a, s = e(0, HIDDEN, t=torch.uint8), e(0, 1, t=torch.int32)
    q, qs = gpu_lib.fp8_grouped_swiglu_1x128(a, s, moe.w13, moe.w13_s, groups, gather=True)
    y = gpu_lib.fp8_grouped_gemm_1x128_128x128(q, qs, moe.w2, moe.w2_s, groups)
    assert q.shape == (0, INTER) and qs.shape == (0, 1) and y.shape == (0, HIDDEN)
    assert gpu_lib.moe_combine(y, groups, w).shape == (0, HIDDEN)
    one = gpu_lib.group_rows(e(0, t=torch.int32), 4)
    out = e(0, HIDDEN)
    assert gpu_lib.lora_add(out, e(0, 64), e(4, 16, 64), e(4, HIDDEN, 16), one) is not None
    # tokens none of whose experts are held
    none = gpu_lib.group_rows(torch.full((5, TOP), -1, dtype=torch.int32, device="cuda"), EXPERTS)
    y = torch.full((15, HIDDEN), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert bool((gpu_lib.moe_combine(y, none, torch.ones(5, TOP, device="cuda")) == 0).all())


def adapters(g, n, rank, K, N):
    return X.bf16(g, n, rank, K, scale=K ** -0.5).cuda(), X.bf16(g, n, N, rank, scale=0.3).cuda(), \
        torch.from_numpy(g.random(n).astype(np.float32) + 0.5).cuda()


def test_projection_with_adapters(gpu_lib):
    """The shared product, then every request's adapter: prompts, single tokens and
    requests without one in one batch."""
    lib, g = gpu_lib, gen(4)
    N, rank, n = 384, 16, 5
    w, ws = lib.fp8_quant_weight_128x128_ue8m0(X.bf16(g, N, HIDDEN, scale=0.05).cuda())
    a, b, scales = adapters(g, n, rank, HIDDEN, N)
    lens, which = [70, 1, 1, 33, 1, 1, 5], [2, 0, -1, 2, 4, 0, -1]
    index = torch.tensor(np.repeat(which, lens).astype(np.int32), device="cuda")
    x = X.bf16(g, len(index), HIDDEN).cuda()
    q, s = lib.fp8_quant_1x128_ue8m0(x)
    base = lib.fp8_gemm_1x128_128x128(q, s, w, ws)
    groups = lib.group_rows(index, n)
    out = lib.lora_add(base.clone(), x, a, b, groups, scales=scales)
    plan = X.plan(index.cpu(), n)
    want, tol = X.lora(base.cpu(), x.cpu(), a.cpu(), b.cpu(), plan[0], plan[1], scales.cpu())
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert torch.equal(out[index < 0], base[index < 0]) and not torch.equal(out[index >= 0], base[index >= 0])


def test_in_graphs(gpu_lib):
    """A step captured once and replayed with other tokens, so other experts and
    adapters, eager work between the replays; every replay against the eager step."""
    lib, g = gpu_lib, gen(5)
    moe = Moe(lib, gen(1))
    a, b, scales = adapters(g, 4, 24, HIDDEN, HIDDEN)

    def step(x, index):
        out, st = moe(x)
        return lib.lora_add(out, x, a, b, lib.group_rows(index, 4), scales=scales), st

    for tokens in (3, 90):
        x = torch.zeros(tokens, HIDDEN, dtype=torch.bfloat16, device="cuda")
        index = torch.zeros(tokens, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x, index)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, st = step(x, index)
        for turn in range(5):
            print("moe graph", tokens, turn, flush=True)
            h = gen(6, tokens, turn)
            x.copy_(X.bf16(h, tokens, HIDDEN).cuda() * (1 + turn))
            index.copy_(torch.from_numpy(h.integers(-1, 4, tokens).astype(np.int32)))
            eager, _ = step(x.clone(), index.clone())
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (tokens, turn)


def test_streams(gpu_lib):
    """Calls on two streams at once, with stream= and with the current stream; each
    with workspaces of its own."""
    lib = gpu_lib
    moe = Moe(lib, gen(1))
    a, b, scales = adapters(gen(7), 4, 16, HIDDEN, HIDDEN)
    xs = [X.bf16(gen(8, i), 200, HIDDEN).cuda() for i in range(4)]
    index = torch.from_numpy(gen(9).integers(-1, 4, 200).astype(np.int32)).cuda()
    groups = lib.group_rows(index, 4)
    want = [moe(x)[0] for x in xs]
    want = [lib.lora_add(o.clone(), x, a, b, groups, scales=scales) for o, x in zip(want, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, x in enumerate(xs):
        with torch.cuda.stream(streams[i % 2]):
            out, _ = moe(x)
            got.append(lib.lora_add(out, x, a, b, groups, scales=scales))
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    s = streams[0]
    z = (xs[0].float() @ moe.router).contiguous()
    torch.cuda.synchronize()
    w, e = lib.moe_route(z, TOP, stream=s)
    gr = lib.group_rows(e, EXPERTS, stream=s)
    q, qs = lib.fp8_quant_1x128_ue8m0(xs[0], stream=s)
    h, hs = lib.fp8_grouped_swiglu_1x128(q, qs, moe.w13, moe.w13_s, gr, gather=True, stream=s)
    y = lib.fp8_grouped_gemm_1x128_128x128(h, hs, moe.w2, moe.w2_s, gr, stream=s)
    out = lib.moe_combine(y, gr, w, stream=s)
    lib.lora_add(out, xs[0], a, b, groups, scales=scales, stream=s)
    s.synchronize()
    w2, e2 = lib.moe_route(z, TOP)
    gr2 = lib.group_rows(e2, EXPERTS)
    q, qs = lib.fp8_quant_1x128_ue8m0(xs[0])
    h, hs = lib.fp8_grouped_swiglu_1x128(q, qs, moe.w13, moe.w13_s, gr2, gather=True)
    ref = lib.moe_combine(lib.fp8_grouped_gemm_1x128_128x128(h, hs, moe.w2, moe.w2_s, gr2), gr2, w2)
    assert torch.equal(out, lib.lora_add(ref, xs[0], a, b, groups, scales=scales))


def test_nan_stays_in_its_row(gpu_lib):
    """A NaN among one place's codes or one adapter row of x reaches no other row."""
    lib, g = gpu_lib, gen(10)
    counts, N, K = [40, 7, 200], 256, 256
    index = X.index_of(counts, g)
    plan = X.plan(index, 3)
    a, ab = X.codes(g, len(index), K), X.scale_bytes(g, len(index), K // 128)
    w, ws = X.codes(g, 3, N, K).cuda(), X.scale_bytes(g, 3, N // 128, K // 128).cuda()
    gr = lib.RowGroups(*(t.cuda() for t in plan))
    bad = a.clone()
    rows = [3, 45, 100]
    bad[rows, 9] = 0x7F
    good = lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w, ws, gr)
    got = lib.fp8_grouped_gemm_1x128_128x128(bad.cuda(), X.words_of(ab).cuda(), w, ws, gr)
    rest = torch.ones(len(index), dtype=torch.bool)
    rest[rows] = False
    assert torch.equal(got[rest.cuda()], good[rest.cuda()]) and bool(torch.isnan(got[rows].float()).all())
    good = lib.fp8_grouped_swiglu_1x128(a.cuda(), X.words_of(ab).cuda(), w, ws, gr)
    got = lib.fp8_grouped_swiglu_1x128(bad.cuda(), X.words_of(ab).cuda(), w, ws, gr)
    assert all(torch.equal(u[rest.cuda()], v[rest.cuda()]) for u, v in zip(got, good))
    la, lb, _ = adapters(g, 3, 16, K, N)
    x, base = X.bf16(g, len(index), K), X.bf16(g, len(index), N).cuda()
    bad = x.clone()
    bad[rows, 100] = float("inf")
    good = lib.lora_add(base.clone(), x.cuda(), la, lb, gr)
    got = lib.lora_add(base.clone(), bad.cuda(), la, lb, gr)
    assert torch.equal(got[rest.cuda()], good[rest.cuda()]) and not bool(torch.isfinite(got[rows].float()).any())


def test_same_bits_again(gpu_lib):
    moe = Moe(gpu_lib, gen(1))
    x = X.bf16(gen(11), 777, HIDDEN).cuda()
    first, _ = moe(x)
    for _ in range(3):
        assert torch.equal(moe(x)[0], first)


# ------------------------------------------------------- offsets past 32 bits

def test_output_past_32_bits(gpu_lib):
    """An output of more than 2^32 bytes: rows on both sides of the border against
    the same rows computed alone."""
    lib, g = gpu_lib, gen(12)
    n, N, K = 270000, 8200, 128
    assert n * N * 2 > 1 << 32
    index = torch.from_numpy((np.arange(n) >= 100).astype(np.int32) + (np.arange(n) >= n - 50)).cuda()
    gr = lib.group_rows(index, 3)
    a, words = torch.randint(0, 120, (n, K), dtype=torch.uint8, device="cuda"), torch.full((n, 1), 127, dtype=torch.int32, device="cuda")
    w, ws = X.codes(g, 3, N, K).cuda(), torch.full((3, -(-N // 128), 1), 127, dtype=torch.uint8, device="cuda")
    out = lib.fp8_grouped_gemm_1x128_128x128(a, words, w, ws, gr)
    border = (1 << 32) // (2 * N)
    for lo, hi in ((0, 100), (border - 40, border + 40), (n - 50, n)):
        e = int(index[lo])
        one = lib.group_rows(torch.zeros(hi - lo, dtype=torch.int32, device="cuda"), 1)
        want = lib.fp8_grouped_gemm_1x128_128x128(a[lo:hi], words[lo:hi], w[e:e + 1], ws[e:e + 1], one)
        assert torch.allclose(out[lo:hi].float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * float(want.float().abs().max()))
    # the sum of rows behind the border, and adapters on an output of that size
    groups = lib.RowGroups(torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"),
                           torch.arange(n, dtype=torch.int32, device="cuda"))
    pick = lib.RowGroups(groups.offsets, groups.rows, torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda").view(n // 2, 2))
    got = lib.moe_combine(out, pick, torch.ones(n // 2, 2, device="cuda"))
    want = (out[n - 1].float() + out[n - 2].float()).to(torch.bfloat16)
    assert torch.equal(got[0], want)
    del got
    x = torch.randn(n, 64, device="cuda").to(torch.bfloat16)
    la, lb, _ = adapters(g, 3, 8, 64, N)
    before = out[border - 5:border + 5].clone()
    lib.lora_add(out, x, la, lb, gr)
    h = x[border - 5:border + 5].float() @ la[1].float().t().contiguous()
    want = before.float() + h @ lb[1].float().t().contiguous()
    assert torch.allclose(out[border - 5:border + 5].float(), want, rtol=2.0 ** -7, atol=1e-3 * float(want.abs().max()))


def test_weights_past_32_bits(gpu_lib):
    """Groups whose weights lie 3 GiB apart."""
    lib, g = gpu_lib, gen(13)
    N, K, far = 300, 256, 3 << 30
    buf = torch.zeros(2 * far + N * K, dtype=torch.uint8, device="cuda")
    w = buf.as_strided((3, N, K), (far, K, 1))
    counts = [5, 40, 9]
    index = X.index_of(counts, g)
    plan = X.plan(index, 3)
    wc = X.codes(g, 3, N, K)
    w.copy_(wc)
    a, ab = X.codes(g, len(index), K), X.scale_bytes(g, len(index), K // 128)
    ws = X.scale_bytes(g, 3, -(-N // 128), K // 128)
    out = lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w, ws.cuda(), lib.RowGroups(*(t.cuda() for t in plan)))
    y, bound = X.product(a, ab, wc, ws, plan[0], torch.arange(len(index)))
    X.check_product(out.cpu(), y, bound)


# ------------------------------------------------------------------- refusals

def test_refusals_of_tensors(gpu_lib):
    lib = gpu_lib
    z = torch.zeros(6, 8, device="cuda")
    i = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    gr = lib.group_rows(i, 3)
    codes, words = torch.zeros(12, 256, dtype=torch.uint8, device="cuda"), torch.zeros(12, 1, dtype=torch.int32, device="cuda")
    w, ws = torch.zeros(3, 256, 256, dtype=torch.uint8, device="cuda"), torch.zeros(3, 2, 2, dtype=torch.uint8, device="cuda")
    b = torch.zeros(12, 64, dtype=torch.bfloat16, device="cuda")
    one = lib.group_rows(torch.zeros(12, dtype=torch.int32, device="cuda"), 3)
    la, lb = torch.zeros(3, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 64, 16, dtype=torch.bfloat16, device="cuda")
    gemm, glu = lib.fp8_grouped_gemm_1x128_128x128, lib.fp8_grouped_swiglu_1x128
    cases = [
        (TypeError, lambda: lib.moe_route(z.double(), 2)), (ValueError, lambda: lib.moe_route(z, 9)), (ValueError, lambda: lib.moe_route(z, 0)),
        (ValueError, lambda: lib.moe_route(z.t(), 2)), (ValueError, lambda: lib.moe_route(z, 2, bias=z[0, :7])),
        (ValueError, lambda: lib.moe_route(z, 2, weights=z)), (TypeError, lambda: lib.moe_route(z, 2, experts=torch.zeros(6, 2, device="cuda"))),
        (TypeError, lambda: lib.group_rows(i.long(), 3)), (ValueError, lambda: lib.group_rows(i, 0)), (ValueError, lambda: lib.group_rows(i, 1025)),
        (ValueError, lambda: lib.group_rows(i.t(), 3)), (ValueError, lambda: lib.group_rows(i.view(3, 2, 2), 3)),
        (ValueError, lambda: lib.group_rows(i, 4, out=gr)),
        (ValueError, lambda: gemm(codes, words, w, ws, gr, gather=True)), (ValueError, lambda: gemm(codes[:6], words[:6], w, ws, gr)),
        (ValueError, lambda: gemm(codes, words, w[:2], ws, gr)), (ValueError, lambda: gemm(codes, words, w, ws[:, :1], gr)),
        (ValueError, lambda: gemm(codes, words[:, :0], w, ws, gr)), (TypeError, lambda: gemm(codes, words, w.int(), ws, gr)),
        (ValueError, lambda: gemm(codes, words, w, ws, lib.RowGroups(gr.offsets, gr.rows[:5], gr.slots))),
        (TypeError, lambda: gemm(codes, words, w, ws, lib.RowGroups(gr.offsets.long(), gr.rows, gr.slots))),
        (ValueError, lambda: gemm(codes, words, w, ws, gr, out=b)), (ValueError, lambda: gemm(codes, words, w.transpose(1, 2), ws, gr)),
        (ValueError, lambda: glu(codes, words, w, ws, gr, q=codes)), (lib.IqpError, lambda: glu(codes, words, w[:, :128], ws[:, :1], gr)),
        (ValueError, lambda: glu(codes, words, w[:, :255], ws, gr)),
        (ValueError, lambda: lib.moe_combine(b, gr, z)), (ValueError, lambda: lib.moe_combine(b[:5], gr, z[:, :2].contiguous())),
        (lib.IqpError, lambda: lib.moe_combine(b[:, :60].contiguous(), gr, z[:, :2].contiguous())),
        (ValueError, lambda: lib.moe_combine(b, gr, z[:, :2].contiguous(), shared=b)),
        (ValueError, lambda: lib.lora_add(b, b, la, lb, gr)), (ValueError, lambda: lib.lora_add(b, b, la[:2], lb, one)),
        (ValueError, lambda: lib.lora_add(b, b, la, lb[:, :60], one)), (TypeError, lambda: lib.lora_add(b.float(), b, la, lb, one)),
        (lib.IqpError, lambda: lib.lora_add(b.clone(), b, la[:, :12].contiguous(), lb[:, :, :12].contiguous(), one)),
        (lib.IqpError, lambda: lib.lora_add(b.clone(), b, la, lb, one, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: lib.lora_add(b.clone(), b, la, lb, one, scales=z[0])),
    ]
    for n, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
            print("no error from case", n)
    torch.cuda.synchronize()
    assert bool((b == 0).all())
