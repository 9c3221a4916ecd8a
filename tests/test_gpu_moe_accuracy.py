"""GPU: how far the products by expert are from exact sums: the matrix cores' own
error, how often a code or an exponent takes the other side of a border, and rows
behind 2^32 bytes of output against their float64 form."""
import numpy as np
import pytest
import torch

import layer_ref as R
import moe_ref as X

pytestmark = pytest.mark.gpu


def gen(*key):
    return np.random.default_rng([96, *key])


def quantised(lib, g, rows, K):
    """Rows as a layer has them: normal values, four channels that stand out."""
    x = X.bf16(g, rows, K)
    x[:, torch.from_numpy(g.integers(0, K, 4))] *= 30
    codes, words = lib.fp8_quant_1x128_ue8m0(x.cuda())
    b = torch.stack([(words.cpu().contiguous().long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, : K // 128]
    return codes, words, codes.cpu().view(torch.uint8), b


def weights(lib, g, groups, N, K):
    pairs = [lib.fp8_quant_weight_128x128_ue8m0(X.bf16(g, N, K, scale=0.02).cuda()) for _ in range(groups)]
    return torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])


@pytest.mark.parametrize("counts", [[16, 3], [60, 17], [128, 100], [190, 140], [256, 200]])
@pytest.mark.parametrize("K", [128, 2048])
def test_products_to_the_cores_precision(gpu_lib, counts, K):
    """Every 64 products are added at a fixed precision below the largest, which
    costs their sum up to 2^-11.3 of it (of one product); 2^-11 of the largest activation
    times the largest weight of the 64 is held to here, a quarter of what the other
    tests allow."""
    print("cores", counts, K, flush=True)
    g = gen(1, K, len(counts))
    index = X.index_of(counts, g)
    plan = X.plan(index, 2)
    a, words, ac, ab = quantised(gpu_lib, g, len(index), K)
    w, ws = weights(gpu_lib, g, 2, 256, K)
    out = gpu_lib.fp8_grouped_gemm_1x128_128x128(a, words, w, ws, gpu_lib.RowGroups(*(t.cuda() for t in plan)))
    y, bound = X.product(ac, ab, w.cpu().view(torch.uint8), ws.cpu(), plan[0], torch.arange(len(index)))
    X.check_product(out.cpu(), y, bound / 4)


@pytest.mark.parametrize("rows,K", [(12, 7168), (64, 512), (250, 2048)])
def test_how_often_codes_and_exponents_differ(gpu_lib, rows, K):
    """One code in 400 and one exponent in 15000 differ from those of exact sums;
    four times as many are too many (and one exponent, where four times as many are
    fewer than one)."""
    print("flips", rows, K, flush=True)
    g = gen(2, rows, K)
    I = 512
    plan = X.plan(torch.zeros(rows, dtype=torch.int32), 1)
    a, words, ac, ab = quantised(gpu_lib, g, rows, K)
    w, ws = weights(gpu_lib, g, 1, 2 * I, K)
    q, qs = gpu_lib.fp8_grouped_swiglu_1x128(a, words, w, ws, gpu_lib.RowGroups(*(t.cuda() for t in plan)))
    y, bound = X.product(ac, ab, w.cpu().view(torch.uint8), ws.cpu(), plan[0], torch.arange(rows))
    h = (y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]).view(rows, I // 128, 128)
    e = torch.ceil(torch.log2(h.abs().amax(2) / 448)).clamp_min(-22)
    v = h / 2.0 ** e[:, :, None]
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    nearest = torch.round(v / step) * step                                   # (ties to even, as the codes are)
    got_e = qs.cpu().contiguous().view(torch.uint8).view(rows, 4).double() - 127
    same = got_e == e
    assert int((~same).sum()) <= max(1, 4 * same.numel() // 15000)
    got = R.E4M3[q.cpu().long()].view_as(v)
    wrong = (got != nearest)[same]
    print("codes", int(wrong.sum()), "of", wrong.numel(), "exponents", int((~same).sum()), "of", same.numel(), flush=True)
    assert int(wrong.sum()) <= wrong.numel() / 100


def test_rows_past_32_bits(gpu_lib):
    """Rows on both sides of 2^31 and 2^32 bytes of output, and the last ones,
    against float64; their weighted sum and their adapters."""
    lib, g = gpu_lib, gen(3)
    n, N, K = 270000, 8200, 256
    index = torch.from_numpy((np.arange(n) >= 100).astype(np.int32) + (np.arange(n) >= n - 50)).cuda()
    gr = lib.group_rows(index, 3)
    a, words = torch.randint(0, 120, (n, K), dtype=torch.uint8, device="cuda"), torch.full((n, 1), 0x7F7F, dtype=torch.int32, device="cuda")
    w, ws = X.codes(g, 3, N, K), X.scale_bytes(g, 3, -(-N // 128), K // 128)
    out = lib.fp8_grouped_gemm_1x128_128x128(a, words, w.cuda(), ws.cuda(), gr)
    places = torch.cat([torch.arange(b - 3, b + 3) for b in ((1 << 31) // (2 * N), (1 << 32) // (2 * N), n - 50, n - 3)])
    offsets = torch.stack([(index.cpu()[places] < e).sum() for e in range(4)])
    y, bound = X.product(a.cpu()[places], torch.full((len(places), 2), 127), w, ws, offsets, torch.arange(len(places)))
    X.check_product(out[places.cuda()].cpu(), y, bound)
    slots = torch.stack([places, places.flip(0)], 1).to(torch.int32)
    weights_ = torch.from_numpy(g.random((len(places), 2)).astype(np.float32))
    pad = torch.full((n // 2 - len(places), 2), -1, dtype=torch.int32)
    pick = lib.RowGroups(gr.offsets, gr.rows, torch.cat([slots, pad]).cuda())
    got = lib.moe_combine(out, pick, torch.cat([weights_, torch.zeros(len(pad), 2)]).cuda())[: len(places)]
    near = out[places.cuda()].cpu()
    local = torch.stack([torch.arange(len(places)), torch.arange(len(places)).flip(0)], 1)
    want, tol = X.combine(near, local, weights_, None)
    assert bool(((got.cpu().double() - want).abs() <= tol).all())
    x = torch.randn(n, 64, device="cuda").to(torch.bfloat16)
    la, lb = X.bf16(g, 3, 8, 64, scale=0.125), X.bf16(g, 3, N, 8, scale=0.3)
    lib.lora_add(out, x, la.cuda(), lb.cuda(), gr)
    want, tol = X.lora(near, x[places.cuda()].cpu(), la, lb, offsets, torch.arange(len(places)), None)
    assert bool(((out[places.cuda()].cpu().double() - want).abs() <= tol).all())
