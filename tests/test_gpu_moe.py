"""GPU: routing, rows sorted by group, the products by group and the weighted sum
against their plain float64 forms (moe_ref), at the sizes and masks where they
can go wrong."""
import numpy as np
import pytest
import torch

import moe_ref as X

pytestmark = pytest.mark.gpu


def gen(*key):
    return np.random.default_rng([91, *key])


# ------------------------------------------------------------------ routing

ROUTE = [(1, 8, 1), (3, 8, 8), (5, 60, 6), (2, 64, 4), (7, 65, 8), (4, 160, 6), (9, 256, 8), (3, 257, 2), (2, 512, 10),
         (3, 1000, 64), (2, 1024, 33), (1, 1, 1)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("M,E,top", ROUTE)
@pytest.mark.parametrize("bias,half,renormalize", [(False, False, True), (True, False, True), (True, True, False), (False, True, False)])
def test_route(gpu_lib, M, E, top, scoring, bias, half, renormalize):
    print("route", M, E, top, scoring, bias, half, renormalize, flush=True)
    g = gen(1, M, E, top, bias)
    z = torch.from_numpy(g.standard_normal((M, E)).astype(np.float32) * 3)
    z = z.to(torch.bfloat16) if half else z
    b = torch.from_numpy(g.standard_normal(E).astype(np.float32)) if bias else None
    w, e = gpu_lib.moe_route(z.cuda(), top, bias=None if b is None else b.cuda(), scoring=scoring, renormalize=renormalize, scale=2.5)
    want, ids = X.route(z, top, b, scoring, renormalize, 2.5)
    assert torch.equal(e.cpu(), ids)
    # one rounding of float64 arithmetic
    assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want.abs() + 2.0 ** -149).all())


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_ties_and_masks(gpu_lib, bias, scoring, renormalize):
    """Equal logits in one lane's values and across lanes, zeros of both signs,
    masked experts (some, all but two, all), the type's lowest value."""
    E, top = 200, 6
    inf = float("inf")
    z = torch.zeros(7, E)
    z[0, 1::2] = -0.0
    z[1] = torch.arange(E) % 3
    z[2] = -inf
    z[3] = -inf
    z[3, [7, 150]] = torch.tensor([1.0, 2.0])
    z[4, ::2] = -inf
    z[5] = torch.finfo(torch.float32).min
    z[5, 199] = 0.0
    z[6, 64:] = -inf
    b = torch.zeros(E) if bias else None
    w, e = gpu_lib.moe_route(z.cuda(), top, bias=b if b is None else b.cuda(), scoring=scoring, renormalize=renormalize)
    want, ids = X.route(z, top, b, scoring, renormalize, 1.0)
    assert torch.equal(e.cpu(), ids), (e, ids)
    assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want.abs() + 2.0 ** -149).all())


def test_route_bad_logits(gpu_lib):
    """NaN and +inf: the token's weights are NaN, its experts distinct and in
    range, the other tokens' as ever."""
    g = gen(2)
    z = torch.from_numpy(g.standard_normal((6, 96)).astype(np.float32))
    good = gpu_lib.moe_route(z.cuda(), 8)
    bad = z.clone()
    bad[1, 5] = float("nan")
    bad[3] = float("nan")
    bad[4, 9] = float("inf")
    for bias in (None, torch.zeros(96, device="cuda")):
        w, e = gpu_lib.moe_route(bad.cuda(), 8, bias=bias)
        for m in range(6):
            ids = e[m].tolist()
            assert len(set(ids)) == 8 and min(ids) >= 0 and max(ids) < 96
            if m in (1, 3, 4):
                assert bool(torch.isnan(w[m]).all()) or m == 4 and bool(torch.isnan(w[m]).any())
            elif bias is None:
                assert torch.equal(w[m], good[0][m]) and torch.equal(e[m], good[1][m])


def test_route_strides_and_out(gpu_lib):
    g = gen(3)
    wide = torch.from_numpy(g.standard_normal((5, 100)).astype(np.float32)).cuda()
    z = wide[:, 3:67]
    w, e = torch.empty(5, 4, device="cuda"), torch.empty(5, 4, dtype=torch.int32, device="cuda")
    r = gpu_lib.moe_route(z, 4, weights=w, experts=e)
    assert r[0] is not None and r[0].data_ptr() == w.data_ptr() and r[1].data_ptr() == e.data_ptr()
    x = gpu_lib.moe_route(z.contiguous(), 4)
    assert torch.equal(w, x[0]) and torch.equal(e, x[1])
    assert gpu_lib.moe_route(z[:0], 4)[0].shape == (0, 4)


# -------------------------------------------------------------------- sorting

@pytest.mark.parametrize("R,G", [(0, 1), (0, 1024), (1, 1), (8, 256), (63, 3), (64, 64), (65, 1), (1000, 7), (2048, 1024), (2049, 9),
                                 (4096, 2), (37056, 256), (50001, 1023)])
@pytest.mark.parametrize("kind", ["even", "skewed", "outside"])
def test_group_rows(gpu_lib, R, G, kind):
    print("group_rows", R, G, kind, flush=True)
    g = gen(4, R, G)
    i = g.integers(0, G, R)
    if kind == "skewed":
        i = np.minimum(i, g.integers(0, G, R) // 4)
    if kind == "outside":
        i = np.where(g.random(R) < 0.3, g.choice([-1, G, -(1 << 31), (1 << 31) - 1], R), i)
    index = torch.from_numpy(i.astype(np.int32))
    got = gpu_lib.group_rows(index.cuda(), G)
    key = torch.where((index >= 0) & (index < G), index, G)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key.sort().values, torch.arange(G + 1, dtype=torch.int32))
    held = int(offsets[G])
    rows = torch.where(torch.arange(R) < held, order, -1)
    slots = torch.full((R,), -1)
    slots[order[:held]] = torch.arange(held)
    for a, b in zip(got, (offsets, rows, slots)):
        assert torch.equal(a.cpu().long(), b.long())


def test_group_rows_shapes_and_workspace(gpu_lib):
    g = gen(5)
    index = torch.from_numpy(g.integers(-1, 40, (3001, 4)).astype(np.int32))
    need = gpu_lib.group_rows_workspace_bytes(index.numel(), 40)
    assert need > 0 and gpu_lib.group_rows_workspace_bytes(100, 40) == 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    out = gpu_lib.RowGroups(*(torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((41,), (12004,), (3001, 4))))
    got = gpu_lib.group_rows(index.cuda(), 40, out=out, workspace=ws[:need])
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out)) and got.slots.shape == (3001, 4)
    assert bool((ws[need:] == 255).all())
    plain = gpu_lib.group_rows(index.cuda(), 40)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    want = X.plan(index, 40)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


# ------------------------------------------------------------------- products

# rows of every group, entries of none
COUNTS = {
    "token": ([0, 1, 0, 1], 0),
    "few": ([1, 0, 2, 15, 16, 3], 5),
    "edges": ([17, 31, 32, 33, 0, 63], 2),
    "middle": ([64, 65, 1, 127, 128], 0),
    "large": ([129, 192, 193, 0, 255], 31),
    "whole": ([256, 257, 300], 0),
    "one": ([700], 3),
    "none": ([0, 0, 0], 9),
    "many": ([int(c) for c in gen(6).integers(0, 4, 300)], 4),
}


def operands(g, counts, none, N, K, top=1, gather=False):
    index = X.index_of(counts, g, none)
    if gather:
        index = index[: len(index) // top * top].view(-1, top)
    offsets, rows, slots = X.plan(index, len(counts))
    M = index.shape[0] if gather else index.numel()
    a, ab = X.codes(g, M, K), X.scale_bytes(g, M, K // 128)
    w, ws = X.codes(g, len(counts), N, K), X.scale_bytes(g, len(counts), -(-N // 128), K // 128)
    src = rows.long().clamp_min(0) // top if gather else torch.arange(index.numel())
    return (offsets, rows, slots), a, ab, w, ws, src


def groups_on_gpu(lib, plan):
    return lib.RowGroups(*(t.cuda() for t in plan))


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K,top,gather", [(256, 256, 1, False), (300, 128, 2, True), (129, 640, 3, True), (1, 384, 1, False), (520, 1024, 1, True)])
def test_grouped_gemm(gpu_lib, name, N, K, top, gather):
    print("grouped_gemm", name, N, K, top, gather, flush=True)
    counts, none = COUNTS[name]
    plan, a, ab, w, ws, src = operands(gen(7, len(name), N, K), counts, none, N, K, top, gather)
    R = len(src)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    got = gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan),
                                                 gather=gather, out=out)
    assert got.data_ptr() == out.data_ptr()
    y, bound = X.product(a, ab, w, ws, plan[0], src)
    X.check_product(out.cpu(), y, bound)
    assert bool((out.cpu()[int(plan[0][-1]):] == 7.0).all())      # places of no group


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("I,K,top,gather", [(128, 256, 1, False), (256, 128, 2, True), (640, 640, 1, False), (512, 384, 4, True)])
def test_grouped_swiglu(gpu_lib, name, I, K, top, gather):
    print("grouped_swiglu", name, I, K, top, gather, flush=True)
    counts, none = COUNTS[name]
    plan, a, ab, w, ws, src = operands(gen(8, len(name), I, K), counts, none, 2 * I, K, top, gather)
    R, nw = len(src), -(-I // 512)
    q = torch.full((R, I), 9, dtype=torch.uint8, device="cuda")
    words = torch.full((R, nw), 0x01010101, dtype=torch.int32, device="cuda")
    gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan), gather=gather,
                                     q=q, q_scales=words)
    y, bound = X.product(a, ab, w, ws, plan[0], src)
    X.check_swiglu(q.cpu(), words.cpu(), y, bound)
    held = int(plan[0][-1])
    assert bool((q.cpu()[held:] == 9).all()) and bool((words.cpu()[held:] == 0x01010101).all())


def test_swiglu_extremes(gpu_lib):
    """Gates far below and above zero, blocks that are all zero: no NaN, the
    exponents' floor, padding bytes of a word."""
    counts, I, K = [3, 70], 256, 128
    plan, a, ab, w, ws, src = operands(gen(9), counts, 0, 2 * I, K)
    a[0] = 0                                         # a row of zeros
    ab[:] = 127
    ws[:] = 127
    w[:, :I] = 0
    w[0, :, 0] = torch.where(torch.arange(2 * I) % 2 == 0, 0x7E, 0xFE).to(torch.uint8)     # +-448 in the first column
    a[:3, 0] = torch.tensor([0, 0x7E, 0xFE], dtype=torch.uint8)
    got = gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan))
    assert not bool(torch.isnan(got[0].view(torch.float8_e4m3fn).float()).any())
    b = got[1].cpu().view(torch.uint8)
    assert bool((b[0, :2] == 127 - 22).all()) and bool((got[0][0] & 127 == 0).all()) and bool((b[:, 2:] == 0).all())
    y, bound = X.product(a, ab, w, ws, plan[0], src)
    X.check_swiglu(got[0].cpu(), got[1].cpu(), y, bound)


def test_products_strides(gpu_lib):
    """Weights that are part of a larger tensor or shared by all groups, scale words
    in columns, rows of a wider a and out, both outputs of odd widths."""
    g = gen(10)
    counts, N, K = [20, 3, 140], 270, 384
    plan, a, ab, w, ws, src = operands(g, counts, 0, N, K)
    gr = groups_on_gpu(gpu_lib, plan)
    R = len(src)
    big_w = torch.zeros(3, N + 50, K + 128, dtype=torch.uint8, device="cuda")
    big_w[:, :N, :K] = w.cuda()
    big_a = torch.zeros(R, K + 64, dtype=torch.uint8, device="cuda")
    big_a[:, :K] = a.cuda()
    words = X.words_of(ab).cuda().t().contiguous().t()
    out = torch.full((R, N + 26), 3.0, dtype=torch.bfloat16, device="cuda")
    call = gpu_lib.fp8_grouped_gemm_1x128_128x128
    plain = call(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), gr)
    call(big_a[:, :K], words, big_w[:, :N, :K], ws.cuda(), gr, out=out[:, :N])
    assert torch.equal(out[:, :N], plain) and bool((out[:, N:] == 3.0).all())
    odd = torch.full((R, N + 3), 3.0, dtype=torch.bfloat16, device="cuda")
    call(big_a[:, :K], words, big_w[:, :N, :K], ws.cuda(), gr, out=odd[:, 1:N + 1])
    assert torch.equal(odd[:, 1:N + 1], plain) and bool((odd[:, N + 1:] == 3.0).all()) and bool((odd[:, 0] == 3.0).all())
    shared = call(a.cuda(), X.words_of(ab).cuda(), w[:1].cuda().expand(3, N, K), ws[:1].cuda().expand(3, -1, -1), gr)
    same = call(a.cuda(), X.words_of(ab).cuda(), w[:1].repeat(3, 1, 1).cuda(), ws[:1].repeat(3, 1, 1).cuda(), gr)
    assert torch.equal(shared, same)
    # the other entry point: words of its output in columns, codes in a wider row
    I = 256
    plan, a, ab, w, ws, src = operands(g, counts, 0, 2 * I, K)
    gr = groups_on_gpu(gpu_lib, plan)
    q = torch.zeros(R, I + 16, dtype=torch.uint8, device="cuda")
    cols = torch.zeros(1, R, dtype=torch.int32, device="cuda").t()
    x = gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), gr)
    gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), gr, q=q[:, :I], q_scales=cols)
    assert torch.equal(q[:, :I], x[0]) and torch.equal(cols, x[1]) and bool((q[:, I:] == 0).all())


def test_products_bad_plan(gpu_lib):
    """Offsets out of range or falling and rows that name no token: nothing is
    written outside the output, rows of the good groups are right."""
    g = gen(11)
    N, K, G = 256, 256, 5
    plan, a, ab, w, ws, src = operands(g, [4, 30, 5, 0, 8], 0, N, K)
    R = len(src)
    offsets = torch.tensor([-5, 4, 2, 34, 1 << 30, -(1 << 31)], dtype=torch.int32)
    rows = plan[1].clone()
    rows[2], rows[3] = -9, 1 << 30
    buf = torch.full((R + 20, N), 5.0, dtype=torch.bfloat16, device="cuda")
    gr = gpu_lib.RowGroups(offsets.cuda(), rows.cuda(), plan[2].view(-1, 1).cuda())
    gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), gr, gather=True, out=buf[10:10 + R])
    assert bool((buf[:10] == 5.0).all()) and bool((buf[10 + R:] == 5.0).all())
    src = rows.long().clamp(0, R - 1)
    y, bound = X.product(a, ab, w, ws, torch.tensor([0, 4, 4, 4, 4, 4]), src)
    X.check_product(buf[10:12].cpu(), y[:2], bound[:2])
    assert bool((buf[12:14] == 0).all())          # rows of no token read zeros


# ---------------------------------------------------------------------- combine

@pytest.mark.parametrize("M,top,d", [(1, 1, 8), (1, 8, 7168), (16, 8, 2048), (7, 3, 2056), (33, 9, 136), (5, 20, 4104)])
@pytest.mark.parametrize("shared", [False, True])
def test_combine(gpu_lib, M, top, d, shared):
    print("combine", M, top, d, shared, flush=True)
    g = gen(12, M, top, d)
    index = torch.from_numpy(g.integers(-1, 9, (M, top)).astype(np.int32))      # some in no group
    plan = X.plan(index, 9)
    y = X.bf16(g, M * top, d)
    y[int(plan[0][-1]):] = float("nan")            # rows of no group are not read
    w = torch.from_numpy(g.random((M, top)).astype(np.float32))
    s = X.bf16(g, M, d) if shared else None
    out = gpu_lib.moe_combine(y.cuda(), groups_on_gpu(gpu_lib, plan), w.cuda(), shared=None if s is None else s.cuda())
    want, tol = X.combine(y, plan[2], w, s)
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    if shared:                                     # in place, and between other columns
        buf = torch.full((M, d + 16), 4.0, dtype=torch.bfloat16, device="cuda")
        buf[:, 8:8 + d] = s.cuda()
        part = buf[:, 8:8 + d]
        gpu_lib.moe_combine(y.cuda(), groups_on_gpu(gpu_lib, plan), w.cuda(), shared=part, out=part)
        assert torch.equal(part, out) and bool((buf[:, :8] == 4.0).all()) and bool((buf[:, 8 + d:] == 4.0).all())


def test_combine_one_dim(gpu_lib):
    g = gen(13)
    index = torch.from_numpy(g.integers(0, 3, 6).astype(np.int32))
    plan = X.plan(index, 3)
    y, w = X.bf16(g, 6, 64), torch.ones(6)
    out = gpu_lib.moe_combine(y.cuda(), groups_on_gpu(gpu_lib, plan), w.cuda())
    assert torch.equal(out.cpu(), y[plan[2].long()])


# ------------------------------------------------- the kernels' other variants

@pytest.mark.parametrize("E,top", [(1, 1), (8, 8), (16, 3), (17, 16), (32, 4), (60, 6), (64, 8), (100, 16), (128, 4), (200, 5), (256, 8)])
@pytest.mark.parametrize("scoring,bias,half", [("softmax", False, False), ("sigmoid", True, False), ("sqrt_softplus", True, True), ("softmax", True, False)])
def test_route_many_tokens(gpu_lib, E, top, scoring, bias, half):
    """Batches that go to the kernel of 16 lanes a token (and a token more than a
    workgroup has), with masked experts, against the plain form on some rows and
    the few tokens' kernel on all."""
    print("route many", E, top, scoring, bias, half, flush=True)
    g = gen(14, E, top)
    M = 40 * E + 5
    z = torch.from_numpy(g.standard_normal((M, E)).astype(np.float32) * 3)
    z[::7, ::3] = -float("inf")
    z[5] = -float("inf")
    z = z.to(torch.bfloat16) if half else z
    b = torch.from_numpy(g.standard_normal(E).astype(np.float32)) if bias else None
    dev = dict(bias=None if b is None else b.cuda(), scoring=scoring, scale=0.75)
    w, e = gpu_lib.moe_route(z.cuda(), top, **dev)
    some = torch.cat((torch.arange(min(M, 64)), torch.arange(M - 20, M))).unique()
    want, ids = X.route(z[some], top, b, scoring, True, 0.75)
    assert torch.equal(e.cpu()[some], ids)
    assert bool(((w.cpu()[some].double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want.abs() + 2.0 ** -149).all())
    step = max(1, 40 * E - 1)
    for lo in range(0, M, step):
        few = gpu_lib.moe_route(z[lo:lo + step].cuda(), top, **dev)
        assert torch.equal(few[1], e[lo:lo + step])
        # (sums of the chosen scores are added up in another order)
        assert bool(((few[0] - w[lo:lo + step]).abs() <= 2.0 ** -23 * w[lo:lo + step]).all())


def test_grouped_many_tiles(gpu_lib):
    """More groups than a round of the search for a tile looks at, and items enough
    for the order by eight chunks."""
    g = gen(15)
    for G, N in ((1000, 300), (300, 4000)):
        print("many tiles", G, N, flush=True)
        counts = [int(c) for c in g.integers(0, 4, G)]
        counts[G - 2] = 270
        plan, a, ab, w, ws, src = operands(g, counts, 3, N, 128)
        out = gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan))
        y, bound = X.product(a, ab, w, ws, plan[0], src)
        X.check_product(out.cpu(), y, bound)


def test_grouped_long_k(gpu_lib):
    """The longest K that is taken, with few rows and with a whole tile of them."""
    g = gen(16)
    for counts in ([3, 0, 1], [20, 260]):
        print("long k", counts, flush=True)
        plan, a, ab, w, ws, src = operands(g, counts, 0, 256, 32768)
        out = gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan))
        y, bound = X.product(a, ab, w, ws, plan[0], src)
        X.check_product(out.cpu(), y, bound)


def test_grouped_offset_start(gpu_lib):
    """Places before the first group and between none: left as they were."""
    g = gen(17)
    plan, a, ab, w, ws, src = operands(g, [9, 20, 4], 0, 256, 256)
    offsets = torch.tensor([5, 9, 29, 31], dtype=torch.int32)
    out = torch.full((33, 256), 6.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(),
                                           gpu_lib.RowGroups(offsets.cuda(), plan[1].cuda(), plan[2].cuda()), out=out)
    y, bound = X.product(a, ab, w, ws, offsets, src)
    X.check_product(out.cpu(), y, bound)
    assert bool((out[:5] == 6.0).all()) and bool((out[31:] == 6.0).all())


@pytest.mark.parametrize("M,E,top", [(9, 64, 8), (5, 128, 5), (7, 200, 8), (9, 256, 8), (3, 500, 40), (4, 1000, 64), (2600, 64, 8)])
@pytest.mark.parametrize("scoring,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True), ("sqrt_softplus", True)])
def test_route_close_logits(gpu_lib, M, E, top, scoring, bias):
    """Logits that differ in their last six bits alone, many of them equal: the
    order hangs on the last bits of the choices, and on the index."""
    print("close logits", M, E, top, scoring, bias, flush=True)
    g = gen(23, M, E, top)
    z = torch.from_numpy((1 + g.integers(0, 64, (M, E)) * 2.0 ** -23).astype(np.float32))
    b = torch.full((E,), 0.5) if bias else None
    w, e = gpu_lib.moe_route(z.cuda(), top, bias=None if b is None else b.cuda(), scoring=scoring)
    want, ids = X.route(z, top, b, scoring, True, 1.0)
    assert torch.equal(e.cpu(), ids)
    assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want.abs()).all())


@pytest.mark.parametrize("N,K,top,gather", [(9 * 256 + 40, 256, 1, False), (5 * 256, 384, 2, True)])
def test_grouped_remainders(gpu_lib, N, K, top, gather):
    """Groups of one, two and three tiles whose last ones are of every body's size,
    and more parts of a tile than come in a row."""
    print("remainders", N, K, top, gather, flush=True)
    g = gen(24, N, K)
    counts = [264, 256, 300, 0, 520, 2, 384, 700, 257, 449]
    plan, a, ab, w, ws, src = operands(g, counts, 4, N, K, top, gather)
    out = gpu_lib.fp8_grouped_gemm_1x128_128x128(a.cuda(), X.words_of(ab).cuda(), w.cuda(), ws.cuda(), groups_on_gpu(gpu_lib, plan), gather=gather)
    y, bound = X.product(a, ab, w, ws, plan[0], src)
    X.check_product(out.cpu(), y, bound)


@pytest.mark.parametrize("E", [8, 64, 256, 300])
@pytest.mark.parametrize("far", [False, True])
def test_route_sigmoids_of_all_sizes(gpu_lib, E, far):
    """Sigmoid scores with a bias for logits from nearly 0 to beyond the range of
    exp, one such logit in a token or none: weights to one rounding, experts as the
    scores in 64 bits order them."""
    print("sigmoids", E, far, flush=True)
    g = gen(25, E, far)
    z = g.standard_normal((40, E)) * 10.0 ** g.uniform(-6, 2, (40, E))
    if far:
        z[::2, 1] = -1e4
        z[1::4, 2] = 3e38
        z[3::4, 3] = -700
    z = torch.from_numpy(z.astype(np.float32))
    b = torch.from_numpy(g.standard_normal(E).astype(np.float32))
    for renormalize in (False, True):
        w, e = gpu_lib.moe_route(z.cuda(), 4, bias=b.cuda(), scoring="sigmoid", renormalize=renormalize)
        want, ids = X.route(z, 4, b, "sigmoid", renormalize, 1.0)
        assert torch.equal(e.cpu(), ids)
        assert bool(((w.cpu().double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want.abs() + 2.0 ** -149).all())
