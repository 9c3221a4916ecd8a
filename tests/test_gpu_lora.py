"""GPU: low-rank adapters added to a projection's output, against the plain
float64 form (moe_ref)."""
import numpy as np
import pytest
import torch

import moe_ref as X

pytestmark = pytest.mark.gpu


def gen(*key):
    return np.random.default_rng([92, *key])


def case(g, counts, none, N, K, rank):
    index = X.index_of(counts, g, none)
    plan = X.plan(index, len(counts))
    M, G = len(index), len(counts)
    return plan, X.bf16(g, M, N), X.bf16(g, M, K), X.bf16(g, G, rank, K, scale=K ** -0.5), X.bf16(g, G, N, rank, scale=0.3), \
        torch.from_numpy(g.random(G).astype(np.float32) * 2 + 0.25)


COUNTS = [([1], 0), ([0, 1, 0, 2], 3), ([15, 16, 17, 0, 33], 4), ([64, 65, 1], 0), ([130, 3], 9), ([1] * 70, 1), ([0, 0], 5)]


@pytest.mark.parametrize("counts,none", COUNTS)
@pytest.mark.parametrize("N,K,rank", [(256, 128, 16), (64, 8, 8), (300, 520, 24), (1, 64, 32), (513, 192, 40), (264, 1032, 64),
                                      (272, 256, 72), (96, 136, 128)])
@pytest.mark.parametrize("scaled", [True, False])
def test_lora(gpu_lib, counts, none, N, K, rank, scaled):
    print("lora", counts[:6], none, N, K, rank, scaled, flush=True)
    plan, out, x, a, b, s = case(gen(1, len(counts), N, K, rank), counts, none, N, K, rank)
    s = s if scaled else None
    want, tol = X.lora(out, x, a, b, plan[0], plan[1], s)
    got = out.cuda()
    r = gpu_lib.lora_add(got, x.cuda(), a.cuda(), b.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)), scales=None if s is None else s.cuda())
    assert r.data_ptr() == got.data_ptr()
    assert bool(((got.cpu().double() - want).abs() <= tol).all())
    none_rows = (plan[2] < 0).nonzero().flatten()
    assert torch.equal(got.cpu()[none_rows], out[none_rows])


def test_lora_long_k(gpu_lib):
    """Sums cut along K (few rows) and not (many)."""
    for counts in ([2, 0, 1], [200, 77]):
        print("lora long", counts, flush=True)
        plan, out, x, a, b, s = case(gen(2, len(counts)), counts, 1, 256, 7168, 16)
        want, tol = X.lora(out, x, a, b, plan[0], plan[1], s)
        got = out.cuda()
        gpu_lib.lora_add(got, x.cuda(), a.cuda(), b.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)), scales=s.cuda())
        assert bool(((got.cpu().double() - want).abs() <= tol).all())


def test_lora_strides(gpu_lib):
    """Column ranges of a wider x and out, an out of odd stride and alignment, rows
    of no group and columns beside the range left as they were, NaN in rows of x
    that have no adapter."""
    plan, out, x, a, b, s = case(gen(3), [20, 3, 70], 6, 200, 256, 16)
    gr = gpu_lib.RowGroups(*(t.cuda() for t in plan))
    M = out.shape[0]
    none = (plan[2] < 0).nonzero().flatten()
    x[none] = float("nan")
    want, tol = X.lora(out, x, a, b, plan[0], plan[1], s)
    bx = torch.full((M, 272), float("inf"), dtype=torch.bfloat16, device="cuda")
    bx[:, 8:264] = x.cuda()
    for pad, at in ((24, 16), (3, 1)):
        bo = torch.full((M, 200 + pad), 2.0, dtype=torch.bfloat16, device="cuda")
        bo[:, at:at + 200] = out.cuda()
        gpu_lib.lora_add(bo[:, at:at + 200], bx[:, 8:264], a.cuda(), b.cuda(), gr, scales=s.cuda())
        assert bool(((bo[:, at:at + 200].cpu().double() - want).abs() <= tol).all())
        assert bool((bo[:, :at] == 2.0).all()) and bool((bo[:, at + 200:] == 2.0).all())


def test_lora_workspace(gpu_lib):
    plan, out, x, a, b, s = case(gen(4), [5, 40], 2, 128, 256, 24)
    gr = gpu_lib.RowGroups(*(t.cuda() for t in plan))
    need = gpu_lib.lora_add_workspace_bytes(47, 2, 24, 256)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")      # NaN everywhere
    one, two = out.cuda(), out.cuda()
    gpu_lib.lora_add(one, x.cuda(), a.cuda(), b.cuda(), gr, workspace=ws[:need])
    gpu_lib.lora_add(two, x.cuda(), a.cuda(), b.cuda(), gr)
    assert torch.equal(one, two) and bool((ws[need:] == 255).all())


def test_lora_many_adapters(gpu_lib):
    """More adapters than a round of the search for a tile looks at."""
    g = gen(5)
    counts = [int(c) for c in g.integers(0, 3, 600)]
    counts[598] = 90
    plan, out, x, a, b, s = case(g, counts, 7, 72, 136, 8)
    want, tol = X.lora(out, x, a, b, plan[0], plan[1], s)
    got = out.cuda()
    gpu_lib.lora_add(got, x.cuda(), a.cuda(), b.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)), scales=s.cuda())
    assert bool(((got.cpu().double() - want).abs() <= tol).all())


def test_lora_bad_plan(gpu_lib):
    """Offsets out of range or falling and rows that name no token: nothing else is
    written, the good groups' rows are right."""
    g = gen(6)
    plan, out, x, a, b, s = case(g, [4, 30, 5, 0, 8], 0, 100, 64, 16)
    M = out.shape[0]
    rows = plan[1].clone()
    rows[2], rows[3] = -9, 1 << 30
    offsets = torch.tensor([-5, 4, 2, 2, 1 << 30, -(1 << 31)], dtype=torch.int32)
    buf = torch.full((M + 20, 100), 5.0, dtype=torch.bfloat16, device="cuda")
    buf[10:10 + M] = out.cuda()
    gpu_lib.lora_add(buf[10:10 + M], x.cuda(), a.cuda(), b.cuda(), gpu_lib.RowGroups(offsets.cuda(), rows.cuda(), plan[2].cuda()), scales=s.cuda())
    want, tol = X.lora(out, x, a, b, torch.tensor([0, 4, 4, 4, 4, 4]), rows, s)
    keep = torch.ones(M, dtype=torch.bool)
    keep[rows[4:].long()] = False                  # (places of the group that begins past the last one)
    assert bool(((buf[10:10 + M].cpu().double() - want).abs() <= tol)[keep].all())
    assert bool((buf[:10] == 5.0).all()) and bool((buf[10 + M:] == 5.0).all())


def test_lora_many_rows_large_rank(gpu_lib):
    """Batches whose first launch has 32 rows a workgroup, on both sides of its border."""
    for counts, rank in (([1100, 37, 0, 900], 64), ([1900, 17], 40), ([2048], 128), ([2080, 1], 72)):
        print("lora large", counts, rank, flush=True)
        plan, out, x, a, b, s = case(gen(7, rank), counts, 5, 40, 200, rank)
        want, tol = X.lora(out, x, a, b, plan[0], plan[1], s)
        got = out.cuda()
        gpu_lib.lora_add(got, x.cuda(), a.cuda(), b.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)), scales=s.cuda())
        assert bool(((got.cpu().double() - want).abs() <= tol).all())
