"""GPU: codes of silu(gate) * up next to the borders between two of them."""
import numpy as np
import pytest
import torch

import moe_ref as X

pytestmark = pytest.mark.gpu



def coded(h):
    """E4M3 magnitude and exponent of the largest value of a block, which the exponent
    puts into (224, 448], and how far from a border between two codes it lies."""
    h = np.abs(np.asarray(h, dtype=np.longdouble))
    e = np.ceil(np.log2(h / 448)).astype(int)
    v = h / np.exp2(e.astype(np.longdouble))
    step = np.where(v < 256, 16, 32)
    return (np.rint(v / step) * step).astype(np.float64), e, np.abs(v / step % 1 - 0.5) * step / v


def cases():
    """(n, s, u): a gate of -n 2^(s - 11), 32 to 84, and an up of u 2^-11, both of twelve
    bits, whose h lies 2^-21.5 to 2^-18.5 of itself from a border. Four roundings of
    float32 do not reach it (an exponential to 2^-23, a sum, a quotient and a product to
    2^-24 each: 2^-21.6); that of -gate log2(e) to float32 within an exponential, 2^-18.5
    of h at most, carries it across."""
    found = []
    u = np.arange(2048, 4096)
    for s in (5, 6):
        for n in range(2048, 4096):
            gate = -n * 2.0 ** (s - 11)
            if gate < -84:
                break
            x = np.longdouble(gate)
            h = np.longdouble(u) * (x / (1 + np.exp(-x))) / 2048
            rough = np.longdouble(u) * (x / (1 + np.exp2(np.longdouble(np.float32(-gate) * np.float32(1.4426950408889634))))) / 2048
            code, e, d = coded(h)
            hit = (d > 2.0 ** -21.5) & (d < 2.0 ** -18.5) & (coded(rough)[0] != code)
            found += [(n, s, int(u[i]), float(code[i]), int(e[i])) for i in np.nonzero(hit)[0]]
    return found


def codes_of(n):
    """n of twelve bits as three E4M3 values of four, each exact: n = 16 (a + b + c)."""
    parts = torch.tensor([n >> 8 << 4, (n >> 4) & 15, (n & 15) / 16], dtype=torch.float32)
    assert float(parts.sum()) * 16 == n
    return parts.to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("rows", [1, 40, 100, 170, 250])
def test_codes_next_to_a_border(gpu_lib, rows):
    """Blocks of one value each, whose code is the nearest."""
    found = cases()
    assert len(found) >= 16
    found = found[:64]
    print("borders", rows, len(found), flush=True)
    I, K = 128 * len(found), 128
    w = torch.zeros(1, 2 * I, K, dtype=torch.uint8)
    ws = torch.zeros(1, 2 * len(found), 1, dtype=torch.uint8)
    for i, (n, s, u, _, _) in enumerate(found):
        w[0, 128 * i + 5, :3] = codes_of(n) | 128
        w[0, I + 128 * i + 5, :3] = codes_of(u)
        ws[0, i, 0], ws[0, len(found) + i, 0] = 127 + s - 11 + 4, 127 - 11 + 4 + 110      # (the exponents' floor is 2^-22)
    a = torch.zeros(rows, K, dtype=torch.uint8)
    a[:, :3] = 0x38      # 1
    words = X.words_of(torch.full((rows, 1), 127, dtype=torch.uint8))
    plan = X.plan(torch.zeros(rows, dtype=torch.int32), 1)
    q, qs = gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), words.cuda(), w.cuda(), ws.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)))
    e = torch.stack([(qs.cpu().long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, : len(found)] - 127
    want_e = torch.tensor([f[4] + 110 for f in found])
    assert bool((e == want_e).all())
    got = q.cpu().view(torch.float8_e4m3fn).double().view(rows, len(found), 128)[:, :, 5]
    want = -torch.tensor([f[3] for f in found], dtype=torch.float64)
    assert bool((got == want).all()), (got != want).sum(1)


@pytest.mark.parametrize("rows", [2, 40])
def test_gates_of_all_sizes(gpu_lib, rows):
    """Gates of 1.5 2^e of either sign from nearly 0 to beyond the range of an
    exponential, one to a block, with ups that keep h in range where it is not 0."""
    gates = [(sign, e, 60 if sign < 0 and 3 <= e <= 5 else -e) for e in range(-119, 120) for sign in (1, -1)]
    n = len(gates)
    print("gates", rows, n, flush=True)
    I, K = 128 * n, 128
    w = torch.zeros(1, 2 * I, K, dtype=torch.uint8)
    ws = torch.zeros(1, 2 * n, 1, dtype=torch.uint8)
    h = np.zeros(n, dtype=np.longdouble)
    for i, (sign, e, u) in enumerate(gates):
        w[0, 128 * i + 77, 0] = 0x3C | (0 if sign > 0 else 128)     # +-1.5
        w[0, I + 128 * i + 77, 0] = 0x38
        ws[0, i, 0], ws[0, n + i, 0] = 127 + e, 127 + u
        x = np.longdouble(sign * 1.5 * 2.0 ** e)
        with np.errstate(over="ignore"):
            h[i] = x / (1 + np.exp(-x)) * np.longdouble(2.0) ** u
    a = torch.zeros(rows, K, dtype=torch.uint8)
    a[:, 0] = 0x38
    words = X.words_of(torch.full((rows, 1), 127, dtype=torch.uint8))
    plan = X.plan(torch.zeros(rows, dtype=torch.int32), 1)
    q, qs = gpu_lib.fp8_grouped_swiglu_1x128(a.cuda(), words.cuda(), w.cuda(), ws.cuda(), gpu_lib.RowGroups(*(t.cuda() for t in plan)))
    got_e = torch.stack([(qs.cpu().long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, :n] - 127
    got = q.cpu().view(torch.float8_e4m3fn).double().view(rows, n, 128)[:, :, 77]
    for i in range(n):
        if abs(h[i]) < 2.0 ** -33:                       # less than half of the least code at the least exponent
            assert bool((got_e[:, i] == -22).all()) and bool((got[:, i] == 0).all()), gates[i]
        else:
            code, e, away = coded(h[i:i + 1])
            assert away[0] > 2.0 ** -21
            assert bool((got_e[:, i] == int(e[0])).all()) and bool((got[:, i] == float(np.sign(h[i])) * code[0]).all()), gates[i]
