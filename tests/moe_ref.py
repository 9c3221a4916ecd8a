"""Plain float64 implementations of the operators whose weights depend on the
token, and the bounds their kernels are held to (test infrastructure only;
shares no code with the kernels). Tensors are on the CPU."""
import numpy as np
import torch

import layer_ref as R


def bf16(g, *shape, scale=1.0):
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def codes(g, *shape):
    """E4M3 codes of normal values (no NaN)."""
    x = torch.from_numpy(g.standard_normal(shape).astype(np.float32) * 8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def scale_bytes(g, *shape, lo=118, hi=130):
    return torch.from_numpy(g.integers(lo, hi, shape).astype(np.uint8))


def words_of(bytes_):
    """Packed words [M, ceil(kb/4)] of scale bytes [M, kb]."""
    M, kb = bytes_.shape
    full = torch.zeros(M, -(-kb // 4) * 4, dtype=torch.uint8)
    full[:, :kb] = bytes_
    return full.view(torch.int32)


def index_of(counts, g, none=0):
    """A shuffled index with counts[e] entries of group e and `none` of none."""
    flat = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [g.choice([-1, len(counts), -7], none)])
    return torch.from_numpy(g.permutation(flat).astype(np.int32))


def plan(index, groups):
    """(offsets, rows, slots) of group_rows, one entry at a time."""
    flat = index.reshape(-1).tolist()
    held = [[i for i, e in enumerate(flat) if e == g] for g in range(groups)]
    offsets, rows, slots = [0], [], [-1] * len(flat)
    for h in held:
        for i in h:
            slots[i] = len(rows)
            rows.append(i)
        offsets.append(len(rows))
    rows += [-1] * (len(flat) - len(rows))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(rows), i32(slots).view(index.shape)


def route(logits, top_k, bias, scoring, renormalize, scale):
    """float64 weights and the experts, by a sort on (choice, index)."""
    z = logits.double().numpy()
    M, E = z.shape
    weights, experts = np.zeros((M, top_k)), np.zeros((M, top_k), dtype=np.int32)
    for m in range(M):
        with np.errstate(all="ignore"):
            if scoring == "softmax":
                top = z[m].max()
                p = np.exp(z[m] - top) if np.isfinite(top) else np.zeros(E)
                p = p / p.sum() if p.sum() else p
            elif scoring == "sigmoid":
                p = 1 / (1 + np.exp(-z[m]))
            else:
                p = np.sqrt(np.logaddexp(z[m], 0))
        c = z[m] if bias is None else np.where(np.isneginf(z[m]), -np.inf, p + bias.double().numpy())
        e = sorted(range(E), key=lambda i: (-c[i], i))[:top_k]
        w = np.where(np.isneginf(z[m][e]), 0.0, p[e])
        if renormalize:
            w = w / w.sum() if w.sum() else np.zeros(top_k)
        weights[m], experts[m] = scale * w, e
    return torch.from_numpy(weights), torch.from_numpy(experts)


def product(a, a_bytes, w, w_scales, offsets, src):
    """float64 (y, bound) [R, N] of the grouped product of E4M3 codes; bound: what
    the matrix cores may be off by, 2^-9 of the largest product of every 64 columns
    (they add products at a fixed precision below the largest). Places of no group
    are NaN."""
    places, N, K = len(src), w.shape[1], w.shape[2]
    y = torch.full((places, N), float("nan"), dtype=torch.float64)
    bound = torch.zeros(places, N, dtype=torch.float64)
    A = R.E4M3[a.long()] * (2.0 ** (a_bytes.double() - 127)).repeat_interleave(128, 1)
    for g in range(w.shape[0]):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        if hi <= lo:
            continue
        x, W = A[src[lo:hi]], R.dequant_tiles(w[g], w_scales[g])
        y[lo:hi] = x @ W.T
        bound[lo:hi] = 2.0 ** -9 * (x.abs().view(-1, K // 64, 64).amax(2) @ W.abs().view(-1, K // 64, 64).amax(2).T)
    return y, bound


def check_product(out, y, bound):
    """bf16 rows against (y, bound): the bound and the rounding."""
    held = ~torch.isnan(y[:, 0])
    d = (out.double() - y)[held].abs()
    assert bool((d <= (bound + 2.0 ** -8 * (y.abs() + bound))[held]).all())


def check_swiglu(q, words, y, bound):
    """Codes and words against silu(gate) up of (y, bound) [R, 2 I].

    |silu'| <= 1.1, so h is off by at most dh = 1.1 bg |u| + |silu(g)| bu + 1.1 bg bu,
    and 2^-19 of itself for float32 (an exponential of |g| < 2^7, a quotient and
    two products). The exponent fits the largest h of the block give or take dh; a
    code is off by half a step of E4M3, 2^-4 of the value, or 2^-10 of the scale."""
    held = ~torch.isnan(y[:, 0])
    y, bound, q, words = y[held], bound[held], q[held], words[held]
    I = y.shape[1] // 2
    gate, up, bg, bu = y[:, :I], y[:, I:], bound[:, :I], bound[:, I:]
    silu = gate * torch.sigmoid(gate)
    h = silu * up
    dh = 1.1 * bg * up.abs() + silu.abs() * bu + 1.1 * bg * bu + 2.0 ** -19 * h.abs()
    b = torch.stack([(words.long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)
    assert bool((b[:, I // 128:] == 0).all())
    e = b[:, : I // 128].double() - 127
    amax, slack = h.abs().view(-1, I // 128, 128).amax(2), dh.view(-1, I // 128, 128).amax(2)
    assert bool((448 * 2.0 ** e >= amax - slack).all()) and bool((e >= -22).all())
    assert bool(((e == -22) | (448 * 2.0 ** (e - 1) < amax + slack)).all())
    step = 2.0 ** e.repeat_interleave(128, 1)
    got = R.E4M3[q.long()] * step
    # (a value over the largest code by less than the bound goes to it)
    assert bool(((got - h).abs() <= dh + torch.maximum(2.0 ** -4 * (h.abs() + dh), 2.0 ** -10 * step)).all())


def combine(y, slots, weights, shared):
    """float64 (out, tol): top_k + 1 float32 sums of products, then bf16."""
    M, top = slots.shape
    out = shared.double().clone() if shared is not None else torch.zeros(M, y.shape[1], dtype=torch.float64)
    mag = out.abs()
    for m in range(M):
        for j in range(top):
            s = int(slots[m, j])
            if 0 <= s < y.shape[0]:
                t = weights[m, j].double() * y[s].double()
                out[m] += t
                mag[m] += t.abs()
    err = (2 * top + 2) * 2.0 ** -24 * mag
    return out, err + 2.0 ** -8 * (out.abs() + err)


def lora(out, x, a, b, offsets, rows, scales):
    """float64 (out, tol). The first product's K and the second's rank float32 sums
    are off by at most (K + 8) and (2 rank + 8) steps of 2^-23 of their terms'
    magnitudes (matrix cores that truncate), h's two bf16 parts by 2^-16 of it, its
    scale by 2^-24, then the sum's rounding to bf16."""
    K, rank = x.shape[1], a.shape[1]
    want, err = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64)
    for g in range(a.shape[0]):
        for i in range(int(offsets[g]), int(offsets[g + 1])):
            m = int(rows[i])
            if not 0 <= m < out.shape[0]:
                continue
            s = 1.0 if scales is None else float(scales[g])
            A, B, v = a[g].double(), b[g].double(), x[m].double()
            h = A @ v
            dh = (K + 8) * 2.0 ** -23 * (A.abs() @ v.abs()) + (2.0 ** -16 + 2.0 ** -23) * h.abs()
            want[m] += s * (B @ h)
            err[m] = abs(s) * (B.abs() @ dh + (2 * rank + 8) * 2.0 ** -23 * (B.abs() @ h.abs())) + 2.0 ** -23 * want[m].abs()
    return want, err + torch.where(err > 0, 2.0 ** -8, 0.0) * (want.abs() + err)
