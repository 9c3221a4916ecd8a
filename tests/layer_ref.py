"""Plain float64 implementations of the attention layer's operators (test
infrastructure only; shares no code with the kernels). Tensors are on the CPU."""
import math

import torch


def e4m3_values() -> torch.Tensor:
    """float64 value of every E4M3 ("fn") code."""
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out.append(math.nan if c & 127 == 127 else -v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


E4M3 = e4m3_values()


def e4m3_code(x: torch.Tensor) -> torch.Tensor:
    """uint8 code of the E4M3 value nearest to each |x| <= 448, ties to the even
    code; the sign of zero is that of x."""
    pos = E4M3[:127]                                   # codes 0 .. 126, increasing
    a = x.abs().double()
    hi = torch.searchsorted(pos, a.contiguous()).clamp(0, 126)
    lo = (hi - 1).clamp_min(0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (pick + 128 * torch.signbit(x)).to(torch.uint8)


def exponent(amax: float) -> int:
    """The least e >= -22 with 448 * 2^e >= max(amax, 1e-4)."""
    a = max(amax, 1e-4)
    e = -22
    while 448.0 * 2.0 ** e < a:
        e += 1
    return e


def append(cache, k, v, table, lens, cu):
    """cache: dict of CPU uint8 tensors k [n, h, b, d], v [n, h, d, b], ks, vs
    [n, h]; changed in place as kv_cache_append_fp8 says."""
    n, h, b, d = cache["k"].shape
    views = {"k": cache["k"], "v": cache["v"].transpose(2, 3)}
    for s in range(len(lens)):
        rows = list(range(cu[s], cu[s + 1]))
        by_block = {}
        for i, r in enumerate(rows):
            p = lens[s] - len(rows) + i
            if p < 0 or p // b >= table.shape[1]:
                continue
            blk = int(table[s, p // b])
            if 0 <= blk < n:
                by_block.setdefault(blk, []).append((p % b, r))
        for blk, items in by_block.items():
            lo = items[0][0]
            for name, x in (("k", k), ("v", v)):
                sc = cache[name + "s"]
                for j in range(h):
                    new = torch.stack([x[r, j] for _, r in items]).double()
                    e = exponent(float(new.abs().max()))
                    if lo:
                        old = int(sc[blk, j]) - 127
                        if e > old:
                            kept = E4M3[views[name][blk, j, :lo].long()]
                            views[name][blk, j, :lo] = e4m3_code(kept * 2.0 ** (old - e))
                        e = max(e, old)
                    views[name][blk, j, lo:lo + len(items)] = e4m3_code(new * 2.0 ** -e)
                    sc[blk, j] = e + 127


def held_values(cache, table, s, length):
    """(k, v, held): float64 [length, h, d] values of a sequence's positions and
    which of them are held."""
    n, h, b, d = cache["k"].shape
    k = torch.zeros(length, h, d, dtype=torch.float64)
    v = torch.zeros(length, h, d, dtype=torch.float64)
    held = torch.zeros(length, dtype=torch.bool)
    for i in range(-(-length // b)):
        blk = int(table[s, i]) if i < table.shape[1] else -1
        if not 0 <= blk < n:
            continue
        m = min(b, length - i * b)
        sk = 2.0 ** (cache["ks"][blk].double() - 127)
        sv = 2.0 ** (cache["vs"][blk].double() - 127)
        k[i * b:i * b + m] = (E4M3[cache["k"][blk, :, :m].long()] * sk[:, None, None]).transpose(0, 1)
        v[i * b:i * b + m] = (E4M3[cache["v"][blk, :, :, :m].long()] * sv[:, None, None]).permute(2, 0, 1)
        held[i * b:i * b + m] = True
    return k, v, held


def attention(q, cache, table, lens, cu, scale, window):
    """float64 (out, tol) of attention_fp8_kv for bf16 q [T, hq, d]; rows past
    cu[-1] are NaN. tol bounds the kernel's distance from out:

    * the rounding to bf16: 2^-8 |out|;
    * the scores: D products summed in float32 and scaled, off by at most
      (D + 3) 2^-23 sum |q k| scale log2(e) + 2^-20 in units of log2 (the last
      term: the subtraction of the maximum and exp2 for scores below 2^3 ..
      2^10), which changes a weight by at most that much relatively;
    * the weights in fp16: 2^-11 relatively, or 2^-25 of the largest w 2^e
      where they are subnormal, times values of at most 448 2^e <= 2 max |v| of
      the block with the largest: length * 2^-24 * max |v| in all.
    """
    T, hq, d = q.shape
    h = cache["k"].shape[1]
    out = torch.full((T, hq, d), math.nan, dtype=torch.float64)
    tol = torch.zeros((T, hq, d), dtype=torch.float64)
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        if n <= 0:
            continue
        length = max(lens[s], 0)
        k, v, held = held_values(cache, table, s, length)
        for i in range(n):
            p = lens[s] - n + i
            t = torch.arange(length)
            seen = held & (t <= p)
            if window:
                seen &= t > p - window
            r = cu[s] + i
            if not seen.any():
                out[r] = 0.0
                continue
            ks, vs = k[seen], v[seen]
            for x in range(hq):
                j = x // (hq // h)
                qq = q[r, x].double()
                z = (ks[:, j] @ qq) * scale
                w = torch.softmax(z, 0)
                out[r, x] = w @ vs[:, j]
                delta = (d + 3) * 2.0 ** -23 * float((ks[:, j].abs() @ qq.abs()).max()) * scale * 1.4427 + 2.0 ** -20
                rel = 2.0 ** -11 + 2 * delta
                tol[r, x] = 2.0 ** -8 * out[r, x].abs() + rel * (w @ vs[:, j].abs()) + \
                    length * 2.0 ** -24 * float(vs[:, j].abs().max())
    return out, tol


def norm_rope(x, w, positions, cos_sin, eps, interleaved):
    """float64 (out, tol) for bf16 x [M, H, D]. tol: the rounding to bf16, and
    2^-19 of the two terms of the rotation for float32: the sum of squares is
    off by at most 21 half steps, its root by half of that, and the products
    and the sum by six more: under 20 * 2^-24."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    rd = cos_sin.shape[1]
    half = rd // 2
    pos = positions.clamp(0, cos_sin.shape[0] - 1)
    c, s = cos_sin[pos, :half].double()[:, None], cos_sin[pos, half:].double()[:, None]
    out, mag = y.clone(), y.abs().clone()
    ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return out, 2.0 ** -8 * out.abs() + 2.0 ** -19 * mag


def dequant_rows(codes, words):
    """float64 [M, K] values of E4M3 codes and packed scale words."""
    M, K = codes.shape
    b = torch.stack([(words.long() >> (8 * t)) & 255 for t in range(4)], -1).flatten(1)[:, : K // 128]
    return E4M3[codes.long()] * (2.0 ** (b.double() - 127)).repeat_interleave(128, 1)


def dequant_tiles(codes, scales):
    """float64 [N, K] values of E4M3 codes and 128x128 tile scales (the last
    row of tiles may be partial)."""
    s = 2.0 ** (scales.double() - 127)
    return E4M3[codes.long()] * s.repeat_interleave(128, 0)[: codes.shape[0]].repeat_interleave(128, 1)
