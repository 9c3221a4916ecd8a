"""The operators around an attention layer with 8-bit operands: cases, inputs, plain forms and work.

Four operators, in the order a layer calls them:

* ``gemm``    block-scaled FP8 product: E4M3 activations with a UE8M0 scale per
  1x128 block times E4M3 weights with one per 128x128 tile, bf16 out;
* ``norm``    RMS norm of every query and key head with the rotary position
  embedding in the same pass;
* ``cache``   keys and values quantised to E4M3 as they are written to a paged
  cache (a UE8M0 scale per block of tokens and head), and read back;
* ``attend``  causal attention of bf16 queries over that cache.

``own`` selects who computes: false, elementary torch operations in float32;
true, the framework's kernels.
"""
import random

import torch

own = False

F8 = torch.float8_e4m3fn


# ----------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of one sequence: the low-rank query projection of a 7168-wide model
        dict(name="gemm_token", op="gemm", m=1, n=1536, k=7168),
        # a decode step of 32 sequences: the output projection of 64 heads of 128
        dict(name="gemm_decode", op="gemm", m=32, n=7168, k=8192),
        # prefill: the query projection of 4632 tokens to 64 heads of 128
        dict(name="gemm_prefill", op="gemm", m=4632, n=8192, k=1536),
        # a short prompt through a fused projection whose width is no multiple of a tile
        dict(name="gemm_ragged", op="gemm", m=777, n=2115, k=7168),
        # a decode step: 16 tokens, 64 query and 8 key heads
        dict(name="norm_decode", op="norm", m=16, hq=64, hk=8, d=128, rope=64, interleaved=False, shared=False),
        # prefill: queries and keys as column ranges of one fused projection's rows
        dict(name="norm_prefill", op="norm", m=4632, hq=64, hk=8, d=128, rope=64, interleaved=False, shared=True),
        # a decode step: one token more in each of 64 sequences, blocks partly filled
        dict(name="cache_decode", op="cache", seqs=64, new_lo=1, new_hi=1, past_lo=1, past_hi=1023, hk=8, d=128, block=64, read=False),
        # three ragged prompts written behind what they share, then read back whole
        dict(name="cache_prefill", op="cache", seqs=3, new_lo=900, new_hi=4632, past_lo=0, past_hi=700, hk=8, d=128, block=64, read=True),
        # a decode step of 64 sequences of very different lengths
        dict(name="attend_decode", op="attend", seqs=64, new_lo=1, new_hi=1, past_lo=127, past_hi=8191, hq=64, hk=8, d=128, block=64, window=0),
        # one long sequence, one token
        dict(name="attend_long", op="attend", seqs=1, new_lo=1, new_hi=1, past_lo=131071, past_hi=131071, hq=64, hk=8, d=128, block=64, window=0),
        # a prompt of 4632 tokens
        dict(name="attend_prefill", op="attend", seqs=1, new_lo=4632, new_hi=4632, past_lo=0, past_hi=0, hq=64, hk=8, d=128, block=64, window=0),
        # prompts being continued beside decoding sequences, short blocks, a sliding window
        dict(name="attend_mixed", op="attend", seqs=9, new_lo=1, new_hi=700, past_lo=0, past_hi=3000, hq=32, hk=4, d=64, block=16, window=1024),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("gemm", "gemm", "norm", "cache", "attend", "attend"))
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 4632), n=_log(rng, 256, 8192), k=128 * _log(rng, 4, 64) if rng.random() < 0.5 else 1536)
    if op == "norm":
        d = rng.choice((64, 128, 256))
        hk = rng.choice((1, 2, 4, 8))
        return dict(op=op, m=_log(rng, 1, 4632), hq=hk * rng.choice((1, 3, 4, 8)), hk=hk, d=d,
                    rope=rng.choice((d // 2, d, 32)), interleaved=rng.random() < 0.5, shared=rng.random() < 0.5)
    hk, d, block = rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    if op == "cache":
        new = _log(rng, 1, 2000)
        return dict(op=op, seqs=_log(rng, 1, 64 if new < 64 else 4), new_lo=max(1, new // 3), new_hi=new, past_lo=0,
                    past_hi=_log(rng, 1, 1000), hk=hk, d=d, block=block, read=rng.random() < 0.5)
    group = rng.choice((1, 3, 4, 8))
    if rng.random() < 0.6:      # decoding: one token or a few drafted ones
        past = _log(rng, 16, 32768)
        new = rng.choice((1, 1, 1, 2, 4))
        seqs = min(_log(rng, 1, 96), max(1, (1 << 19) // past))
        return dict(op=op, seqs=seqs, new_lo=new, new_hi=new, past_lo=past // 4, past_hi=past, hq=hk * group, hk=hk, d=d,
                    block=block, window=rng.choice((0, 0, 777)))
    new = _log(rng, 8, 2500)
    return dict(op=op, seqs=_log(rng, 1, 6), new_lo=max(1, new // 4), new_hi=new, past_lo=0, past_hi=_log(rng, 1, 2000),
                hq=hk * group, hk=hk, d=d, block=block, window=rng.choice((0, 0, 333)))


def _lens(case):
    """(new tokens, tokens held before) of every sequence, from the case alone: the largest of each
    range is always there, the others are spread over the range."""
    r = random.Random("%(seqs)d %(new_lo)d %(new_hi)d %(past_lo)d %(past_hi)d" % case)
    new = [case["new_hi"]] + [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"] - 1)]
    past = [case["past_hi"]] + [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"] - 1)]
    return new, past


def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = k // 128
        return {"bytes": m * k + n * k + 2 * m * n + 4 * m * -(-blocks // 4) + -(-n // 128) * blocks, "flops": 2 * m * n * k}
    if case["op"] == "norm":
        values = case["m"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 4 * values + case["m"] * (8 + 4 * case["rope"]) + 4 * case["d"], "flops": 8 * values}
    new, past = _lens(case)
    if case["op"] == "cache":
        row = 2 * case["hk"] * case["d"]                    # a token's keys and values
        touched = sum(-(-(p + t) // case["block"]) - p // case["block"] for t, p in zip(new, past))
        moved = 3 * row * sum(new) + 4 * case["hk"] * touched
        if case["read"]:
            moved += 3 * row * sum(t + p for t, p in zip(new, past))
        return {"bytes": moved, "flops": 2 * row * sum(new)}
    pairs = rows = 0
    for t, p in zip(new, past):
        w = case["window"] or p + t
        pairs += sum(min(i + 1, w) for i in range(p, p + t))
        rows += min(p + t, w + t - 1)
    kept = 2 * case["hk"] * case["d"] * rows
    return {"bytes": kept + 2 * case["hk"] * rows // case["block"] + 4 * sum(new) * case["hq"] * case["d"],
            "flops": 4 * case["d"] * case["hq"] * pairs}


# ---------------------------------------------------------------- inputs

def _power(e):
    """2^e in float32 for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_of(amax):
    """ceil(log2(amax / 448)), exact, for amax raised to at least 1e-4 (so at least -22)."""
    m, e = torch.frexp(amax.float().clamp_min(1e-4))        # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    return e.to(torch.int32) - 9 + (m > 0.875)


def _rows_in_blocks(x):
    """[M, K] -> E4M3 codes (uint8) and packed words of UE8M0 bytes, four 128-blocks to an int32."""
    m, k = x.shape
    b = x.float().view(m, k // 128, 128)
    e = _scale_of(b.abs().amax(2))
    codes = (b * _power(-e)[:, :, None]).to(F8).view(torch.uint8).view(m, k)
    bytes_ = torch.zeros(m, -(-k // 512) * 4, dtype=torch.uint8, device=x.device)
    bytes_[:, : k // 128] = e + 127
    return codes, bytes_.view(torch.int32)


def _weights_in_tiles(w):
    """[N, K], N a multiple of 128 -> E4M3 codes and UE8M0 bytes [N/128, K/128]."""
    n, k = w.shape
    t = w.float().view(n // 128, 128, k // 128, 128)
    e = _scale_of(t.abs().amax((1, 3)))
    codes = (t * _power(-e)[:, None, :, None]).to(F8).view(torch.uint8).view(n, k)
    return codes, (e + 127).to(torch.uint8)


def _cache_of(g, blocks, hk, d, block, dev):
    """A cache in use: every block holds codes and the scale that they were written with."""
    spread = torch.rand(d, generator=g, device=dev) * 2 + 0.25        # channels differ in size
    k = torch.randn(blocks, hk, block, d, generator=g, device=dev) * spread
    v = torch.randn(blocks, hk, d, block, generator=g, device=dev) * spread[:, None]
    ke, ve = _scale_of(k.abs().amax((2, 3))), _scale_of(v.abs().amax((2, 3)))
    k = (k * _power(-ke)[:, :, None, None]).to(F8).view(torch.uint8)
    v = (v * _power(-ve)[:, :, None, None]).to(F8).view(torch.uint8)
    return k, v, (ke + 127).to(torch.uint8), (ve + 127).to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        x = torch.randn(m, k, generator=g, device=dev)
        x[:, torch.randint(0, k, (4,), generator=g, device=dev)] *= 30    # a few channels stand out
        a, a_scales = _rows_in_blocks(x.to(torch.bfloat16))
        w = torch.randn(-(-n // 128) * 128, k, generator=g, device=dev) * 0.02
        w, w_scales = _weights_in_tiles(w)
        return dict(case=case, a=a, a_scales=a_scales, w=w[:n], w_scales=w_scales)
    if case["op"] == "norm":
        m, hq, hk, d, rope = (case[x] for x in ("m", "hq", "hk", "d", "rope"))
        size = 2.0 ** (torch.rand(m, hq + 2 * hk, 1, generator=g, device=dev) * 4 - 2)
        x = (torch.randn(m, hq + 2 * hk, d, generator=g, device=dev) * size).to(torch.bfloat16).view(m, -1)
        q, k = x[:, : hq * d], x[:, hq * d : (hq + hk) * d]
        if not case["shared"]:
            q, k = q.contiguous(), k.contiguous()
        qw, kw = ((1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2))
        length = 8192
        angle = torch.arange(length, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rope, 2, device=dev, dtype=torch.float64) / rope)
        table = torch.cat((angle.cos(), angle.sin()), 1).float()
        first = torch.randint(0, length - m, (1,), generator=g, device=dev)
        return dict(case=case, q=q, k=k, qw=qw, kw=kw, positions=first + torch.arange(m, device=dev), table=table)
    new, past = _lens(case)
    hk, d, block = case["hk"], case["d"], case["block"]
    lens = [t + p for t, p in zip(new, past)]
    width = -(-max(lens) // block)
    used = [-(-n // block) for n in lens]
    blocks = sum(used) + 5
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), 0, dtype=torch.int32)
    at = torch.tensor([0] + used).cumsum(0).tolist()
    order = order.cpu()
    for s, n in enumerate(used):
        table[s, :n] = order[at[s] : at[s] + n]
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    k, v, ks, vs = _cache_of(g, blocks, hk, d, block, dev)
    state = dict(case=case, k_cache=k, v_cache=v, k_scales=ks, v_scales=vs, table=table.to(dev), cu=cu.to(dev),
                 lens=torch.tensor(lens, dtype=torch.int32, device=dev), total=sum(new), most=max(new), longest=max(lens))
    if case["op"] == "cache":
        size = 2.0 ** (torch.rand(sum(new), 1, 1, generator=g, device=dev) * 3 - 1.5)
        state["k"], state["v"] = ((torch.randn(sum(new), hk, d, generator=g, device=dev) * size).to(torch.bfloat16)
                                  for _ in range(2))
        state["held"] = sum(lens)
        state["cu_held"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(dev)
    else:
        state["q"] = torch.randn(sum(new), case["hq"], d, generator=g, device=dev).to(torch.bfloat16)
    return state


# ------------------------------------------------------------------ runs

def run(state):
    return _RUN[state["case"]["op"]](state)


def _gemm(s):
    if own:
        import fp4_quantized_prep_amd as iqp
        return iqp.fp8_gemm_1x128_128x128(s["a"], s["a_scales"], s["w"], s["w_scales"])
    m, k = s["a"].shape
    n = s["w"].shape[0]
    sa = _power(s["a_scales"].view(torch.uint8)[:, : k // 128].to(torch.int32) - 127)
    sw = _power(s["w_scales"].to(torch.int32) - 127).repeat_interleave(128, 0)[:n]
    a = s["a"].view(F8).float().view(m, k // 128, 128) * sa[:, :, None]
    w = s["w"].view(F8).float().view(n, k // 128, 128) * sw[:, :, None]
    return (a.view(m, k) @ w.view(n, k).t()).to(torch.bfloat16)


def _norm(s):
    c = s["case"]
    if own:
        import fp4_quantized_prep_amd as iqp
        return iqp.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["table"], eps=1e-6, head_dim=c["d"],
                                rope_layout="interleaved" if c["interleaved"] else "half_split")
    m, half = c["m"], c["rope"] // 2
    row = s["table"][s["positions"]]
    cos, sin = row[:, None, :half], row[:, None, half:]

    def one(x, w):
        x = x.reshape(m, -1, c["d"]).float()
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w.float()
        if c["interleaved"]:
            a, b = x[:, :, 0 : 2 * half : 2], x[:, :, 1 : 2 * half : 2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
        else:
            a, b = x[:, :, :half], x[:, :, half : 2 * half]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
        return torch.cat((turned, x[:, :, 2 * half :]), 2).view(m, -1).to(torch.bfloat16)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _places(lens, cu, total):
    """Sequence and position of each of `total` rows: the rows of a sequence are its last tokens."""
    row = torch.arange(total, device=lens.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, (row - cu[seq + 1] + lens[seq]).long()


def _cache(s):
    c = s["case"]
    if own:
        import fp4_quantized_prep_amd as iqp
        cache = iqp.Fp8KvCache(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        iqp.kv_cache_append_fp8(s["k"], s["v"], cache, s["table"], s["lens"], s["cu"])
        if c["read"]:
            return (*iqp.kv_cache_read_fp8(cache, s["table"], s["lens"], s["cu_held"], s["held"]), cache.k_scales, cache.v_scales)
        return cache.k.view(F8), cache.v.view(F8), cache.k_scales, cache.v_scales
    block = c["block"]
    seq, pos = _places(s["lens"], s["cu"], s["total"])
    held, at = s["table"][seq, pos // block].long(), pos % block
    first = (s["lens"] - (s["cu"][1:] - s["cu"][:-1])).long()          # the first new position of each sequence
    old_block = s["table"].gather(1, (first // block).clamp_max(s["table"].shape[1] - 1)[:, None])[:, 0].long()
    before = (torch.arange(block, device=pos.device) < (first % block)[:, None]) & (s["cu"][1:] > s["cu"][:-1])[:, None]

    def one(x, codes, scales, rows):       # rows: the codes with a block's tokens in the third place
        amax = torch.zeros(scales.shape, device=x.device).index_reduce_(0, held, x.float().abs().amax(2), "amax")
        fresh = torch.zeros(scales.shape[0], device=x.device).index_reduce_(0, held, (at == 0).float(), "amax") > 0
        touched = torch.zeros(scales.shape[0], device=x.device).index_fill_(0, held, 1.0) > 0
        old = scales.to(torch.int32) - 127
        need = _scale_of(amax)
        e = torch.where(touched[:, None], torch.where(fresh[:, None], need, torch.maximum(need, old)), old)
        kept = rows[old_block].view(F8).float()
        grown = (kept * _power((old - e)[old_block].clamp(-126, 0))[:, :, None, None]).to(F8).view(torch.uint8)
        rows[old_block] = torch.where(before[:, None, :, None], grown, rows[old_block])
        rows[held, :, at] = (x.float() * _power(-e[held])[:, :, None]).to(F8).view(torch.uint8)
        scales.copy_(e + 127)

    one(s["k"], s["k_cache"], s["k_scales"], s["k_cache"])
    one(s["v"], s["v_cache"], s["v_scales"], s["v_cache"].transpose(2, 3))
    if not c["read"]:
        return s["k_cache"].view(F8), s["v_cache"].view(F8), s["k_scales"], s["v_scales"]
    seq, pos = _places(s["lens"], s["cu_held"], s["held"])
    held, at = s["table"][seq, pos // block].long(), pos % block
    k = s["k_cache"][held, :, at].view(F8).float() * _power(s["k_scales"][held].to(torch.int32) - 127)[:, :, None]
    v = s["v_cache"][held, :, :, at].view(F8).float() * _power(s["v_scales"][held].to(torch.int32) - 127)[:, :, None]
    return k.to(torch.bfloat16), v.to(torch.bfloat16), s["k_scales"], s["v_scales"]


def _attend(s):
    c = s["case"]
    if own:
        import fp4_quantized_prep_amd as iqp
        cache = iqp.Fp8KvCache(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        return iqp.attention_fp8_kv(s["q"], cache, s["table"], s["lens"], s["cu"], window=c["window"])
    hq, hk, d, block = c["hq"], c["hk"], c["d"], c["block"]
    n, length, most = s["lens"].shape[0], s["table"].shape[1] * block, s["most"]
    t = s["table"].long()
    k = s["k_cache"][t].view(F8).float() * _power(s["k_scales"][t].to(torch.int32) - 127)[..., None, None]
    v = s["v_cache"][t].view(F8).float() * _power(s["v_scales"][t].to(torch.int32) - 127)[..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(n, hk, d, length)              # tokens last
    v = v.permute(0, 2, 1, 4, 3).reshape(n, hk, length, d)
    new = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(most, device=t.device)
    row = (s["cu"][:-1, None] + torch.minimum(i, new[:, None] - 1)).long()
    q = s["q"][row].float().view(n, most, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    score = (q @ k * d ** -0.5).view(n, hk, hq // hk, most, length)
    here = (s["lens"] - new)[:, None] + i                               # [n, most]: the position of a query
    there = torch.arange(length, device=t.device)
    seen = there <= here[:, :, None]
    if c["window"]:
        seen &= there > here[:, :, None] - c["window"]
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    score -= score.amax(4, keepdim=True).clamp_min(-1e30)
    score.exp_()
    total = score.sum(4, keepdim=True)
    out = (score.view(n, hk, -1, length) @ v).view(n, hk, -1, most, d) / total.clamp_min(1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)
    seq, pos = _places(s["lens"], s["cu"], s["total"])
    return out[seq, pos - (s["lens"] - new)[seq]].to(torch.bfloat16)


_RUN = {"gemm": _gemm, "norm": _norm, "cache": _cache, "attend": _attend}


# ----------------------------------------------------------------- exact

def _two(dev):
    """2^(b - 127) in float64 for every UE8M0 byte b."""
    return torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device=dev)


def _e4m3(dev):
    """The value of every E4M3 code in float64."""
    out = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append(float("nan") if c & 127 == 127 else -x if c >> 7 else x)
    return torch.tensor(out, dtype=torch.float64, device=dev)


def _nearest_e4m3(x):
    """The E4M3 value nearest to each x (float64), ties to the even code."""
    e = torch.frexp(x)[1].clamp_min(-5) - 1                             # |x| in [2^e, 2^(e+1)), subnormals below 2^-6
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    dev = torch.device("cuda")
    two, value = _two(dev), _e4m3(dev)
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        shift = torch.arange(0, 32, 8, device=dev)
        bytes_ = (s["a_scales"].long()[:, :, None] >> shift & 255).flatten(1)
        out = torch.zeros(m, n, dtype=torch.float64, device=dev)
        for j in range(k // 128):
            cols = slice(128 * j, 128 * j + 128)
            a = value[s["a"][:, cols].long()] * two[bytes_[:, j]][:, None]
            w = value[s["w"][:, cols].long()] * two[s["w_scales"][:, j].long()].repeat_interleave(128)[:n, None]
            out.addmm_(a, w.t().contiguous())
        return out
    if case["op"] == "norm":
        half = case["rope"] // 2
        turn = torch.complex(s["table"][:, :half].double(), s["table"][:, half:].double())[s["positions"]]

        def one(x, w):
            x = x.double().reshape(case["m"], -1, case["d"])
            y = x / torch.sqrt(x.square().sum(2, keepdim=True) / case["d"] + 1e-6) * w.double()
            if case["interleaved"]:
                z = torch.complex(y[..., : 2 * half : 2], y[..., 1 : 2 * half : 2]) * turn[:, None]
                y[..., : 2 * half : 2], y[..., 1 : 2 * half : 2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :half], y[..., half : 2 * half]) * turn[:, None]
                y[..., :half], y[..., half : 2 * half] = z.real, z.imag
            return y.reshape(case["m"], -1)

        return one(s["q"], s["qw"]), one(s["k"], s["kw"])
    new, past = _lens(case)
    block, table = case["block"], s["table"].tolist()
    if case["op"] == "cache":
        kept = [value[s["k_cache"].long()], value[s["v_cache"].long()].transpose(2, 3).contiguous()]
        scales = [s["k_scales"].long() - 127, s["v_scales"].long() - 127]
        at = 0
        for i, (t, p) in enumerate(zip(new, past)):
            for b in range(p // block, -(-(p + t) // block)):
                lo, hi = max(p - b * block, 0), min(p + t - b * block, block)
                rows = slice(at + b * block + lo - p, at + b * block + hi - p)
                for x, codes, e in ((s["k"], *(kept[0], scales[0])), (s["v"], *(kept[1], scales[1]))):
                    x = x[rows].double()
                    need = torch.searchsorted(448 * two, x.abs().amax((0, 2)).clamp_min(1e-4)) - 127     # the least with 448 2^e >= amax
                    h = table[i][b]
                    if lo:
                        need = torch.maximum(need, e[h])
                        codes[h, :, :lo] = _nearest_e4m3(codes[h, :, :lo] * two[e[h] - need + 127][:, None, None])
                    codes[h, :, lo:hi] = _nearest_e4m3(x / two[need + 127][:, None]).transpose(0, 1)
                    e[h] = need
            at += t
        if not case["read"]:
            return kept[0], kept[1].transpose(2, 3).contiguous(), None, None
        out = []
        for codes, e in zip(kept, scales):
            whole = (codes * two[e + 127][:, :, None, None]).transpose(1, 2)      # [blocks, tokens, heads, d]
            out.append(torch.cat([whole[table[i][: -(-(t + p) // block)]].flatten(0, 1)[: t + p]
                                  for i, (t, p) in enumerate(zip(new, past))]))
        return out[0], out[1], None, None
    if 8 * max(t * (t + p) for t, p in zip(new, past)) * case["hq"] // case["hk"] > 16 << 30:
        return None
    hq, hk, d = case["hq"], case["hk"], case["d"]
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device=dev)
    at = 0
    for i, (t, p) in enumerate(zip(new, past)):
        n = t + p
        h = s["table"][i, : -(-n // block)].long()
        here = torch.arange(p, n, device=dev)[:, None]
        there = torch.arange(n, device=dev)[None]
        unseen = (there > here) | ((there <= here - case["window"]) if case["window"] else False)
        for j in range(hk):
            k = value[s["k_cache"][h, j].long()] * two[s["k_scales"][h, j].long()][:, None, None]
            v = value[s["v_cache"][h, j].long()] * two[s["v_scales"][h, j].long()][:, None, None]
            k, v = k.flatten(0, 1)[:n], v.transpose(1, 2).flatten(0, 1)[:n]
            for x in range(j * (hq // hk), (j + 1) * (hq // hk)):
                z = s["q"][at : at + t, x].double() @ k.t().contiguous() / d ** 0.5
                out[at : at + t, x] = torch.softmax(z.masked_fill(unseen, float("-inf")), 1) @ v
        at += t
    return out
