"""Operators whose weights depend on the token: experts and adapters. Cases, inputs, plain forms and work.

Five operators, beside the layer's block-scaled FP8 product:

* ``route``    the top experts of every token from the router's logits, their weights, and the tokens
  sorted by expert (the plan that the products below read);
* ``swiglu``   the experts' first product, gate and up halves at once, E4M3 activations (a UE8M0 scale per
  1x128 block) times E4M3 weights (one per 128x128 tile), silu(gate) * up, quantised again in 1x128 blocks;
* ``product``  the same kind of product for rows sorted by group, bf16 out (the experts' second product);
* ``combine``  every token's weighted sum of its experts' rows, with the shared expert's row;
* ``lora``     low-rank bf16 adapters of many requests added to a shared projection's output.

``own`` selects who computes: false, elementary torch operations in float32 (the router in float64); true,
the framework's kernels.
"""
import random

import torch

own = False

F8 = torch.float8_e4m3fn


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one token through a router of 256 experts that balances its load with a bias
        dict(name="route_token", op="route", m=1, groups=256, top=8, scoring="sigmoid", bias=True, half=False, skew=0.5),
        # a prompt of 4632 tokens through it
        dict(name="route_prefill", op="route", m=4632, groups=256, top=8, scoring="sigmoid", bias=True, half=False, skew=0.5),
        # a decode step of 32 tokens, 8 of 64 experts each: the first product reads nearly all of the weights
        dict(name="swiglu_decode", op="swiglu", m=32, groups=64, top=8, n=2048, k=7168, skew=0.5),
        # a prompt of 4632 tokens, about 580 rows an expert
        dict(name="swiglu_prefill", op="swiglu", m=4632, groups=64, top=8, n=2048, k=7168, skew=0.5),
        # one token's second product: eight experts, one row each
        dict(name="product_token", op="product", m=1, groups=64, top=8, n=7168, k=2048, gather=False, skew=0.5),
        # the prompt's second product
        dict(name="product_prefill", op="product", m=4632, groups=64, top=8, n=7168, k=2048, gather=False, skew=0.5),
        # few popular experts, a width that is no multiple of a tile, rows gathered from the tokens
        dict(name="product_ragged", op="product", m=777, groups=40, top=4, n=2115, k=1536, gather=True, skew=1.5),
        # a decode step of 16 tokens
        dict(name="combine_decode", op="combine", m=16, top=8, d=7168, shared=True),
        # the prompt
        dict(name="combine_prefill", op="combine", m=4632, top=8, d=7168, shared=True),
        # a decode step of 64 requests over 32 adapters of rank 16: the low-rank query projection
        dict(name="lora_decode", op="lora", m=64, requests=64, groups=32, rank=16, n=1536, k=7168),
        # four prompts of one batch, adapters of rank 64 beside the projection to 64 heads of 128
        dict(name="lora_prefill", op="lora", m=4632, requests=4, groups=8, rank=64, n=8192, k=1536),
        # prompts beside decoding requests, odd sizes
        dict(name="lora_mixed", op="lora", m=999, requests=41, groups=20, rank=24, n=2115, k=7168),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("route", "swiglu", "swiglu", "product", "product", "combine", "lora", "lora"))
    groups = rng.choice((8, 16, 40, 64, 128))
    top = rng.choice((1, 2, 4, 6, 8))
    skew = rng.choice((0.0, 0.5, 1.5))
    if op == "route":
        return dict(op=op, m=_log(rng, 1, 4632), groups=rng.choice((8, 60, 64, 160, 256)), top=top,
                    scoring=rng.choice(("softmax", "sigmoid", "sqrt_softplus")), bias=rng.random() < 0.5, half=rng.random() < 0.3, skew=skew)
    if op == "combine":
        return dict(op=op, m=_log(rng, 1, 4632), top=top, d=8 * _log(rng, 64, 896), shared=rng.random() < 0.5)
    if op == "lora":
        m = _log(rng, 1, 4632)
        return dict(op=op, m=m, requests=min(m, _log(rng, 1, 128)), groups=_log(rng, 1, 64), rank=8 * _log(rng, 1, 16),
                    n=_log(rng, 256, 8192), k=8 * _log(rng, 64, 896))
    m = _log(rng, 1, 4096)
    while groups * top * m > 1 << 21:      # (many rows of many experts cost the most)
        m = max(1, m // 2)
    if op == "swiglu":
        return dict(op=op, m=m, groups=groups, top=top, n=128 * _log(rng, 2, 16), k=128 * _log(rng, 4, 56), skew=skew)
    return dict(op=op, m=m, groups=groups, top=top, n=_log(rng, 256, 7168), k=128 * _log(rng, 2, 32), gather=rng.random() < 0.5,
                skew=skew)


def _reached(case):
    """Groups that a batch reaches, of `groups`, were they all as likely."""
    return min(case["groups"], round(case["groups"] * (1 - (1 - case["top"] / case["groups"]) ** case["m"])) or 1)


def work(case):
    op, m = case["op"], case["m"]
    if op == "route":
        flat = m * case["top"]
        return {"bytes": m * case["groups"] * (2 if case["half"] else 4) + 16 * flat + 4 * case["groups"], "flops": 12 * m * case["groups"]}
    if op == "combine":
        d, top = case["d"], case["top"]
        return {"bytes": 2 * m * d * (top + 1 + case["shared"]) + 8 * m * top, "flops": 2 * m * d * (top + case["shared"])}
    n, k = case["n"], case["k"]
    if op == "lora":
        adapters = min(case["groups"], case["requests"])
        return {"bytes": 2 * m * k + 4 * m * n + 2 * adapters * case["rank"] * (n + k), "flops": 2 * m * case["rank"] * (n + k)}
    r, kb = m * case["top"], k // 128
    read = (m if op == "swiglu" or case["gather"] else r) * (k + 4 * -(-kb // 4))
    if op == "swiglu":
        return {"bytes": read + _reached(case) * 2 * n * (k + kb // 128) + r * (n + 4 * -(-n // 512)), "flops": 4 * r * n * k}
    return {"bytes": read + _reached(case) * (n * k + -(-n // 128) * kb) + 2 * r * n, "flops": 2 * r * n * k}


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


def _expert_weights(g, groups, n, k, dev):
    """E4M3 codes [groups, n, k] and UE8M0 bytes [groups, ceil(n / 128), k / 128] of random weights."""
    rows = -(-n // 128) * 128
    codes = torch.empty(groups, rows, k, dtype=torch.uint8, device=dev)
    scales = torch.empty(groups, rows // 128, k // 128, dtype=torch.uint8, device=dev)
    for i in range(groups):
        t = (torch.randn(rows, k, generator=g, device=dev) * 0.02).view(rows // 128, 128, k // 128, 128)
        e = _scale_of(t.abs().amax((1, 3)))
        codes[i] = (t * _power(-e)[:, None, :, None]).to(F8).view(torch.uint8).view(rows, k)
        scales[i] = e + 127
    return codes[:, :n], scales


def _logits(g, m, groups, skew, dev):
    """A router's logits: some experts are more popular than others."""
    return torch.randn(m, groups, generator=g, device=dev) + skew * torch.randn(groups, generator=g, device=dev)


def _plan(index, groups):
    """The flat entries of `index` sorted by group: (offsets [groups + 1], rows, slots in index's shape). An
    entry outside [0, groups) is in no group: rows ends with -1 for each of them, and its slot is -1."""
    flat = index.reshape(-1)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(groups + 1, dtype=key.dtype, device=key.device))
    place = torch.arange(flat.shape[0], device=key.device)
    rows = torch.where(place < offsets[groups], order, -1)
    slots = torch.empty_like(order).scatter_(0, order, torch.where(place < offsets[groups], place, -1))
    return offsets.to(torch.int32), rows.to(torch.int32), slots.view(index.shape).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, m = case["op"], case["m"]
    if op == "route":
        logits = 1.5 * _logits(g, m, case["groups"], case["skew"], dev)
        bias = 0.2 * torch.randn(case["groups"], generator=g, device=dev) if case["bias"] else None
        return dict(case=case, logits=logits.to(torch.bfloat16) if case["half"] else logits, bias=bias)
    if op == "combine":
        groups = 64
        index = torch.topk(_logits(g, m, groups, 0.5, dev), case["top"], 1).indices.to(torch.int32)
        weights = torch.softmax(torch.randn(m, case["top"], generator=g, device=dev), 1)
        y, shared = (torch.randn(rows, case["d"], generator=g, device=dev).to(torch.bfloat16) for rows in (m * case["top"], m))
        return dict(case=case, plan=_plan(index, groups), y=y, weights=weights, shared=shared if case["shared"] else None)
    n, k, groups = case["n"], case["k"], case["groups"]
    if op == "lora":
        adapter = torch.randint(0, groups, (case["requests"],), generator=g, device=dev)
        adapter[torch.rand(case["requests"], generator=g, device=dev) < 0.1] = -1           # requests without one
        cuts = torch.cat([torch.randperm(m - 1, generator=g, device=dev)[: case["requests"] - 1] + 1,
                          torch.zeros(1, dtype=torch.int64, device=dev)]).sort().values
        request = torch.searchsorted(cuts, torch.arange(m, device=dev), right=True) - 1
        plan = _plan(adapter[request].to(torch.int32), groups)
        most = int((plan[0][1:] - plan[0][:-1]).max())
        x = torch.randn(m, k, generator=g, device=dev).to(torch.bfloat16)
        a = (torch.randn(groups, case["rank"], k, generator=g, device=dev) * k ** -0.5).to(torch.bfloat16)
        b = (torch.randn(groups, n, case["rank"], generator=g, device=dev) * 0.05).to(torch.bfloat16)
        scales = 0.5 + 1.5 * torch.rand(groups, generator=g, device=dev)
        out = torch.randn(m, n, generator=g, device=dev).to(torch.bfloat16)
        return dict(case=case, plan=plan, most=max(1, most), x=x, a=a, b=b, scales=scales, out=out)
    index = torch.topk(_logits(g, m, groups, case["skew"], dev), case["top"], 1).indices.to(torch.int32)
    plan = _plan(index, groups)
    most = int((plan[0][1:] - plan[0][:-1]).max())
    gather = op == "swiglu" or case["gather"]
    x = torch.randn(m if gather else m * case["top"], k, generator=g, device=dev)
    x[:, torch.randint(0, k, (4,), generator=g, device=dev)] *= 30    # a few channels stand out
    a, a_scales = _rows_in_blocks(x.to(torch.bfloat16))
    w, w_scales = _expert_weights(g, groups, 2 * n if op == "swiglu" else n, k, dev)
    return dict(case=case, plan=plan, most=most, a=a, a_scales=a_scales, w=w, w_scales=w_scales)


# ------------------------------------------------------------------ runs

def run(state):
    return _RUN[state["case"]["op"]](state)


def _route(s):
    c = s["case"]
    if own:
        import fp4_quantized_prep_amd as iqp
        weights, experts = iqp.moe_route(s["logits"], c["top"], bias=s["bias"], scoring=c["scoring"], scale=2.5)
        plan = iqp.group_rows(experts, c["groups"])
        return weights, experts, plan.offsets, plan.rows, plan.slots
    z = s["logits"].double()
    if c["scoring"] == "softmax":
        p = (z - z.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
    elif c["scoring"] == "sigmoid":
        p = 1 / (1 + (-z).exp())
    else:
        p = (z.clamp_min(0) + torch.log1p((-z.abs()).exp())).sqrt()
    choice = z if s["bias"] is None else p + s["bias"].double()
    experts = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, : c["top"]]
    weights = p.gather(1, experts)
    weights = 2.5 * weights / weights.sum(1, keepdim=True)
    experts = experts.to(torch.int32)
    return weights.float(), experts, *_plan(experts, c["groups"])


def _by_group(plan, most):
    """Places [groups, most] of each group's rows (the last ones repeat where a group has fewer), and for
    every place its group and its number within it."""
    offsets = plan[0].long()
    place = (offsets[:-1, None] + torch.arange(most, device=offsets.device)).clamp_max(plan[1].shape[0] - 1)
    at = torch.arange(plan[1].shape[0], device=offsets.device)
    group = torch.searchsorted(offsets[1:].contiguous(), at, right=True).clamp_max(offsets.shape[0] - 2)
    return place, group, (at - offsets[group]).clamp_max(most - 1)


def _grouped(s):
    """Every place's row of its group's product, float32."""
    place, group, number = _by_group(s["plan"], s["most"])
    k, n = s["a"].shape[1], s["w"].shape[1]
    src = place
    if s["case"]["op"] == "swiglu" or s["case"]["gather"]:
        src = s["plan"][1].long()[place].clamp_min(0) // s["case"]["top"]
    a = s["a"].view(F8).float().unflatten(1, (k // 128, 128))
    a = (a * _power(s["a_scales"].view(torch.uint8)[:, : k // 128].to(torch.int32) - 127)[:, :, None]).flatten(1)
    w = s["w"].view(F8).float().unflatten(2, (k // 128, 128))
    w = (w * _power(s["w_scales"].to(torch.int32) - 127).repeat_interleave(128, 1)[:, :n, :, None]).flatten(2)
    return torch.bmm(a[src], w.transpose(1, 2))[group, number]


def _swiglu(s):
    if own:
        import fp4_quantized_prep_amd as iqp
        q, words = iqp.fp8_grouped_swiglu_1x128(s["a"], s["a_scales"], s["w"], s["w_scales"], iqp.RowGroups(*s["plan"]), gather=True)
    else:
        gate, up = _grouped(s).chunk(2, 1)
        q, words = _rows_in_blocks(gate / (1 + (-gate).exp()) * up)
    return q.view(F8), words.view(torch.uint8)[:, : s["case"]["n"] // 128].view(torch.float8_e8m0fnu)


def _product(s):
    if own:
        import fp4_quantized_prep_amd as iqp
        return iqp.fp8_grouped_gemm_1x128_128x128(s["a"], s["a_scales"], s["w"], s["w_scales"], iqp.RowGroups(*s["plan"]),
                                                  gather=s["case"]["gather"])
    return _grouped(s).to(torch.bfloat16)


def _combine(s):
    if own:
        import fp4_quantized_prep_amd as iqp
        return iqp.moe_combine(s["y"], iqp.RowGroups(*s["plan"]), s["weights"], shared=s["shared"])
    out = (s["y"].float()[s["plan"][2].long()] * s["weights"][:, :, None]).sum(1)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return out.to(torch.bfloat16)


def _lora(s):
    if own:
        import fp4_quantized_prep_amd as iqp
        return iqp.lora_add(s["out"], s["x"], s["a"], s["b"], iqp.RowGroups(*s["plan"]), scales=s["scales"])
    offsets, rows, slots = s["plan"]
    place, group, number = _by_group(s["plan"], s["most"])
    x = s["x"].float()[rows.long()[place].clamp_min(0)]
    h = torch.bmm(x, s["a"].float().transpose(1, 2)) * s["scales"][:, None, None]
    slot = slots.long().clamp_min(0)
    added = torch.bmm(h, s["b"].float().transpose(1, 2))[group[slot], number[slot]]
    s["out"].copy_(torch.where(slots[:, None] >= 0, s["out"].float() + added, s["out"].float()))
    return s["out"]


_RUN = {"route": _route, "swiglu": _swiglu, "product": _product, "combine": _combine, "lora": _lora}


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
    op = case["op"]
    if work(case)["flops"] > 6e14 and op != "route":
        return None
    s = prepare(case, seed)
    dev = torch.device("cuda")
    if op == "route":
        z = s["logits"].double()
        if case["scoring"] == "softmax":
            p = torch.softmax(z, 1)
        elif case["scoring"] == "sigmoid":
            p = torch.sigmoid(z)
        else:
            p = torch.logaddexp(z, torch.zeros_like(z)).sqrt()
        left = z.clone() if s["bias"] is None else p + s["bias"].double()
        number = torch.arange(case["groups"], device=dev)
        got = []
        for _ in range(case["top"]):
            best = left.max(1, keepdim=True).values
            first = torch.where(left == best, number, case["groups"]).min(1, keepdim=True).values
            got.append(p.gather(1, first))
            left.scatter_(1, first, float("-inf"))
        got = torch.cat(got, 1)
        return 2.5 * got / got.sum(1, keepdim=True), None, None, None, None
    offsets, rows, slots = s["plan"]
    at = offsets.tolist()
    if op == "combine":
        out = s["shared"].double() if case["shared"] else torch.zeros(case["m"], case["d"], dtype=torch.float64, device=dev)
        for j in range(case["top"]):
            out = out + s["weights"][:, j, None].double() * s["y"][slots[:, j].long()].double()
        return out
    if op == "lora":
        out = s["out"].double()
        for i in range(case["groups"]):
            r = rows[at[i] : at[i + 1]].long()
            if len(r):
                h = s["x"][r].double() @ s["a"][i].double().t().contiguous()
                out[r] += s["scales"][i].double() * (h @ s["b"][i].double().t().contiguous())
        return out
    two, value = _two(dev), _e4m3(dev)
    k, n = case["k"], s["w"].shape[1]
    shift = torch.arange(0, 32, 8, device=dev)
    words = (s["a_scales"].long()[:, :, None] >> shift & 255).flatten(1)
    gather = op == "swiglu" or case["gather"]
    out = torch.empty(rows.shape[0], n, dtype=torch.float64, device=dev)
    for i in range(case["groups"]):
        r = torch.arange(at[i], at[i + 1], device=dev)
        if len(r) == 0:
            continue
        if gather:
            r = rows[r].long() // case["top"]
        a = value[s["a"][r].long()] * two[words[r][:, : k // 128]].repeat_interleave(128, 1)
        w = value[s["w"][i].long()] * two[s["w_scales"][i].long()].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        out[at[i] : at[i + 1]] = a @ w.t().contiguous()
    if op == "product":
        return out
    h = (out[:, : n // 2] * torch.sigmoid(out[:, : n // 2]) * out[:, n // 2 :]).unflatten(1, (n // 256, 128))
    byte = torch.searchsorted(448 * two, h.abs().amax(2).clamp_min(1e-4))          # the least with 448 2^(byte - 127) >= amax
    return _nearest_e4m3(h / two[byte][:, :, None]).flatten(1), two[byte]
