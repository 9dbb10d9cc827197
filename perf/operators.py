"""Measured cases of the expert layer with 4-bit activations: routing from
router logits, MXFP4 quantization, the SiLU-gated MXFP4 quantization, the
grouped MXFP4 x MXFP4 product, and the whole layer.

``own = False`` computes each pass in plain torch operations, ``own = True``
makes the framework's calls. Sizes are the workloads of ``synth/configs.py``
(decode: 288 experts, 4096 -> 512, top-8; padded and full: 32 experts,
7168 -> 2048, top-8; sweep: 256 experts, 6144 -> 256, top-8, Zipf routing).

MXFP4 tensors: E2M1 codes two per byte, the even column in the low nibble
(magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 the sign), and one E8M0 byte b
(2**(b - 127), 255 = NaN) per 32 consecutive columns of a row. Quantization of
a block takes b = floor(log2(amax)) - 2 + 127, at least 0, and rounds x / 2**(b
- 127) to the nearest magnitude, ties to the even code, saturating at 6.
"""

import math

import torch

own = False

FLT_MAX = 3.4028234663852886e38
BLOCK = 32


# ---- cases -------------------------------------------------------------------

def _route(tokens, experts, topk, score, dtype, bias=False, groups=1, top_groups=1, group_top=1,
           masked=False, renormalize=True, scale=1.0):
    return {"op": "route", "tokens": tokens, "experts": experts, "topk": topk, "score": score,
            "dtype": dtype, "bias": bias, "groups": groups, "top_groups": top_groups,
            "group_top": group_top, "masked": masked, "renormalize": renormalize, "scale": scale}


def _rows(op, tokens, experts, topk, zipf, align):
    return {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "zipf": zipf,
            "align": align}


def listed():
    return [
        # One decode step's routing, and a prompt's with expert groups and a
        # selection bias.
        {"name": "route 1 of 288", **_route(1, 288, 8, "softmax", "float32")},
        {"name": "route 4096 of 256 groups",
         **_route(4096, 256, 8, "sigmoid", "float32", bias=True, groups=8, top_groups=4, group_top=2,
                  scale=2.5)},
        # The FC1 input of a decode step and of a prompt: quantized, and read back.
        {"name": "quant 4x4096", "op": "quant", "rows": 4, "cols": 4096},
        {"name": "quant 4096x7168", "op": "quant", "rows": 4096, "cols": 7168},
        # The FC2 input of a small ragged batch and of a prompt.
        {"name": "silu 512x256", **_rows("silu", 64, 256, 8, True, 16), "inter": 256,
         "act": "swiglu_clamp"},
        {"name": "silu 32768x2048", **_rows("silu", 4096, 32, 8, False, 1), "inter": 2048,
         "act": "swiglu"},
        # FC1 of a small ragged batch, FC2 of a batch of 512 tokens, FC1 of a prompt.
        {"name": "gemm 512 rows 6144-512", **_rows("gemm", 64, 256, 8, True, 16), "k": 6144, "n": 512,
         "gather": True},
        {"name": "gemm 4096 rows 2048-7168", **_rows("gemm", 512, 32, 8, False, 1), "k": 2048,
         "n": 7168, "gather": False},
        {"name": "gemm 32768 rows 7168-4096", **_rows("gemm", 4096, 32, 8, False, 1), "k": 7168,
         "n": 4096, "gather": True},
        # The whole layer: one and four tokens of a decode step, and a prompt.
        {"name": "layer 1 token", **_rows("layer", 1, 288, 8, False, 16), "hidden": 4096, "inter": 512,
         "act": "swiglu"},
        {"name": "layer 4 tokens", **_rows("layer", 4, 288, 8, False, 16), "hidden": 4096,
         "inter": 512, "act": "swiglu_clamp"},
        {"name": "layer 4096 tokens", **_rows("layer", 4096, 32, 8, False, 16), "hidden": 7168,
         "inter": 2048, "act": "swiglu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quant", "silu", "gemm", "layer", "layer"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.randint(2, 512 // groups)
        top_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(8, top_groups * (experts // groups)))
        return _route(_log(rng, 1, 4096), experts, topk, rng.choice(["softmax", "sigmoid"]),
                      rng.choice(["float32", "bfloat16", "float16"]), bias=rng.random() < 0.5,
                      groups=groups, top_groups=top_groups, group_top=rng.choice([1, 2]),
                      masked=rng.random() < 0.3, renormalize=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]))
    if op == "quant":
        return {"op": "quant", "rows": _log(rng, 1, 4096), "cols": 128 * rng.randint(1, 56)}
    topk = rng.randint(1, 8)
    experts = rng.randint(max(4, topk), 288)
    tokens = _log(rng, 1, 4096)
    case = _rows(op, tokens, experts, topk, rng.random() < 0.3, rng.choice([1, 16]))
    if op == "silu":
        return {**case, "inter": 128 * rng.randint(1, 16),
                "act": rng.choice(["swiglu", "swiglu_clamp", "swiglu_clamp_after_silu"])}
    # Expert weights at most those of the 32-expert layer.
    inter = 128 * rng.randint(1, 16)
    hidden = 128 * rng.randint(2, 56)
    case["experts"] = max(topk, min(experts, 32 * 2048 * 7168 // (inter * hidden)))
    if op == "gemm":
        if rng.random() < 0.5:
            return {**case, "k": hidden, "n": 2 * inter, "gather": True}
        return {**case, "k": inter, "n": hidden, "gather": False}
    return {**case, "hidden": hidden, "inter": inter,
            "act": rng.choice(["swiglu", "swiglu_clamp", "swiglu_clamp_after_silu"])}


CLAMP = 7.0


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _mx_weights(g, experts, rows, cols):
    """Random E2M1 codes and scales of an RMS near 0.02."""
    codes = torch.randint(0, 256, (experts, rows, cols // 2), generator=g, device="cuda",
                          dtype=torch.uint8)
    scales = torch.randint(117, 122, (experts, rows, cols // BLOCK), generator=g, device="cuda",
                           dtype=torch.uint8)
    return codes, scales


def _routing(g, case):
    logits = _normal(g, case["tokens"], case["experts"])
    if case["zipf"]:
        rank = torch.randperm(case["experts"], generator=g, device="cuda") + 1
        logits = logits - 1.1 * torch.log(rank.float())
    top, ids = torch.topk(torch.softmax(logits, 1), case["topk"], dim=1)
    return ids.int(), (top / top.sum(1, keepdim=True)).float()


def _segments(ids, experts, align):
    """The rows of each expert, in pair order, segments rounded up to ``align``."""
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=experts)
    ends = torch.cumsum((counts + align - 1) // align * align, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    order = torch.argsort(flat, stable=True)  # pairs by expert, then by pair
    first = torch.cumsum(counts, 0) - counts
    rank = torch.arange(flat.numel(), device="cuda") - first[flat[order]]
    rows = offsets[flat[order]] + rank
    used = min(experts, flat.numel())
    cap = (flat.numel() + used * (align - 1)) // align * align
    row_to_pair = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    row_to_pair[rows] = order.int()
    return {"counts": counts.int(), "offsets": offsets.int(), "row_to_pair": row_to_pair,
            "row_cap": cap, "busiest": int(counts.max())}


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "route":
        dtype = getattr(torch, case["dtype"])
        logits = 1.5 * _normal(g, case["tokens"], case["experts"])
        if case["masked"]:  # experts that are switched off, for some tokens all of them
            off = torch.rand(logits.shape, generator=g, device="cuda") < 0.2
            off |= torch.rand((case["tokens"], 1), generator=g, device="cuda") < 0.02
            logits = logits.masked_fill(off, float("-inf"))
        s["logits"] = logits.to(dtype)
        s["bias"] = 0.1 * _normal(g, case["experts"]) if case["bias"] else None
        s["ids"] = torch.empty((case["tokens"], case["topk"]), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((case["tokens"], case["topk"]), dtype=torch.float32, device="cuda")
        return s
    if case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _normal(g, rows, cols).bfloat16()
        s["codes"] = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((rows, cols // BLOCK), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        return s
    ids, w = _routing(g, case)
    if case["op"] == "layer":
        h, i, e = case["hidden"], case["inter"], case["experts"]
        s["ids"], s["w"] = ids, w
        s["x"] = _normal(g, case["tokens"], h).bfloat16()
        s["w1"], s["w1s"] = _mx_weights(g, e, 2 * i, h)
        s["w2"], s["w2s"] = _mx_weights(g, e, h, i)
        s["busiest"] = int(torch.bincount(ids.reshape(-1).long()).max())
        s["out"] = torch.empty((case["tokens"], h), dtype=torch.bfloat16, device="cuda")
        s["workspace"] = None
        return s
    s.update(_segments(ids, case["experts"], case["align"]))
    if case["op"] == "silu":
        r, i = s["row_cap"], case["inter"]
        s["gate_up"] = (2.0 * _normal(g, r, 2 * i)).bfloat16()
        s["codes"] = torch.zeros((r, i // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((r, i // BLOCK), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty((r, i), dtype=torch.bfloat16, device="cuda")
        return s
    a_rows = case["tokens"] if case["gather"] else s["row_cap"]
    s["a"], s["a_scales"] = _mx_quantize(_normal(g, a_rows, case["k"]).bfloat16())
    s["w"], s["w_scales"] = _mx_weights(g, case["experts"], case["n"], case["k"])
    s["out"] = torch.zeros((s["row_cap"], case["n"]), dtype=torch.bfloat16, device="cuda")
    return s


# ---- plain forms ---------------------------------------------------------------

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_quantize(x):
    """(codes [rows, cols / 2], scale bytes [rows, cols / 32]) of x."""
    blocks = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = blocks.abs().amax(2)
    byte = torch.where(amax > 0, torch.frexp(amax)[1] - 3 + 127, 0).clamp(0, 254)
    byte = torch.where(torch.isfinite(amax), byte, 255)
    a = torch.ldexp(blocks.double(), (127 - byte)[:, :, None]).abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    code = code + 8 * torch.signbit(blocks)
    code = torch.where(torch.isfinite(amax)[:, :, None], code, 0).reshape(x.shape).to(torch.uint8)
    return code[:, 0::2] + 16 * code[:, 1::2], byte.to(torch.uint8)


def _mx_values(codes, scales):
    """float32 values of codes [..., cols / 2] with scale bytes [..., cols / 32]."""
    table = torch.tensor(_MAGNITUDES + tuple(-m for m in _MAGNITUDES), device=codes.device)
    # Both values of a byte, by the byte.
    bytes_ = torch.arange(256, device=codes.device)
    pairs = torch.stack([table[bytes_ & 15], table[bytes_ >> 4]], 1)
    v = pairs[codes.int()]  # [..., cols / 2, 2]
    scale = torch.exp2(scales.float() - 127.0)
    scale = torch.where(scales == 255, float("nan"), scale)
    v = v.reshape(scales.shape + (BLOCK,)) * scale[..., None]
    return v.reshape(codes.shape[:-1] + (2 * codes.shape[-1],))


def _swiglu(gate_up, act):
    """float32 SiLU(gate) * up of BF16 values, in 64 bits and rounded once."""
    gate, up = gate_up.double().chunk(2, dim=-1)
    if act == "swiglu_clamp":
        gate = gate.clamp(max=CLAMP)
    silu = gate / (1.0 + torch.exp(-gate))
    if act == "swiglu_clamp_after_silu":
        silu = silu.clamp(max=CLAMP)
    if act != "swiglu":
        up = up.clamp(-CLAMP, CLAMP)
    return (silu * up).float()


def _grouped(a, a_scales, w, w_scales, counts, offsets, src, row_cap, busiest):
    """BF16 rows of the grouped product, zeros where no expert has a row."""
    # The experts with rows are among the most loaded min(E, rows) ones.
    experts = torch.argsort(counts, descending=True)[:min(counts.numel(), row_cap)].long()
    j = torch.arange(busiest, device=counts.device)
    live = j < counts[experts][:, None]
    rows = torch.where(live, offsets[:-1].long()[experts][:, None] + j, row_cap)
    from_a = torch.cat([src, src.new_zeros(1)])[rows]
    tokens = _mx_values(a, a_scales)[from_a]
    c = torch.matmul(tokens, _mx_values(w[experts], w_scales[experts]).transpose(1, 2))
    out = torch.zeros((row_cap + 1, w.shape[1]), dtype=torch.bfloat16, device=a.device)
    out[rows] = c.bfloat16()
    return out[:row_cap]


def _plain_route(s):
    x = torch.where(torch.isnan(s["logits"]), float("-inf"), s["logits"].double()).clamp(max=FLT_MAX)
    top = x.amax(1, keepdim=True)
    top = torch.where(top > float("-inf"), top, 0.0)
    if s["score"] == "softmax":
        p = torch.exp(x - top)
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    pick = x if s["bias"] is None else torch.where(x > float("-inf"), p + s["bias"].double(),
                                                   float("-inf"))
    t, e = x.shape
    if s["groups"] > 1:
        v = pick if s["bias"] is not None or s["group_top"] == 1 else torch.where(
            x > float("-inf"), p, float("-inf"))
        best = torch.sort(v.reshape(t, s["groups"], -1), dim=2, descending=True)[0]
        best = best[:, :, :s["group_top"]]
        value = torch.where(best > float("-inf"), best, 0.0).sum(2)
        value = torch.where(best[:, :, 0] > float("-inf"), value, float("-inf"))
        order = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        kept = kept[:, :, None].expand(-1, -1, e // s["groups"]).reshape(t, e)
        pick = torch.where(kept, pick, float("-inf"))
    value, ids = torch.sort(pick, dim=1, descending=True, stable=True)
    value, ids = value[:, :s["topk"]], ids[:, :s["topk"]]
    ok = value > float("-inf")
    w = torch.where(ok, p.gather(1, ids), 0.0)
    if s["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(ok, ids, -1).int(), (w * s["scale"]).float()


def _plain_silu(s):
    h = _swiglu(s["gate_up"], s["act"])
    codes, scales = _mx_quantize(h)
    row = torch.arange(s["row_cap"], device="cuda")
    live = s["row_to_pair"] >= 0
    values = torch.where(live[row][:, None], _mx_values(codes, scales), 0.0)
    return values.bfloat16()


def _plain_layer(s):
    t, k = s["ids"].shape
    # Rows in pair order per expert: a row per pair, sorted by expert.
    flat = s["ids"].reshape(-1).long()
    counts = torch.zeros(s["experts"], dtype=torch.long, device="cuda").scatter_add_(
        0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    pair = torch.argsort(flat, stable=True)
    codes, scales = _mx_quantize(s["x"])
    c1 = _grouped(codes, scales, s["w1"], s["w1s"], counts, offsets, pair // k, t * k, s["busiest"])
    codes, scales = _mx_quantize(_swiglu(c1, s["act"]))
    y = _grouped(codes, scales, s["w2"], s["w2s"], counts, offsets,
                 torch.arange(t * k, device="cuda"), t * k, s["busiest"])
    by_pair = torch.empty_like(y)
    by_pair[pair] = y
    return (by_pair.float().reshape(t, k, -1) * s["w"][:, :, None]).sum(1).bfloat16()


def run(s):
    op = s["op"]
    if own:
        import block_fp8_mixture_amd as moe
        if op == "route":
            return moe.moe_route(s["logits"], s["topk"], score=s["score"], bias=s["bias"],
                                 renormalize=s["renormalize"], scale=s["scale"],
                                 num_groups=s["groups"], top_groups=s["top_groups"],
                                 group_top=s["group_top"], ids=s["ids"], weights=s["w"])
        if op == "quant":
            moe.moe_act_quant(s["x"], "mxfp4", xq=s["codes"], xs=s["scales"])
            return moe.moe_mxfp4_dequant(s["codes"], s["scales"], out=s["out"])
        if op == "silu":
            moe.moe_silu_mul_quant(s["gate_up"], s["counts"], s["offsets"], s["act"], CLAMP, "mxfp4",
                                   hq=s["codes"], hs=s["scales"])
            return moe.moe_mxfp4_dequant(s["codes"], s["scales"], out=s["out"])
        if op == "gemm":
            return moe.moe_grouped_gemm_mxfp4(
                s["a"], s["a_scales"], "mxfp4", s["w"], s["w_scales"], s["counts"], s["offsets"],
                s["row_cap"], a_row_map=s["row_to_pair"] if s["gather"] else None,
                a_row_div=s["topk"] if s["gather"] else 1, max_rows_per_expert=s["tokens"],
                out=s["out"])
        out, s["workspace"] = moe.moe_forward(
            s["x"], s["ids"], s["w"], s["w1"], s["w1s"], s["w2"], s["w2s"], "mxfp4", s["act"], CLAMP,
            s["align"], out=s["out"], workspace=s["workspace"], weight_fmt="mxfp4")
        return out
    if op == "route":
        return _plain_route(s)
    if op == "quant":
        return _mx_values(*_mx_quantize(s["x"])).bfloat16()
    if op == "silu":
        return _plain_silu(s)
    if op == "gemm":
        rows = s["row_to_pair"].long().clamp(min=0) // s["topk"] if s["gather"] else torch.arange(
            s["row_cap"], device="cuda")
        return _grouped(s["a"], s["a_scales"], s["w"], s["w_scales"], s["counts"], s["offsets"],
                        rows, s["row_cap"], s["busiest"])
    return _plain_layer(s)


# ---- what a pass cannot do without ------------------------------------------------

def _touched(case):
    """Experts that the pairs of a case reach, as expected of even routing."""
    pairs, e = case["tokens"] * case["topk"], case["experts"]
    return min(e, pairs, e * (1.0 - (1.0 - case["topk"] / e) ** case["tokens"]))


def work(case):
    op = case["op"]
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        t, e = case["tokens"], case["experts"]
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * case["topk"],
                "flops": 4 * t * e}
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n, "flops": 3 * n}
    pairs = case["tokens"] * case["topk"]
    if op == "silu":
        n = pairs * case["inter"]
        return {"bytes": 4 * n + 2 * n, "flops": 6 * n}
    mx = 0.5 + 1.0 / BLOCK
    if op == "gemm":
        k, n = case["k"], case["n"]
        a_rows = case["tokens"] if case["gather"] else pairs
        return {"bytes": mx * (_touched(case) * n * k + a_rows * k) + 2 * pairs * n,
                "flops": 2 * pairs * n * k}
    h, i = case["hidden"], case["inter"]
    return {"bytes": mx * _touched(case) * 3 * h * i + 4 * case["tokens"] * h + 8 * pairs,
            "flops": 2 * pairs * 3 * h * i}


# ---- 64 bits ------------------------------------------------------------------------

def _exact_round(a):
    """Magnitudes to the E2M1 grid: steps of 0.5 below 2, of 1 below 4, of 2 above."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return (torch.round(a / step) * step).clamp(max=6.0)


def _exact_mx(x):
    """The 64-bit values that the quantization of x stands for."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    amax = b.abs().max(-1, keepdim=True)[0]
    power = torch.floor(torch.log2(amax.clamp(min=2.0 ** -125))) - 2
    q = torch.sign(b) * _exact_round(b.abs() / 2.0 ** power) * 2.0 ** power
    return q.flatten(-2)


def _exact_values(codes, scales):
    nibbles = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    exp, man = (nibbles >> 1) & 3, nibbles & 1
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (exp - 1)).double()
    v = torch.where(nibbles >= 8, -mag, mag).unflatten(-1, (-1, BLOCK))
    return (v * 2.0 ** (scales.double() - 127)[..., None]).flatten(-2)


def _exact_swiglu(gu, act):
    i = gu.shape[1] // 2
    g, u = gu[:, :i].double(), gu[:, i:].double()
    if act == "swiglu_clamp":
        g = torch.minimum(g, torch.tensor(CLAMP, dtype=torch.float64, device=g.device))
    s = g * torch.sigmoid(g)
    if act == "swiglu_clamp_after_silu":
        s = torch.minimum(s, torch.tensor(CLAMP, dtype=torch.float64, device=g.device))
    if act != "swiglu":
        u = torch.maximum(torch.minimum(u, torch.full_like(u, CLAMP)), torch.full_like(u, -CLAMP))
    return (s * u).float()


def _exact_route(s):
    # A token at a time would take minutes: the same steps, in another order.
    x = s["logits"].double().cpu()
    e, k = x.shape[1], s["topk"]
    dead = ~(x > float("-inf"))
    score = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
    score = torch.where(dead, 0.0, score)
    key = score if s["bias"] is None else score + s["bias"].double().cpu()
    if s["groups"] > 1:
        size = e // s["groups"]
        v = torch.where(dead, float("-inf"), key).reshape(-1, s["groups"], size)
        best = torch.topk(v, min(s["group_top"], size), dim=2)[0]
        value = torch.where(torch.isinf(best), 0.0, best).sum(2)
        value = torch.where(torch.isinf(best[:, :, 0]), float("-inf"), value)
        worst = torch.argsort(value, dim=1, descending=True, stable=True)[:, s["top_groups"]:]
        lost = torch.zeros_like(value).scatter_(1, worst, 1.0).bool()
        dead = dead | lost.repeat_interleave(size, 1)
    key = torch.where(dead, float("-inf"), key)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    gone = torch.gather(dead, 1, ids)
    w = torch.where(gone, 0.0, torch.gather(score, 1, ids))
    if s["renormalize"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return None, w * s["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quant":
        return _exact_mx(s["x"])
    if op == "silu":
        out = torch.zeros((s["row_cap"], case["inter"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            a, n = int(s["offsets"][e]), int(s["counts"][e])
            if n:
                out[a:a + n] = _exact_mx(_exact_swiglu(s["gate_up"][a:a + n], case["act"]))
        return out
    if op == "gemm":
        out = torch.zeros((s["row_cap"], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            a, n = int(s["offsets"][e]), int(s["counts"][e])
            if n:
                rows = torch.arange(a, a + n, device="cuda")
                if case["gather"]:
                    rows = s["row_to_pair"][a:a + n].long() // case["topk"]
                out[a:a + n] = _exact_values(s["a"][rows], s["a_scales"][rows]) @ _exact_values(
                    s["w"][e], s["w_scales"][e]).T
        return out
    x = _exact_mx(s["x"])
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        t, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel():
            c1 = (x[t] @ _exact_values(s["w1"][e], s["w1s"][e]).T).bfloat16()
            y = _exact_mx(_exact_swiglu(c1, case["act"])) @ _exact_values(s["w2"][e], s["w2s"][e]).T
            out[t] += s["w"][t, slot].double()[:, None] * y.bfloat16().double()
    return out
