"""Measured cases of what stands around the expert layer: the RMS norm with the
residual's addition and quantized output, 4-bit integer weights with group
scales (made and read back), and products of BF16 tokens with them, dense and
per expert.

``own = False`` computes each pass in plain torch operations, ``own = True``
makes the framework's calls. Sizes are the workloads of ``synth/configs.py``
(decode: 288 experts, 4096 -> 512, top-8; padded and full: 32 experts,
7168 -> 2048, top-8; sweep: 256 experts, 6144 -> 256, top-8, Zipf routing).

Norm: h = bf16(x + residual), y = bf16(h / sqrt(mean(h^2) + eps) * weight), y's
FP8 codes per 128 columns (scale max(amax / 448, 1 / 229376), powers of two
rounded up) or MXFP4 (codes per 32 columns under 2**(floor(log2 amax) - 2)).

4-bit integer weights: w = s * (q - z), q in 0..15, two codes per byte with the
even column in the low nibble; a scale s and a zero point z (8 where there are
none) per group of columns of a row.
"""

import math

import torch

own = False

EPS = 1e-6
CLAMP = 7.0
BLOCK = 32


# ---- cases -------------------------------------------------------------------

def _norm(rows, hidden, fmt, residual=True, weight="bfloat16", live=None):
    return {"op": "norm", "rows": rows, "hidden": hidden, "fmt": fmt, "residual": residual,
            "weight": weight, "live": rows if live is None else live}


def _weights(rows, cols, group, symmetric, scale="bfloat16", dtype="bfloat16"):
    return {"op": "weights", "rows": rows, "cols": cols, "group": group, "symmetric": symmetric,
            "scale": scale, "dtype": dtype}


def _linear(tokens, k, n, group, zeros, act, scale="bfloat16"):
    return {"op": "linear", "tokens": tokens, "k": k, "n": n, "group": group, "zeros": zeros,
            "act": act, "scale": scale}


def _experts(tokens, experts, topk, zipf, k, n, group, zeros, act, gather, align=16, scale="bfloat16"):
    return {"op": "experts", "tokens": tokens, "experts": experts, "topk": topk, "zipf": zipf,
            "align": align, "k": k, "n": n, "group": group, "zeros": zeros, "act": act,
            "gather": gather, "scale": scale}


def listed():
    return [
        # The norm in front of a decode step's layer, of a prompt's, and of a
        # batch whose layer takes 4-bit activations.
        {"name": "norm 1x4096", **_norm(1, 4096, "fp32")},
        {"name": "norm 4096x7168", **_norm(4096, 7168, "ue8m0")},
        {"name": "norm 509x6144 mxfp4", **_norm(509, 6144, "mxfp4")},
        # One expert's FC1 weights made and read back, and eight larger experts'
        # with zero points in small groups.
        {"name": "weights 1024x4096", **_weights(1024, 4096, 128, True)},
        {"name": "weights 32768x7168", **_weights(32768, 7168, 32, False, "float16")},
        # A shared expert beside the routed ones: FC1 of one token, FC2 of a
        # batch; and a projection of a short prompt.
        {"name": "linear 1 token 7168-4096", **_linear(1, 7168, 4096, 128, False, "swiglu")},
        {"name": "linear 16 tokens 2048-7168", **_linear(16, 2048, 7168, 32, True, None, "float16")},
        {"name": "linear 300 tokens 6144-1000", **_linear(300, 6144, 1000, 64, True, None)},
        # Routed experts: FC1 of one token, of a ragged batch and of a prompt,
        # FC2 of a longer prompt.
        {"name": "experts 1 token 4096-1024",
         **_experts(1, 288, 8, False, 4096, 1024, 128, False, "swiglu", True)},
        {"name": "experts 64 tokens 6144-512",
         **_experts(64, 256, 8, True, 6144, 512, 32, True, "swiglu_clamp", True)},
        {"name": "experts 1024 tokens 7168-4096",
         **_experts(1024, 32, 8, False, 7168, 4096, 128, False, "swiglu", True)},
        {"name": "experts 2048 tokens 2048-7168",
         **_experts(2048, 32, 8, False, 2048, 7168, 128, False, None, False)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2 * 2048 * 8 * 2048 * 7168
MOST_WEIGHTS = 32 * 4096 * 7168


def draw(rng):
    op = rng.choice(["norm", "weights", "linear", "linear", "experts", "experts"])
    if op == "norm":
        rows = _log(rng, 1, 4096)
        return _norm(rows, 128 * rng.randint(1, 56), rng.choice([None, "fp32", "pow2", "ue8m0", "mxfp4"]),
                     rng.random() < 0.75, rng.choice(["bfloat16", "float32"]),
                     rng.randint(0, rows) if rng.random() < 0.2 else rows)
    group = rng.choice([32, 64, 128])
    scale = rng.choice(["bfloat16", "float16"])
    if op == "weights":
        return _weights(_log(rng, 1, 16384), group * rng.randint(1, 7168 // group), group,
                        rng.random() < 0.5, scale, rng.choice(["bfloat16", "float16", "float32"]))
    act = rng.choice([None, None, "swiglu", "swiglu_clamp", "swiglu_clamp_after_silu"])
    k, n = group * rng.randint(1, 7168 // group), _log(rng, 8, 7168)
    if act is not None:
        n += n % 2
    zeros = rng.random() < 0.5
    if op == "linear":
        return _linear(_log(rng, 1, 2048), k, n, group, zeros, act, scale)
    topk = rng.randint(1, 8)
    experts = max(topk, min(rng.randint(4, 288), MOST_WEIGHTS // (k * n)))
    zipf = rng.random() < 0.3
    tokens = min(_log(rng, 1, 256 if zipf else 4096), max(1, MOST_FLOPS // (2 * topk * k * n)))
    return _experts(tokens, experts, topk, zipf, k, n, group, zeros, act, rng.random() < 0.5,
                    rng.choice([1, 16]), scale)


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _int4(g, lead, n, k, case):
    """Random codes, scales around 0.01 and zero points around 8."""
    groups = k // case["group"]
    codes = torch.randint(0, 256, lead + (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(lead + (n, groups), generator=g, device="cuda") * 0.012 + 0.004
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(5, 12, lead + (n, groups), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales.to(getattr(torch, case["scale"])), zeros


def _routing(g, case):
    logits = _normal(g, case["tokens"], case["experts"])
    if case["zipf"]:
        rank = torch.randperm(case["experts"], generator=g, device="cuda") + 1
        logits = logits - 1.1 * torch.log(rank.float())
    return torch.topk(logits, case["topk"], dim=1)[1]


def _segments(ids, experts, align):
    """The rows of each expert, in pair order, segments rounded up to ``align``."""
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=experts)
    ends = torch.cumsum((counts + align - 1) // align * align, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    order = torch.argsort(flat, stable=True)  # pairs by expert, then by pair
    first = torch.cumsum(counts, 0) - counts
    rows = offsets[flat[order]] + torch.arange(flat.numel(), device="cuda") - first[flat[order]]
    used = min(experts, flat.numel())
    cap = (flat.numel() + used * (align - 1)) // align * align
    row_to_pair = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    row_to_pair[rows] = order.int()
    return {"counts": counts.int(), "offsets": offsets.int(), "row_to_pair": row_to_pair,
            "row_cap": cap, "busiest": int(counts.max())}


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        rows, hidden, fmt = case["rows"], case["hidden"], case["fmt"]
        # A few channels of a residual stream are much larger than the others.
        spread = torch.exp(0.5 * _normal(g, hidden))
        s["x"] = (_normal(g, rows, hidden) * spread).bfloat16()
        s["r"] = (3.0 * _normal(g, rows, hidden) * spread).bfloat16() if case["residual"] else None
        s["gamma"] = (1.0 + 0.2 * _normal(g, hidden)).to(getattr(torch, case["weight"]))
        s["t_live"] = torch.tensor([case["live"]], dtype=torch.int32, device="cuda")
        s["y"] = torch.zeros((rows, hidden), dtype=torch.bfloat16, device="cuda")
        s["h"] = torch.zeros_like(s["y"]) if case["residual"] else None
        s["xq"] = s["xs"] = s["values"] = None
        if fmt == "mxfp4":
            s["xq"] = torch.zeros((rows, hidden // 2), dtype=torch.uint8, device="cuda")
            s["xs"] = torch.zeros((rows, hidden // BLOCK), dtype=torch.uint8, device="cuda")
            s["values"] = torch.zeros_like(s["y"])
        elif fmt is not None:
            s["xq"] = torch.zeros((rows, hidden), dtype=torch.uint8, device="cuda")
            s["xs"] = torch.zeros((hidden // 128, rows), device="cuda",
                                  dtype=torch.uint8 if fmt == "ue8m0" else torch.float32)
        return s
    if case["op"] == "weights":
        rows, cols, groups = case["rows"], case["cols"], case["cols"] // case["group"]
        w = _normal(g, rows, cols)
        # Rows and groups of different sizes and, for zero points, off centre.
        size = 0.02 * torch.exp(0.5 * _normal(g, rows, groups))
        w = w.reshape(rows, groups, -1) * size[:, :, None]
        if not case["symmetric"]:
            w = w + (size * _normal(g, rows, groups))[:, :, None]
        s["w"] = w.reshape(rows, cols).to(getattr(torch, case["dtype"]))
        s["codes"] = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((rows, groups), dtype=getattr(torch, case["scale"]), device="cuda")
        s["zeros"] = None
        if not case["symmetric"]:
            s["zeros"] = torch.empty((rows, groups), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        return s
    k, n = case["k"], case["n"]
    out_n = n if case["act"] is None else n // 2
    if case["op"] == "linear":
        s["a"] = _normal(g, case["tokens"], k).bfloat16()
        s["w"], s["ws"], s["wz"] = _int4(g, (), n, k, case)
        s["out"] = torch.empty((case["tokens"], out_n), dtype=torch.bfloat16, device="cuda")
        return s
    ids = _routing(g, case)
    s.update(_segments(ids, case["experts"], case["align"]))
    s["a"] = _normal(g, case["tokens"] if case["gather"] else s["row_cap"], k).bfloat16()
    s["w"], s["ws"], s["wz"] = _int4(g, (case["experts"],), n, k, case)
    s["out"] = torch.zeros((s["row_cap"], out_n), dtype=torch.bfloat16, device="cuda")
    return s


# ---- plain forms ---------------------------------------------------------------

def _fp8(y, fmt):
    """(codes, scales [cols / 128, rows]) of BF16 y."""
    v = y.double().reshape(y.shape[0], -1, 128)
    s = (v.abs().amax(2) / 448.0).float().clamp(min=1.0 / 229376.0)
    if fmt != "fp32":
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    q = (v / s.double()[:, :, None]).float().reshape(y.shape).to(torch.float8_e4m3fn)
    s = s.t().contiguous()
    return q, (torch.log2(s) + 127.0).to(torch.uint8) if fmt == "ue8m0" else s


def _mx_values(y):
    """BF16 values that the MXFP4 quantization of y stands for."""
    b = y.double().reshape(y.shape[0], -1, BLOCK)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(min=-127)
    a = torch.ldexp(b, -e[:, :, None]).abs()
    m = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + 2.0 * (a > 5.0))
    return (torch.copysign(m, b) * torch.ldexp(torch.ones_like(amax), e)[:, :, None]).reshape(
        y.shape).bfloat16()


def _plain_norm(s):
    live = s["live"]
    x = s["x"][:live]
    h = x if s["r"] is None else (x.float() + s["r"][:live].float()).bfloat16()
    d = h.double()
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = (d * rstd * s["gamma"].double()).float().bfloat16()
    out = {"y": torch.zeros_like(s["y"])}
    out["y"][:live] = y
    if s["r"] is not None:
        out["h"] = torch.zeros_like(s["h"])
        out["h"][:live] = h
    if s["fmt"] == "mxfp4":
        out["values"] = torch.zeros_like(s["values"])
        out["values"][:live] = _mx_values(y)
    elif s["fmt"] is not None:
        q, scales = _fp8(y, s["fmt"])
        out["xq"] = torch.zeros_like(s["xq"])
        out["xq"][:live] = q.view(torch.uint8)
        out["xq"] = out["xq"].view(torch.float8_e4m3fn)
        out["xs"] = torch.zeros_like(s["xs"])
        out["xs"][:, :live] = scales
    return out


def _plain_weights(s):
    """Codes, scales and zero points, and the values that they stand for."""
    scale_type = getattr(torch, s["scale"])
    w = s["w"].double().reshape(s["rows"], -1, s["group"])
    if s["symmetric"]:
        scale = (w.abs().amax(2) / 7.0).float().to(scale_type)
        zero = torch.full_like(scale, 8.0, dtype=torch.float64)
    else:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        scale = ((hi - lo).float().double() / 15.0).float().to(scale_type)
        by = torch.where(scale > 0, scale.double(), 1.0)
        zero = torch.where(scale > 0, torch.round(-lo / by), 0.0).clamp(0, 15)
    by = torch.where(scale > 0, scale.double(), 1.0)[:, :, None]
    q = torch.where(scale[:, :, None] > 0, torch.round(w / by), 0.0) + zero[:, :, None]
    q = q.clamp(0, 15).reshape(s["rows"], -1).to(torch.uint8)
    codes = q[:, 0::2] + 16 * q[:, 1::2]
    values = _int4_values(codes, scale, zero.to(torch.uint8))
    return values.bfloat16(), scale, None if s["symmetric"] else zero.to(torch.uint8)


def _int4_values(codes, scales, zeros):
    """float32 values of codes [..., k / 2]."""
    q = torch.stack([codes & 15, codes >> 4], -1).float()
    q = q.reshape(scales.shape + (-1,))
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((q - z) * scales.float()[..., None]).reshape(codes.shape[:-1] + (-1,))


def _gated(c, act):
    """SiLU(gate) * up of float32 columns, or c itself."""
    if act is None:
        return c
    gate, up = c.chunk(2, dim=-1)
    if act == "swiglu_clamp":
        gate = gate.clamp(max=CLAMP)
    silu = gate / (1.0 + torch.exp(-gate))
    if act == "swiglu_clamp_after_silu":
        silu = silu.clamp(max=CLAMP)
    if act != "swiglu":
        up = up.clamp(-CLAMP, CLAMP)
    return silu * up


def _plain_experts(s):
    counts, cap = s["counts"].long(), s["row_cap"]
    src = s["row_to_pair"].long().clamp(min=0) // s["topk"] if s["gather"] else torch.arange(
        cap, device="cuda")
    # The experts with rows are among the most loaded min(E, rows) ones.
    experts = torch.argsort(counts, descending=True)[:min(counts.numel(), cap)]
    j = torch.arange(s["busiest"], device="cuda")
    rows = torch.where(j < counts[experts][:, None], s["offsets"][:-1].long()[experts][:, None] + j, cap)
    tokens = s["a"][torch.cat([src, src.new_zeros(1)])[rows]].float()
    w = _int4_values(s["w"][experts], s["ws"][experts], None if s["wz"] is None else s["wz"][experts])
    c = _gated(torch.matmul(tokens, w.transpose(1, 2)), s["act"])
    out = torch.zeros((cap + 1, c.shape[2]), dtype=torch.bfloat16, device="cuda")
    out[rows] = c.bfloat16()
    return out[:cap]


def run(s):
    op = s["op"]
    if own:
        import block_fp8_mixture_amd as moe
        if op == "norm":
            moe.moe_rmsnorm_quant(s["x"], s["gamma"], EPS, s["fmt"], residual=s["r"], t_live=s["t_live"],
                                  residual_out=s["h"], y=s["y"], xq=s["xq"], xs=s["xs"])
            out = {"y": s["y"]}
            if s["r"] is not None:
                out["h"] = s["h"]
            if s["fmt"] == "mxfp4":
                out["values"] = moe.moe_mxfp4_dequant(s["xq"], s["xs"], out=s["values"])
            elif s["fmt"] is not None:
                out["xq"], out["xs"] = s["xq"].view(torch.float8_e4m3fn), s["xs"]
            return out
        if op == "weights":
            moe.moe_int4_quant(s["w"], s["group"], s["symmetric"], codes=s["codes"], scales=s["scales"],
                               zeros=s["zeros"])
            return moe.moe_int4_dequant(s["codes"], s["scales"], s["zeros"], out=s["out"]), s["scales"], s["zeros"]
        if op == "linear":
            return moe.moe_gemm_int4(s["a"], s["w"], s["ws"], s["wz"], act=s["act"], clamp_limit=CLAMP,
                                     out=s["out"])
        return moe.moe_grouped_gemm_int4(
            s["a"], s["w"], s["ws"], s["counts"], s["offsets"], s["row_cap"], w_zeros=s["wz"],
            a_row_map=s["row_to_pair"] if s["gather"] else None, a_row_div=s["topk"] if s["gather"] else 1,
            max_rows_per_expert=s["tokens"], act=s["act"], clamp_limit=CLAMP, out=s["out"])
    if op == "norm":
        return _plain_norm(s)
    if op == "weights":
        return _plain_weights(s)
    if op == "linear":
        w = _int4_values(s["w"], s["ws"], s["wz"])
        return _gated(torch.matmul(s["a"].float(), w.t()), s["act"]).bfloat16()
    return _plain_experts(s)


# ---- what a pass cannot do without ------------------------------------------------

def _touched(case):
    """Experts that the pairs of a case reach, as expected of even routing."""
    pairs, e = case["tokens"] * case["topk"], case["experts"]
    return min(e, pairs, e * (1.0 - (1.0 - case["topk"] / e) ** case["tokens"]))


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["live"] * case["hidden"]
        size = 2 + 2 + (4 if case["residual"] else 0)
        if case["fmt"] == "mxfp4":  # written, and read back as values
            size += 2 * (0.5 + 1.0 / BLOCK) + 2
        elif case["fmt"] is not None:
            size += 1 + (1 if case["fmt"] == "ue8m0" else 4) / 128
        return {"bytes": size * n + (2 if case["weight"] == "bfloat16" else 4) * case["hidden"],
                "flops": 10 * n}
    per = 0.5 + (2 if case.get("symmetric", not case.get("zeros")) else 3) / case["group"]
    if op == "weights":
        n = case["rows"] * case["cols"]
        return {"bytes": ((4 if case["dtype"] == "float32" else 2) + 2 * per + 2) * n, "flops": 6 * n}
    k, n = case["k"], case["n"]
    out_n = n if case["act"] is None else n // 2
    if op == "linear":
        t = case["tokens"]
        return {"bytes": per * n * k + 2 * t * (k + out_n), "flops": 2 * t * n * k}
    pairs = case["tokens"] * case["topk"]
    a_rows = case["tokens"] if case["gather"] else pairs
    return {"bytes": per * _touched(case) * n * k + 2 * (a_rows * k + pairs * out_n),
            "flops": 2 * pairs * n * k}


# ---- 64 bits ------------------------------------------------------------------------

def _grid(v, bits, least, most):
    """v to the nearest value of ``bits`` fraction bits, exponents from ``least``."""
    a = v.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=least)
    step = 2.0 ** (e - bits)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=most)


def _exact_norm(s):
    n, t = s["live"], s["rows"]
    x = s["x"].double()
    h = x if s["r"] is None else x + s["r"].double()
    b = h if s["r"] is None else h.float().bfloat16().double()  # the stored sum, which is normed
    y = b * torch.rsqrt(b.square().sum(1, keepdim=True) / s["hidden"] + EPS) * s["gamma"].double()
    gone = torch.arange(t, device="cuda")[:, None] >= n
    out = {"y": y.masked_fill(gone, 0.0)}
    if s["r"] is not None:
        out["h"] = h.masked_fill(gone, 0.0)
    q = y.float().bfloat16().double()
    if s["fmt"] == "mxfp4":
        q = q.unflatten(1, (-1, BLOCK))
        top = q.abs().max(2, keepdim=True)[0]
        power = torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2
        out["values"] = (_grid(q / 2.0 ** power, 1, 0, 6.0) * 2.0 ** power).flatten(1).masked_fill(gone, 0.0)
    elif s["fmt"] is not None:
        q = q.unflatten(1, (-1, 128))
        scale = torch.maximum(q.abs().max(2)[0] / 448.0, torch.full((), 1.0 / 229376.0, device="cuda"))
        if s["fmt"] != "fp32":
            scale = 2.0 ** torch.ceil(torch.log2(scale.float().double()))
        else:
            scale = scale.float().double()
        # The codes go by the quotient in 32 bits: it decides what is a tie.
        q = (q / scale[:, :, None]).float().double()
        out["xq"] = _grid(q, 3, -6, 448.0).flatten(1).masked_fill(gone, 0.0)
        out["xs"] = None if s["fmt"] == "ue8m0" else scale.masked_fill(gone, 0.0).t()
    return out


def _exact_weights(s):
    kind = getattr(torch, s["scale"])
    values, scales = [], []
    for part in s["w"].split(4096):
        w = part.double().unflatten(1, (-1, s["group"]))
        if s["symmetric"]:
            real = w.abs().max(2, keepdim=True)[0] / 7
        else:
            real = (w.max(2, keepdim=True)[0].clamp(min=0) - w.min(2, keepdim=True)[0].clamp(max=0)) / 15
        scale = real.float().to(kind).double()  # the stored scale, by which the codes go
        z = 8.0
        if not s["symmetric"]:
            z = (w.min(2, keepdim=True)[0].clamp(max=0) / -scale).nan_to_num(0.0).round().clamp(0, 15)
        q = ((w / scale).nan_to_num(0.0).round() + z).clamp(0, 15)
        values.append(((q - z) * scale).flatten(1))
        scales.append(real.squeeze(2))
    return torch.cat(values), torch.cat(scales), None


def _exact_weight(codes, scales, zeros):
    q = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device="cuda")
    q[..., 0::2] = (codes % 16).double()
    q[..., 1::2] = (codes // 16).double()
    each = q.shape[-1] // scales.shape[-1]
    z = torch.full(scales.shape, 8, device="cuda") if zeros is None else zeros
    return scales.double().repeat_interleave(each, -1) * (q - z.double().repeat_interleave(each, -1))


def _exact_gated(c, act):
    if act is None:
        return c
    i = c.shape[1] // 2
    g, u = c[:, :i], c[:, i:]
    top = torch.full((), CLAMP, dtype=torch.float64, device="cuda")
    if act == "swiglu_clamp":
        g = torch.minimum(g, top)
    g = g * torch.sigmoid(g)
    if act == "swiglu_clamp_after_silu":
        g = torch.minimum(g, top)
    return g * (u if act == "swiglu" else torch.maximum(torch.minimum(u, top), -top))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "weights":
        return _exact_weights(s)
    if case["op"] == "linear":
        w = _exact_weight(s["w"], s["ws"], s["wz"])
        return _exact_gated(torch.mm(s["a"].double(), w.t()), case["act"])
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        first, rows = int(s["offsets"][e]), int(s["counts"][e])
        if rows:
            at = torch.arange(first, first + rows, device="cuda")
            if case["gather"]:
                at = s["row_to_pair"][first:first + rows].long() // case["topk"]
            w = _exact_weight(s["w"][e], s["ws"][e], None if s["wz"] is None else s["wz"][e])
            out[first:first + rows] = _exact_gated(torch.mm(s["a"][at].double(), w.t()), case["act"])
    return out
