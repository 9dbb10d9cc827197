"""4-bit activations and the router, in numpy fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* ``mxfp4_quantize`` -- OCP Microscaling v1.0 conversion to MXFP4: per 32
  consecutive values the scale is 2**(floor(log2(amax)) - 2) (2 = the exponent
  of E2M1's largest power of two), its byte at least 0; elements round to the
  nearest E2M1 magnitude of |x| / scale, ties to the even code, saturating at
  6, sign kept. All-zero blocks take byte 0; a block holding an infinity or a
  NaN takes byte 255 and zero codes.
* ``gemm_rows_mx4`` -- rows of the product of two MXFP4 tensors, each value
  e2m1(code) * 2**(byte - 127), summed in fp64, rounded once to BF16.
* ``token_forward_mx4`` -- the layer token by token: quantize, FC1, SiLU * up,
  quantize, FC2, weighted sum, with the roundings of the whole layer (C1 and
  the expert outputs to BF16, SiLU * up to float32).
* ``route`` -- top-k routing, one token at a time in plain Python.
"""

import math

import numpy as np

from .fp_formats import bf16_bits_to_f64, bf16_from_f64, e2m1_decode
from .moe import MX_BLOCK, mxfp4_dequant, swiglu

_MAGNITUDES = e2m1_decode(np.arange(8, dtype=np.uint8))


def mxfp4_quantize(v):
    """Rows of float values [rows, cols] -> (codes uint8 [rows, cols/2], bytes uint8 [rows, cols/32])."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    b = v.reshape(rows, cols // MX_BLOCK, MX_BLOCK)
    amax = np.max(np.abs(b), axis=2)  # NaN if any is
    finite = np.isfinite(amax)
    _, ex = np.frexp(np.where(finite & (amax > 0), amax, 1.0))  # amax = m * 2**ex, m in [0.5, 1)
    byte = np.where(amax > 0, np.maximum(ex - 1 - 2 + 127, 0), 0)
    byte = np.where(finite, byte, 255)
    r = np.abs(np.where(finite[:, :, None], b, 0.0)) * np.exp2(127.0 - np.where(finite, byte, 127))[:, :, None]
    # Nearest by distance to every magnitude; of two equally near, the even code.
    dist = np.abs(r[..., None] - _MAGNITUDES)
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best
    code = np.where(near[..., 0::2].any(-1), 2 * near[..., 0::2].argmax(-1), near.argmax(-1))
    code = np.where(finite[:, :, None], code | (np.signbit(b).astype(np.int64) << 3), 0)
    code = code.reshape(rows, cols).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte.astype(np.uint8)


def gemm_rows_mx4(a_codes, a_scales, w_codes, w_scales):
    """BF16 bits [m, N] and the sums of magnitudes [m, N] (for error bounds)."""
    a, w = mxfp4_dequant(a_codes, a_scales), mxfp4_dequant(w_codes, w_scales)
    return bf16_from_f64(a @ w.T), np.abs(a) @ np.abs(w).T


def token_forward_mx4(x_bits, topk_ids, topk_w, w1, w2, num_experts, t_live, act="swiglu",
                      clamp_limit=np.inf, rounding="divide", expert_start=0):
    """(out fp64 [t_live, H] before its BF16 rounding, sum of |w| |y| [t_live, H])."""
    ids = np.asarray(topk_ids).astype(np.int64) - int(expert_start)
    hidden = np.asarray(x_bits).shape[1]
    out, mag = np.zeros((t_live, hidden)), np.zeros((t_live, hidden))
    for t in range(t_live):
        xq, xs = mxfp4_quantize(bf16_bits_to_f64(np.asarray(x_bits)[t:t + 1]))
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if not 0 <= e < num_experts:
                continue
            c1 = bf16_bits_to_f64(gemm_rows_mx4(xq, xs, w1[0][e], w1[1][e])[0])
            i = c1.shape[1] // 2
            h = swiglu(c1[:, :i], c1[:, i:], act, clamp_limit, rounding)
            hq, hs = mxfp4_quantize(h)
            y = bf16_bits_to_f64(gemm_rows_mx4(hq, hs, w2[0][e], w2[1][e])[0])[0]
            out[t] += float(topk_w[t, k]) * y
            mag[t] += abs(float(topk_w[t, k])) * np.abs(y)
    return out, mag


def route(logits, topk, score="softmax", bias=None, renormalize=True, scale=1.0, num_groups=1,
          top_groups=1, group_top=1):
    """(ids int32 [t, topk], weights float64 [t, topk]) of float logits [t, E]."""
    logits = np.asarray(logits, dtype=np.float64)
    t_n, e_n = logits.shape
    ids = np.full((t_n, topk), -1, np.int32)
    weights = np.zeros((t_n, topk))
    size = e_n // num_groups
    top_float = float(np.finfo(np.float32).max)
    for t in range(t_n):
        row = [-math.inf if math.isnan(v) else min(float(v), top_float) for v in logits[t]]
        top = max(row)
        if score == "softmax":
            ex = [0.0 if v == -math.inf else math.exp(v - top) for v in row]
            total = math.fsum(ex)
            s = [v / total if total > 0 else 0.0 for v in ex]
        else:
            s = [(1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 if v < -709 else math.exp(v)) for v in row]
        sel = [v if bias is None else s[e] + float(bias[e]) for e, v in enumerate(row)]
        ok = [row[e] > -math.inf and sel[e] > -math.inf for e in range(e_n)]  # NaN: not greater
        cand = [e for e in range(e_n) if ok[e]]
        if num_groups > 1:
            val = []
            for g in range(num_groups):
                use = s if bias is None and group_top == 2 else sel
                best = sorted((use[e] for e in cand if e // size == g), reverse=True)[:group_top]
                val.append((sum(best) if best else -math.inf, -g))
            kept = {-g for _, g in sorted(val, reverse=True)[:top_groups]}
            cand = [e for e in cand if e // size in kept]
        cand.sort(key=lambda e: (-sel[e], e))
        cand = cand[:topk]
        total = math.fsum(s[e] for e in cand)
        for k, e in enumerate(cand):
            ids[t, k] = e
            w = s[e] if not renormalize else (s[e] / total if total > 0 else 0.0)
            weights[t, k] = w * scale
    return ids, weights
