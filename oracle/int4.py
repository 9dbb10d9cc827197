"""RMS norm and 4-bit integer weights, in numpy fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* ``rmsnorm`` -- h = bf16(x + residual), y = bf16(fl32(h / sqrt(mean(h^2) +
  eps) * weight)), the sum exactly rounded (math.fsum).
* ``int4_quantize`` -- codes, scales and zero points of weights per group of
  columns; quotients in fp64, where ties of float operands are exact (a
  quotient of a 24-bit and an 11-bit number that is not k + 1/2 is further
  than 2**-40 from it).
* ``int4_values`` -- the values s (q - z) of such weights.
* ``gemm_int4`` -- the product's sums in fp64, and the magnitudes that its
  error bound goes by.
"""

import math

import numpy as np

from .fp_formats import bf16_bits_to_f64, bf16_from_f64


def rmsnorm(x_bits, weight, eps, residual_bits=None):
    """(h bits, y bits) of BF16 bits [rows, hidden] and float64 weight [hidden]."""
    x = bf16_bits_to_f64(x_bits)
    if residual_bits is not None:
        with np.errstate(invalid="ignore", over="ignore"):
            x = (x.astype(np.float32) + bf16_bits_to_f64(residual_bits).astype(np.float32)).astype(np.float64)
    h_bits = bf16_from_f64(x)
    h = bf16_bits_to_f64(h_bits)
    y = np.empty_like(h)
    with np.errstate(all="ignore"):
        for r in range(h.shape[0]):
            sq = h[r] * h[r]
            total = math.fsum(sq) if np.isfinite(sq).all() else float(sq.sum())
            y[r] = h[r] / np.sqrt(np.float64(total) / h.shape[1] + eps) * weight
        return h_bits, bf16_from_f64(y.astype(np.float32).astype(np.float64))


def scale_round(s, kind):
    """float32 scales to their stored bits (uint16) and float64 values."""
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "fp16":
            h = np.asarray(s, np.float32).astype(np.float16)
            return h.view(np.uint16), h.astype(np.float64)
        bits = bf16_from_f64(np.asarray(s, np.float32).astype(np.float64))
        return bits, bf16_bits_to_f64(bits)


def scale_values(bits, kind):
    if kind == "fp16":
        return np.asarray(bits, np.uint16).view(np.float16).astype(np.float64)
    return bf16_bits_to_f64(bits)


def int4_quantize(w, group, symmetric, kind="bf16"):
    """(codes uint8 [rows, cols/2], scale bits uint16, zeros uint8 or None) of
    float32-valued weights [rows, cols]."""
    w = np.asarray(w, np.float64)
    rows, cols = w.shape
    g = w.reshape(rows, cols // group, group)
    with np.errstate(all="ignore"):
        finite = np.isfinite(g).all(2)
        v = np.where(finite[:, :, None], g, 0.0)
        if symmetric:
            raw = np.abs(v).max(2).astype(np.float32) / np.float32(7)
        else:
            lo, hi = np.minimum(v.min(2), 0), np.maximum(v.max(2), 0)
            raw = (hi - lo).astype(np.float32) / np.float32(15)
        bits, s = scale_round(raw, kind)
        live = finite & np.isfinite(s) & (s > 0)
        by = np.where(live, s, 1.0)
        if symmetric:
            z = np.full(live.shape, 8.0)
        else:
            z = np.where(live, np.clip(np.rint(-lo / by), 0, 15), 0.0)
        n = np.where(live[:, :, None], np.rint(v / by[:, :, None]), 0.0)
        q = np.clip(n + z[:, :, None], 0, 15).reshape(rows, cols).astype(np.uint8)
        nan = np.uint16(0x7E00 if kind == "fp16" else 0x7FC0)
        bits = np.where(finite & np.isfinite(s), bits, nan).astype(np.uint16)
    return q[:, 0::2] | (q[:, 1::2] << 4), bits, None if symmetric else z.astype(np.uint8)


def int4_parts(codes, scales, zeros):
    """(q - z, q, z) float64 [..., cols] of codes, per column."""
    codes = np.asarray(codes, np.uint8)
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.float64)
    each = q.shape[-1] // scales.shape[-1]
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, np.float64)
    z = np.repeat(z, each, -1)
    return q - z, q, z


def int4_values(codes, scales, zeros=None):
    """fp64 values of codes [..., cols/2] with fp64 scales [..., cols/group]."""
    d, _, _ = int4_parts(codes, scales, zeros)
    return d * np.repeat(scales, d.shape[-1] // scales.shape[-1], -1)


def gemm_int4(a, codes, scales, zeros=None):
    """(sums [m, n], magnitudes of the terms within groups [m, n], of the
    groups' sums [m, n]) of fp64 rows a [m, k] with one matrix [n, k]."""
    d, q, z = int4_parts(codes, scales, zeros)
    group = d.shape[1] // scales.shape[1]
    s = np.repeat(scales, group, -1)
    out = a @ (d * s).T
    # A group's sum is formed as sum a (16 + q) - (16 + z) sum a.
    terms = np.abs(a) @ ((32 + q + z) * np.abs(s)).T
    sums = np.zeros_like(out)
    for g in range(scales.shape[1]):
        c = slice(g * group, (g + 1) * group)
        sums += np.abs(a[:, c] @ d[:, c].T) * np.abs(scales[:, g])
    return out, terms, sums
