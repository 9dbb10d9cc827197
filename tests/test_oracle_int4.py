"""Pins of the oracle's norm and 4-bit integer weights to something other than
itself: exact rational arithmetic and closed forms."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from tests.exact import round_binary


def _f(v):
    return Fraction(float(v))


@pytest.mark.parametrize("kind,frac,emin", [("bf16", 7, -126), ("fp16", 10, -14)])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_quantize_by_rationals(group, symmetric, kind, frac, emin):
    g = np.random.default_rng([31, group, symmetric])
    w = (g.standard_normal((2, 2 * group)) * 0.1 + (0 if symmetric else 0.05)).astype(np.float32)
    w[0, :group] = 0.0
    # Values half way between two codes (the scale is 1/8 or 1/4 exactly).
    w[1, :group] = (g.integers(-13, 15, group) / 16).astype(np.float32)
    w[1, 0], w[1, 1] = (0.875, -0.5) if symmetric else (0.9375, -0.9375)
    codes, bits, zeros = oracle.int4_quantize(w, group, symmetric, kind)
    s = oracle.scale_values(bits, kind)
    q = np.stack([codes & 15, codes >> 4], -1).reshape(w.shape)
    for r in range(2):
        for c in range(2):
            v = [_f(x) for x in w[r, c * group:(c + 1) * group]]
            if symmetric:
                span, by = max(abs(x) for x in v), 7
            else:
                span, by = round_binary(max(max(v), 0) - min(min(v), 0), 23, -126), 15
            want = round_binary(round_binary(span / by, 23, -126), frac, emin)
            assert _f(s[r, c]) == want
            z = 8 if symmetric else 0
            if want and not symmetric:
                z = min(max(round(-min(min(v), Fraction(0)) / want), 0), 15)
            if not symmetric:
                assert zeros[r, c] == z
            for j, x in enumerate(v):
                n = round(x / want) if want else 0
                assert q[r, c * group + j] == min(max(n + z, 0), 15)


def test_int4_quantize_of_what_is_not_finite():
    w = np.ones((1, 128), np.float32)
    w[0, 3], w[0, 40] = np.inf, np.nan
    w[0, 64:96] = 0
    for symmetric, code in ((True, 0x88), (False, 0)):
        codes, bits, zeros = oracle.int4_quantize(w, 32, symmetric)
        assert list(bits[0, :3]) == [0x7FC0, 0x7FC0, 0] and np.isfinite(oracle.scale_values(bits, "bf16")[0, 2:]).all()
        assert (codes[0, :48] == code).all()
        assert symmetric or (zeros[0, :3] == 0).all()
    # A scale past FP16's range
    _, bits, _ = oracle.int4_quantize(np.full((1, 32), 1e6, np.float32), 32, True, "fp16")
    assert bits[0, 0] == 0x7E00


def test_int4_values_and_products_by_hand():
    codes = np.array([[0x10, 0xF8] + [0x88] * 14], np.uint8)
    s = np.array([[0.5]])
    v = oracle.int4_values(codes, s)
    assert list(v[0, :4]) == [-4.0, -3.5, 0.0, 3.5] and (v[0, 4:] == 0).all()
    v = oracle.int4_values(codes, s, np.array([[3]], np.uint8))
    assert list(v[0, :4]) == [-1.5, -1.0, 2.5, 6.0]
    a = np.zeros((1, 32))
    a[0, :4] = [1, 2, 4, 8]
    out, terms, sums = oracle.gemm_int4(a, codes, s)
    assert out[0, 0] == -4 - 7 + 28 and sums[0, 0] == 17
    assert terms[0, 0] == 0.5 * (1 * (40 + 0) + 2 * (40 + 1) + 4 * (40 + 8) + 8 * (40 + 15))


def test_rmsnorm_by_rationals():
    g = np.random.default_rng(32)
    x = oracle.bf16_from_f64(g.standard_normal((3, 128)) * 2)
    r = oracle.bf16_from_f64(g.standard_normal((3, 128)))
    x[2] = 0
    r[2] = 0
    w = g.standard_normal(128).astype(np.float32).astype(np.float64)
    h, y = oracle.rmsnorm(x, w, 1e-6, r)
    xv, rv, yv = (oracle.bf16_bits_to_f64(b) for b in (x, r, y))
    hv = oracle.bf16_bits_to_f64(h)
    for i in range(3):
        for j in range(128):
            assert _f(hv[i, j]) == round_binary(_f(xv[i, j]) + _f(rv[i, j]), 7, -126)
        # (y / w)^2 (mean + eps) = h^2, to BF16's half step twice over
        mean = sum(_f(v) ** 2 for v in hv[i]) / 128 + Fraction(1e-6)
        for j in range(128):
            got, want = float((_f(yv[i, j]) / _f(w[j])) ** 2 * mean), float(_f(hv[i, j]) ** 2)
            assert abs(got - want) <= 2.0 ** -7 * want * 1.01
    assert (y[2] & 0x7FFF == 0).all()
