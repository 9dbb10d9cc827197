"""Pins of the 4-bit activation oracle: the quantization against exact
rationals and hand-packed bytes, the product against exact rationals, the
layer against the dense formula, and the router against hand-worked tokens and
its softmax / sigmoid closed forms."""

import math
from fractions import Fraction

import numpy as np
import pytest

import oracle

GRID = [Fraction(0), Fraction(1, 2), Fraction(1), Fraction(3, 2), Fraction(2), Fraction(3), Fraction(4),
        Fraction(6)]


def _nearest(r):
    """Index of the grid value nearest to the rational r >= 0, ties to the even index."""
    d = [abs(r - g) for g in GRID]
    best = min(d)
    near = [i for i, v in enumerate(d) if v == best]
    return near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]


def _block_by_rationals(v):
    amax = max(abs(Fraction(float(x))) for x in v)
    e = -127 + 2  # byte 0
    if amax > 0:
        e = math.floor(math.log2(float(amax)))
        while Fraction(2) ** e > amax:
            e -= 1
        while Fraction(2) ** (e + 1) <= amax:
            e += 1
    byte = max(e - 2 + 127, 0)
    scale = Fraction(2) ** (byte - 127)
    return [_nearest(abs(Fraction(float(x))) / scale) | (8 if math.copysign(1.0, x) < 0 else 0) for x in v], byte


@pytest.mark.parametrize("exp", [-149, -140, -127, -126, -125, -124, -20, 0, 7, 120, 127])
def test_quantization_against_rationals(exp):
    g = np.random.default_rng(exp + 200)
    v = (g.uniform(-1, 1, 320) * g.choice([1.0, 0.3, 0.05], 320)).astype(np.float32)
    v[::7] = g.choice([0.0, -0.0, 0.25, -0.75, 0.625, 0.875, 0.4375, 0.3125, 1.0], v[::7].shape)
    with np.errstate(under="ignore"):
        v = np.ldexp(v, exp).astype(np.float32)
    codes, scales = oracle.mxfp4_quantize(v.reshape(1, -1))
    got = oracle.fp4_unpack(codes)[0]
    for b in range(10):
        want, byte = _block_by_rationals(v[32 * b:32 * b + 32])
        assert scales[0, b] == byte
        assert got[32 * b:32 * b + 32].tolist() == want


def test_quantization_by_hand():
    v = np.zeros((2, 64))
    v[0, :9] = [4.0, 5.0, -6.0, 7.9, 2.5, 3.5, 0.25, -0.75, -0.0]  # amax in [4, 8): scale 1
    v[1, 3] = np.nan
    v[1, 40] = -np.inf
    codes, scales = oracle.mxfp4_quantize(v)
    assert scales.tolist() == [[127, 0], [255, 255]]
    # 4 -> 6, 5 -> 4 (tie to even), -6 -> -6, 7.9 -> 6, 2.5 -> 2, 3.5 -> 4, 0.25 -> 0, -0.75 -> -1, -0
    assert codes[0, :5].tolist() == [0x66, 0x7F, 0x64, 0xA0, 0x08]
    assert not codes[0, 5:].any() and not codes[1].any()


def test_quantized_values_decode_to_themselves():
    g = np.random.default_rng(3)
    codes = g.integers(0, 256, (5, 64), dtype=np.uint8)
    codes[:, ::16] |= 0x07  # a magnitude of 6 in every block, so its scale is found again
    scales = g.integers(0, 250, (5, 4), dtype=np.uint8)
    c, s = oracle.mxfp4_quantize(oracle.mxfp4_dequant(codes, scales))
    assert np.array_equal(c, codes) and np.array_equal(s, scales)


def test_product_against_rationals():
    g = np.random.default_rng(4)
    a, w = (g.integers(0, 256, (r, 32), dtype=np.uint8) for r in (2, 3))
    sa, sw = (g.integers(100, 150, (r, 2), dtype=np.uint8) for r in (2, 3))
    bits, mag = oracle.gemm_rows_mx4(a, sa, w, sw)

    def value(codes, scales, r, k):
        n = int(codes[r, k // 2]) >> (4 * (k % 2)) & 15
        return (-1 if n & 8 else 1) * GRID[n & 7] * Fraction(2) ** (int(scales[r, k // 32]) - 127)
    for i in range(2):
        for j in range(3):
            terms = [value(a, sa, i, k) * value(w, sw, j, k) for k in range(64)]
            want = oracle.bf16_from_f64(np.array(float(sum(terms))))
            assert bits[i, j] == want
            assert mag[i, j] == pytest.approx(float(sum(abs(t) for t in terms)), rel=1e-12)


def test_layer_of_one_expert_is_the_dense_formula():
    g = np.random.default_rng(5)
    h, i = 128, 128
    x = oracle.bf16_from_f64(g.standard_normal((3, h)))
    w1 = (g.integers(0, 256, (1, 2 * i, h // 2), dtype=np.uint8), g.integers(118, 122, (1, 2 * i, h // 32), dtype=np.uint8))
    w2 = (g.integers(0, 256, (1, h, i // 2), dtype=np.uint8), g.integers(118, 122, (1, h, i // 32), dtype=np.uint8))
    ids = np.array([[0], [0], [5]], np.int32)
    out, mag = oracle.token_forward_mx4(x, ids, np.full((3, 1), 0.5, np.float32), w1, w2, 1, 3)
    xd = oracle.mxfp4_dequant(*oracle.mxfp4_quantize(oracle.bf16_bits_to_f64(x)))
    c1 = oracle.bf16_bits_to_f64(oracle.bf16_from_f64(xd @ oracle.mxfp4_dequant(w1[0][0], w1[1][0]).T))
    hh = (c1[:, :i] / (1 + np.exp(-c1[:, :i])) * c1[:, i:]).astype(np.float32)
    y = oracle.bf16_bits_to_f64(oracle.bf16_from_f64(
        oracle.mxfp4_dequant(*oracle.mxfp4_quantize(hh)) @ oracle.mxfp4_dequant(w2[0][0], w2[1][0]).T))
    np.testing.assert_array_equal(out[:2], 0.5 * y[:2])
    assert not out[2].any() and not mag[2].any()  # another rank's expert
    np.testing.assert_array_equal(mag[:2], 0.5 * np.abs(y[:2]))


def test_route_by_hand():
    l = np.array([[1.0, 3.0, 3.0, 2.0]])
    ids, w = oracle.route(l, 3)
    e = [math.exp(v) for v in (3, 3, 2)]
    assert ids.tolist() == [[1, 2, 3]]  # a tie: the lower index first
    assert w[0] == pytest.approx([v / sum(e) for v in e], rel=1e-14)
    _, w = oracle.route(l, 2, renormalize=False, scale=2.0)
    assert w[0] == pytest.approx([2 * math.exp(3) / (2 * math.exp(3) + math.exp(1) + math.exp(2))] * 2, rel=1e-14)
    # the bias moves the choice, not the weight
    ids, w = oracle.route(l, 1, score="sigmoid", bias=np.array([9.0, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[0]] and w[0, 0] == pytest.approx(1 / (1 + math.exp(-1)), rel=1e-14)


def test_route_groups_by_hand():
    # groups (0, 1), (2, 3), (4, 5): best 5, 4, 4.5; sums of sigmoids differ
    l = np.array([[5.0, -9.0, 4.0, 4.0, 4.5, -2.0]])
    assert oracle.route(l, 2, num_groups=3, top_groups=1)[0].tolist() == [[0, 1]]
    assert oracle.route(l, 2, "sigmoid", num_groups=3, top_groups=1, group_top=2)[0].tolist() == [[2, 3]]
    assert oracle.route(l, 3, num_groups=3, top_groups=2)[0].tolist() == [[0, 4, 5]]
    # equal groups: the lower one
    assert oracle.route(np.ones((1, 6)), 2, num_groups=3, top_groups=1)[0].tolist() == [[0, 1]]


def test_route_masked_tokens():
    inf = math.inf
    l = np.array([[-inf, 1.0, math.nan, -inf], [-inf] * 4, [inf, 0.0, inf, -inf]])
    ids, w = oracle.route(l, 3)
    assert ids.tolist() == [[1, -1, -1], [-1, -1, -1], [0, 2, 1]]
    assert w.tolist() == [[1.0, 0, 0], [0, 0, 0], [0.5, 0.5, 0]]
