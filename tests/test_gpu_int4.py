"""4-bit integer weights on the GPU against the fp64 oracle: quantization and
dequantization bit for bit, products within bounds derived here.

A product's BF16 output is off by half a step of its value (2**-8), and the sums
before it: within a group of G columns the matrix cores add G products of
magnitude |a| (16 + q) and the sum of a as often, each addition off by at most
2**-23 of what the group's magnitudes add up to, so (G + 2) 2**-23 T with T the
scaled magnitudes sum s |a| (32 + q + z); a group's result is then scaled
(2**-24 twice) and added to the others, (groups + 8) 2**-24 U with U the sum of
the groups' magnitudes. Gated: SiLU's slope is at most 1.1, so an error dg of
the gate and du of the up give 1.1 |u| dg + |SiLU(g)| du + 1.1 dg du, and the
fp32 exponential, quotient and product 2**-20 of the result. With more than
EXACT_ROWS rows the weights may be the BF16 values of moe_int4_dequant, rounded
in the reference too (every row of a product is then within the bound of that
reference, or every one of the exact one's), and one sum runs over K: of its additions, a product's
four at a time at least, each is off by at most 2**-23 of the sum of
magnitudes: (K / 4 + 16) 2**-23 sum |a w|. Sums that are exact in fp32 (small integers, scales that are powers of two) are compared bit
for bit."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
import oracle
from tests.gpu_helpers import POISON_BF16, dev, down, say, up

pytestmark = pytest.mark.gpu

INF = float("inf")
ACTS = [None, "swiglu", "swiglu_clamp", "swiglu_clamp_after_silu"]
EXACT_ROWS = 64
KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _rng(*key):
    return np.random.default_rng([int(k) for k in key])


def _bf16(a):
    return oracle.bf16_from_f64(np.asarray(a, np.float64))


def _i32(v):
    return up(np.asarray(v, np.int32))


def _scales(bits, kind):
    return up(np.asarray(bits, np.uint16)).view(KINDS[kind])


# ---- quantization ------------------------------------------------------------

def _typed(w, dtype):
    t = torch.from_numpy(np.asarray(w, np.float32)).to(dtype)
    return t.to(dev()), t.double().numpy()


def _check_quant(w, dtype, group, symmetric, kind):
    t, v = _typed(w, dtype)
    codes, scales, zeros = moe.moe_int4_quant(t, group, symmetric, KINDS[kind])
    want = oracle.int4_quantize(v, group, symmetric, kind)
    assert np.array_equal(down(scales.view(torch.int16)), want[1])
    if symmetric:
        assert zeros is None
    else:
        assert np.array_equal(down(zeros), want[2])
    assert np.array_equal(down(codes), want[0])
    out = moe.moe_int4_dequant(codes, scales, zeros)
    s = oracle.scale_values(want[1], kind)
    with np.errstate(invalid="ignore"):
        ref = oracle.int4_values(want[0], s, want[2])
    got = out.double().cpu().numpy()
    dead = np.isnan(ref)
    assert np.array_equal(np.isnan(got), dead)
    assert np.array_equal(down(out.view(torch.int16))[~dead], _bf16(np.where(dead, 0, ref))[~dead])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantization_matches_oracle(dtype, group, symmetric, kind):
    g = _rng(400, group, symmetric)
    for rows, groups in ((1, 1), (3, 5), (130, 7), (257, 16)):
        say(f"int4 quant {rows} x {groups * group} {dtype} {symmetric} {kind}")
        w = g.standard_normal((rows, groups * group)) * np.exp(g.standard_normal((rows, 1)))
        w[0, :group] = 0.0
        if rows > 1:
            w[1, :group] = np.abs(w[1, :group])   # one sign
            w[2, :group] = 0.37                   # one value
            w[2, group:] = -np.abs(w[2, group:])
        _check_quant(0.05 * w, dtype, group, symmetric, kind)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantization_at_ties(symmetric):
    """Quotients exactly half way between two codes go to the even one, and a
    float32's distance from that decides otherwise."""
    g = _rng(401)
    w = (g.integers(-13, 15, (64, 64)) / 16).astype(np.float32)
    w[:, 0], w[:, 1] = (0.875, -0.5) if symmetric else (0.9375, -0.9375)
    w[1::2, 2:] = np.nextafter(w[1::2, 2:], np.float32(2) * g.choice([-1, 1], (32, 62)).astype(np.float32))
    for group in (32, 64):
        if group == 32:
            w[:, 32], w[:, 33] = w[:, 0], w[:, 1]
        _check_quant(w, torch.float32, group, symmetric, "bf16")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("symmetric", [True, False])
def test_quantization_of_the_ends_of_the_range(symmetric, kind):
    g = _rng(402)
    w = g.standard_normal((14, 128)).astype(np.float32)
    for r, e in enumerate((-149, -140, -133, -127, -100, -64, -62, -24, -16, -10, 15, 18, 100, 125)):
        w[r] = (w[r] * np.float32(2.0) ** np.float32(e / 2)) * np.float32(2.0) ** np.float32(e - e / 2)
    _check_quant(w, torch.float32, 32, symmetric, kind)
    w = g.standard_normal((6, 128)).astype(np.float32)
    w[0, 5], w[1, 40], w[2, 70], w[3, 100] = np.inf, -np.inf, np.nan, -np.nan
    w[4, :32] = 3.4e38
    w[4, 1] = -3.4e38
    for group in (32, 128):
        _check_quant(w, torch.float32, group, symmetric, kind)


def test_dequantization_of_any_zero_point_and_scale():
    g = _rng(403)
    codes = g.integers(0, 256, (40, 128), dtype=np.uint8)
    zeros = g.integers(0, 256, (40, 8), dtype=np.uint8)
    for kind in ("bf16", "fp16"):
        bits = g.integers(0, 1 << 16, (40, 8)).astype(np.uint16)
        s = oracle.scale_values(bits, kind)
        with np.errstate(invalid="ignore", over="ignore"):
            ref = oracle.int4_values(codes, s, zeros)
        out = moe.moe_int4_dequant(up(codes), _scales(bits, kind), up(zeros))
        ok = np.isfinite(ref)
        got = out.double().cpu().numpy()
        assert np.array_equal(down(out.view(torch.int16))[ok], _bf16(np.where(ok, ref, 0))[ok])
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        inf = np.isinf(ref)
        assert np.array_equal(got[inf], ref[inf])


def test_quantization_of_leading_dimensions_and_none():
    w = torch.randn((3, 5, 96), device=dev()).bfloat16()
    codes, scales, zeros = moe.moe_int4_quant(w, 32, symmetric=False)
    assert codes.shape == (3, 5, 48) and scales.shape == zeros.shape == (3, 5, 3)
    c2, s2, z2 = moe.moe_int4_quant(w.view(15, 96), 32, symmetric=False)
    assert torch.equal(c2, codes.view(15, 48)) and torch.equal(s2, scales.view(15, 3)) and torch.equal(z2, zeros.view(15, 3))
    assert torch.equal(moe.moe_int4_dequant(codes, scales, zeros).view(15, 96), moe.moe_int4_dequant(c2, s2, z2))
    codes, scales, _ = moe.moe_int4_quant(torch.empty((0, 64), device=dev()), 64)
    assert moe.moe_int4_dequant(codes, scales).shape == (0, 64)
    one = moe.moe_int4_quant(w[0, 0], 32)
    assert one[0].shape == (48,) and moe.moe_int4_dequant(one[0], one[1]).shape == (96,)


# ---- products ------------------------------------------------------------------

def _weights(g, lead, n, k, group, zeros, kind, exact=False):
    """(codes, scale bits, fp64 scales, zeros or None) of [lead..., n, k]."""
    shape = tuple(lead) + (n,)
    codes = g.integers(0, 256, shape + (k // 2,), dtype=np.uint8)
    s = np.exp2(g.integers(-3, 3, shape + (k // group,))) if exact else g.uniform(0.004, 0.016, shape + (k // group,))
    s = s * g.choice([-1.0, 1.0], s.shape)
    bits, s = oracle.scale_round(s.astype(np.float32), kind)
    z = g.integers(0, 16, s.shape, dtype=np.uint8) if zeros else None
    return codes, bits, s, z


def _silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def _reference(a, codes, s, z, act, lim, many=False):
    """(values, error bounds without the final rounding) [m, n_out] in fp64."""
    k, groups = a.shape[1], s.shape[1]
    if many:
        w = oracle.bf16_bits_to_f64(_bf16(oracle.int4_values(codes, s, z)))
        out = a @ w.T
        err = (k / 4 + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)
    else:
        out, terms, sums = oracle.gemm_int4(a, codes, s, z)
        err = (k // groups + 2) * 2.0 ** -23 * terms + (groups + 8) * 2.0 ** -24 * sums
    if act is None:
        return out, err
    n = out.shape[1] // 2
    gate, u, dg, du = out[:, :n], out[:, n:], err[:, :n], err[:, n:]
    if act == "swiglu_clamp":
        gate = np.minimum(gate, lim)
    si = _silu(gate)
    if act == "swiglu_clamp_after_silu":
        si = np.minimum(si, lim)
    if act != "swiglu":
        u = np.clip(u, -lim, lim)
    v = si * u
    return v, 1.1 * np.abs(u) * dg + np.abs(si) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(v)


def _off(bits, ref, err):
    got = oracle.bf16_bits_to_f64(bits)
    bound = err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    return ~(np.abs(got - ref) <= bound), got, bound


def _close_many(bits, many, what, *args):
    """Within the bound of the exact form, or with more rows of the rounded one."""
    if many and not _off(bits, *_reference(*args, many=True))[0].any():
        return
    _close(bits, *_reference(*args), what)


def _close(bits, ref, err, what=""):
    bad, got, bound = _off(bits, ref, err)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3], bound[bad][:3])


def _linear(g, rows, k, n, group, zeros=False, act=None, kind="bf16", lim=1.5, live=None, exact=False):
    codes, bits, s, z = _weights(g, (), n, k, group, zeros, kind, exact)
    av = g.integers(-3, 4, (rows, k)).astype(np.float64) if exact else g.standard_normal((rows, k))
    ab = _bf16(av)
    out_n = n if act is None else n // 2
    out = torch.full((rows, out_n), POISON_BF16, dtype=torch.int16, device=dev())
    got = moe.moe_gemm_int4(up(ab), up(codes), _scales(bits, kind), None if z is None else up(z), act=act,
                            clamp_limit=lim, t_live=None if live is None else _i32([live]), out=out)
    assert got is out
    m = rows if live is None else live
    a = oracle.bf16_bits_to_f64(ab[:m])
    if exact and act is None:
        ref = _reference(a, codes, s, z, act, lim)[0]
        assert np.array_equal(down(out)[:m] & 0x7FFF, _bf16(ref) & 0x7FFF)
        assert np.array_equal(oracle.bf16_bits_to_f64(down(out)[:m]), oracle.bf16_bits_to_f64(_bf16(ref)))
    _close_many(down(out)[:m], m > EXACT_ROWS, (rows, k, n, group, zeros, act, kind), a, codes, s, z, act, lim)
    assert (down(out)[m:] == POISON_BF16).all()


LINEAR = [
    # rows, k, n
    (1, 32, 1), (1, 64, 2), (1, 128, 17), (1, 4096, 1024), (1, 7168, 4096), (2, 96, 33), (3, 160, 31),
    (4, 2880, 96), (5, 512, 512), (15, 640, 130), (16, 2048, 300), (17, 1024, 64), (31, 256, 1000),
    (32, 384, 16), (33, 416, 34), (48, 1152, 200), (64, 512, 256), (65, 128, 258), (100, 1408, 142),
    (129, 896, 128), (200, 288, 520), (300, 6144, 100), (513, 256, 384),
    # the tiled forms: 64 x 256, 128 x 256 and 128 x 512 tiles, whole and not
    (300, 544, 4099), (260, 256, 7168), (700, 384, 3100), (1030, 256, 4096), (1100, 416, 16390),
    (2048, 160, 8192), (2000, 96, 8001),
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,k,n", LINEAR)
def test_linear_matches_oracle(rows, k, n, group):
    if k % group:
        k = (k // group + 1) * group
    g = _rng(410, rows, k, n, group)
    for i, act in enumerate((None, ACTS[1 + (rows + n) % 3])):
        m = n if act is None else n + n % 2
        say(f"int4 linear {rows} x {k} -> {m} group {group} {act}")
        _linear(g, rows, k, m, group, zeros=(rows + i) % 2 == 1, act=act, kind=("bf16", "fp16")[(n + i) % 2])
        if act is None:
            _linear(g, rows, k, m, group, zeros=(rows + i) % 2 == 0, exact=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 9, 40, 300])
def test_linear_activations_and_zero_points(rows, act):
    g = _rng(411, rows)
    for zeros in (False, True):
        for kind in ("bf16", "fp16"):
            _linear(g, rows, 512, 192, 64, zeros, act, kind)


@pytest.mark.parametrize("live", [0, 1, 7, 50])
def test_linear_of_live_rows(live):
    g = _rng(412, live)
    _linear(g, 50, 256, 72, 32, True, None, live=live)
    _linear(g, 50, 256, 72, 128, False, "swiglu", live=live)


def test_linear_of_no_rows():
    g = _rng(413)
    codes, bits, _, _ = _weights(g, (), 8, 64, 32, False, "bf16")
    out = moe.moe_gemm_int4(torch.empty((0, 64), dtype=torch.bfloat16, device=dev()), up(codes), _scales(bits, "bf16"))
    assert out.shape == (0, 8) and out.dtype == torch.bfloat16


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_columns_that_cancel(rows):
    """Rows of one sign and weights of both: the offset's part of a group's sum
    is several times what stays."""
    g = _rng(414, rows)
    codes, bits, s, z = _weights(g, (), 48, 1024, 128, True, "fp16")
    ab = _bf16(100 + np.abs(g.standard_normal((rows, 1024))))
    out = moe.moe_gemm_int4(up(ab), up(codes), _scales(bits, "fp16"), up(z))
    _close_many(down(out.view(torch.int16)), rows > EXACT_ROWS, rows, oracle.bf16_bits_to_f64(ab), codes, s, z, None, INF)


@pytest.mark.parametrize("rows", [3, 70, 300])
@pytest.mark.parametrize("act", [None, "swiglu_clamp", "swiglu_clamp_after_silu"])
def test_nan_and_infinity_stay_in_their_rows(act, rows):
    g = _rng(415, rows)
    codes, bits, s, z = _weights(g, (), 64, 256, 64, False, "bf16")
    ab = _bf16(g.standard_normal((rows, 256)))
    clean = moe.moe_gemm_int4(up(ab), up(codes), _scales(bits, "bf16"), act=act, clamp_limit=1.0)
    bad = ab.copy()
    bad[1, 17], bad[rows - 1, 255] = 0x7FC0, 0x7F80
    out = moe.moe_gemm_int4(up(bad), up(codes), _scales(bits, "bf16"), act=act, clamp_limit=1.0)
    ok = np.ones(rows, bool)
    ok[[1, rows - 1]] = False
    assert torch.equal(out.view(torch.int16)[torch.from_numpy(ok)], clean.view(torch.int16)[torch.from_numpy(ok)])
    assert out[1].isnan().all()
    if act is None:  # a clamp takes an infinite sum to its limit
        assert not out[rows - 1].isfinite().any()
    # A scale that is NaN: its weight row's column alone
    bits[5, 1] = 0x7FC0
    out = moe.moe_gemm_int4(up(ab), up(codes), _scales(bits, "bf16"), act=act, clamp_limit=1.0)
    assert out[:, 5].isnan().all()
    keep = [c for c in range(out.shape[1]) if c != 5]
    assert torch.equal(out.view(torch.int16)[:, keep], clean.view(torch.int16)[:, keep])


@pytest.mark.parametrize("rows", [4, 12, 40, 300])
@pytest.mark.parametrize("act", ACTS[1:])
def test_gates_of_any_size(act, rows):
    """The exponential's overflow and underflow: SiLU goes to 0 and to its argument."""
    values = [0.0, 1e-30, 1.0, 20.0, 87.0, 88.5, 89.0, 100.0, 104.0, 127.0, 128.0, 150.0, 1e4, 1e15]
    values = [x for v in values for x in (v, -v)]
    lim = 1e3
    codes, bits, s, z = _weights(_rng(416), (), 8, 64, 32, False, "bf16", exact=True)
    codes[:] = 0x99  # 1
    bits[:], s[:] = 0x3F80, 1.0
    av = np.zeros((rows, 64))
    for r in range(rows):
        av[r, r * 7 % 64] = values[r % len(values)]
    ab = _bf16(av)
    out = moe.moe_gemm_int4(up(ab), up(codes), _scales(bits, "bf16"), act=act, clamp_limit=lim)
    a = oracle.bf16_bits_to_f64(ab)
    x = a.sum(1, keepdims=True)
    gate = np.minimum(x, lim) if act == "swiglu_clamp" else x
    with np.errstate(over="ignore"):
        ref = gate / (1.0 + np.exp(-gate))
    if act == "swiglu_clamp_after_silu":
        ref = np.minimum(ref, lim)
    u = x if act == "swiglu" else np.clip(x, -lim, lim)
    ref = np.repeat(ref * u, 4, 1)
    # The sums are exact; the exponential's argument is off by 2**-24 of itself at most.
    # In fp32 it is infinite for gates below -128 ln 2 = -88.7, and SiLU zero: there
    # |g| e**g, falling, is at most 88.8 * 2**-128 < 2**-121, times up.
    got = oracle.bf16_bits_to_f64(down(out.view(torch.int16)))
    bound = np.abs(ref) * (2.0 ** -8 + 2.0 ** -20 + 2.0 ** -23 * np.minimum(np.abs(gate), 200)) + 2.0 ** -126
    bound = bound + np.where(gate < -88.7, 2.0 ** -121 * np.abs(u), 0.0)
    assert (np.abs(got - ref) <= bound).all(), np.argwhere(~(np.abs(got - ref) <= bound))[:4]


# ---- per expert ------------------------------------------------------------------

def _aligned(counts, align):
    ends = np.cumsum((np.asarray(counts) + align - 1) // align * align)
    return np.asarray(counts, np.int32), np.concatenate([[0], ends]).astype(np.int32)


def _grouped(g, counts, align, k, n, group, zeros=False, act=None, kind="bf16", gather=0, bound=0, cap=0,
             slack=0, lim=1.5, exact=False):
    """gather > 0: rows come from a tensor of tokens through a map with that
    divisor; cap > 0: the batched layout."""
    e = len(counts)
    if cap:
        c, o = np.asarray(counts, np.int32), np.arange(e + 1, dtype=np.int64) * cap
        row_cap = e * cap
    else:
        c, o = _aligned(counts, align)
        row_cap = int(o[-1]) + slack
    codes, bits, s, z = _weights(g, (e,), n, k, group, zeros, kind, exact)
    a_rows = max(3, row_cap // 2) if gather else max(row_cap, 1)
    av = g.integers(-3, 4, (a_rows, k)).astype(np.float64) if exact else g.standard_normal((a_rows, k))
    ab = _bf16(av)
    a = oracle.bf16_bits_to_f64(ab)
    row_map = None
    src = np.arange(max(row_cap, 1))
    if gather:
        row_map = g.integers(0, a_rows * gather, max(row_cap, 1)).astype(np.int32)
        src = row_map // gather
        for x in range(0, row_cap, 7):  # rows without a source
            row_map[x] = (-1, -gather, a_rows * gather, 2 ** 31 - 1)[x // 7 % 4]
            src[x] = -1
    out_n = n if act is None else n // 2
    out = torch.full((max(row_cap, 1), out_n), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_int4(up(ab), up(codes), _scales(bits, kind), up(c), None if cap else up(o.astype(np.int32)),
                              row_cap, w_zeros=None if z is None else up(z),
                              a_row_map=None if row_map is None else up(row_map), a_row_div=max(gather, 1),
                              expert_cap=cap, max_rows_per_expert=bound, act=act, clamp_limit=lim, out=out)
    got = down(out)
    live = np.zeros(max(row_cap, 1), bool)
    for x in range(e):
        m = min(int(c[x]), int(o[x + 1] - o[x]))
        if m <= 0:
            continue
        at = slice(int(o[x]), int(o[x]) + m)
        live[at] = True
        rows = np.where((src[at] >= 0)[:, None], a[src[at]], 0.0)
        args = (rows, codes[x], s[x], None if z is None else z[x], act, lim)
        many = m > EXACT_ROWS and min(bound or row_cap, cap or row_cap) > EXACT_ROWS
        _close_many(got[at], many, (x, counts, k, n, group), *args)
        ref = _reference(*args)[0]
        if exact and act is None:
            assert np.array_equal(oracle.bf16_bits_to_f64(got[at]), oracle.bf16_bits_to_f64(_bf16(ref)))
    assert (got[~live] == POISON_BF16).all()
    return got


COUNTS = [
    [1], [0, 0, 1], [0, 0, 0], [1, 1, 1, 1, 1, 1, 1, 1], [0, 5, 0, 16, 1, 17, 0], [33, 0, 64, 2, 65, 1],
    [0] * 70 + [3] + [0] * 90 + [1, 2], [130, 1, 0, 300, 64], [1000, 3],
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("ci", range(len(COUNTS)))
def test_grouped_matches_oracle(ci, group):
    counts = COUNTS[ci]
    g = _rng(420, ci, group)
    for i, (align, gather, act) in enumerate(((16, 0, None), (1, 2, "swiglu"), (16, 3, "swiglu_clamp"))):
        say(f"int4 grouped {counts[:8]} align {align} gather {gather} {act} group {group}")
        _grouped(g, counts, align, 384, 66 + 32 * i, group, zeros=i != 1, act=act, kind=("bf16", "fp16")[i % 2],
                 gather=gather, bound=max(counts), slack=(0, 5, 40)[i])
    _grouped(g, counts, 8, 256, 47, group, exact=True, zeros=True)


@pytest.mark.parametrize("counts,cap", [([3, 0, 4, 4], 4), ([17, 99, 0], 20), ([150, 0, 256], 256)])
def test_grouped_batched_layout(counts, cap):
    """masked_m may exceed the capacity; rows past the mask are untouched."""
    g = _rng(421, cap)
    _grouped(g, counts, 1, 256, 64, 64, cap=cap, zeros=True)
    _grouped(g, counts, 1, 256, 64, 32, cap=cap, act="swiglu", gather=2)


@pytest.mark.parametrize("k,n", [(256, 64), (96, 3100)])
def test_grouped_batched_counts_far_past_the_capacity(k, n):
    """Every expert has its capacity's rows then, the last one too."""
    _grouped(_rng(425, n), [9, 5000, 1 << 30, 200, 128, 130], 1, k, n, 32, cap=128, zeros=True)
    _grouped(_rng(426, n), [5000] * 40 + [3], 1, k, n, 32, cap=66)


@pytest.mark.parametrize("bound", [0, 1, 16, 17, 64, 65, 300])
def test_any_bound_gives_every_row(bound):
    """The bound selects kernels; a row count past it is computed all the same."""
    _grouped(_rng(422), [5, 0, 70, 20, 140], 16, 512, 96, 128, bound=bound, zeros=True)
    _grouped(_rng(423), [5, 0, 70, 20, 140], 16, 512, 96, 32, bound=bound, act="swiglu")


def test_endpoints_that_are_no_segments():
    """Offsets or counts that moe_align never makes: no row outside is written."""
    g = _rng(424)
    codes, bits, _, _ = _weights(g, (4,), 32, 128, 64, False, "bf16")
    a = torch.randn((64, 128), device=dev()).bfloat16()
    for counts, offsets in (([5, -3, 2, 4], [0, 16, 32, 48, 64]), ([5, 5, 5, 5], [0, 80, 32, -4, 900]),
                            ([2 ** 31 - 1] * 4, [0, 16, 32, 48, 64])):
        out = torch.full((70, 32), POISON_BF16, dtype=torch.int16, device=dev())
        moe.moe_grouped_gemm_int4(a, up(codes), _scales(bits, "bf16"), _i32(counts), _i32(offsets), 64, out=out)
        assert (down(out)[64:] == POISON_BF16).all()


def test_same_call_same_bits():
    g = _rng(425)
    codes, bits, _, z = _weights(g, (3,), 160, 1024, 32, True, "bf16")
    a = torch.randn((200, 1024), device=dev()).bfloat16()
    c, o = _aligned([100, 0, 70], 16)
    args = (a, up(codes), _scales(bits, "bf16"), up(c), up(o), 192)
    one = moe.moe_grouped_gemm_int4(*args, w_zeros=up(z))
    for _ in range(3):
        two = moe.moe_grouped_gemm_int4(*args, w_zeros=up(z), out=torch.zeros_like(one))
        live = torch.arange(192, device=dev())
        live = (live < 100) | ((live >= 112) & (live < 182))
        assert torch.equal(one.view(torch.int16)[live], two.view(torch.int16)[live])


# ---- the whole step ----------------------------------------------------------------

def _layer(x, r, gamma, router, w1, w2, e, topk, t_live=None, bufs=None):
    """Norm, routing, alignment, FC1 with SwiGLU, FC2 and the top-k sum."""
    b = bufs or {}
    t = x.shape[0]
    y, _, _, h = moe.moe_rmsnorm_quant(x, gamma, 1e-6, None, residual=r, t_live=t_live, y=b.get("y"),
                                       residual_out=b.get("h"))
    logits = y.float() @ router
    ids, tw = moe.moe_route(logits, topk, t_live=t_live)
    cap = moe.moe_min_row_cap(t, topk, e, 16)
    al = moe.moe_align(ids, e, 16, cap, t_live=t_live)
    c1 = moe.moe_grouped_gemm_int4(y, w1[0], w1[1], al["counts"], al["offsets"], cap, w_zeros=w1[2],
                                   a_row_map=al["row_to_pair"], a_row_div=topk, max_rows_per_expert=t, act="swiglu")
    c2 = moe.moe_grouped_gemm_int4(c1, w2[0], w2[1], al["counts"], al["offsets"], cap, w_zeros=w2[2],
                                   max_rows_per_expert=t)
    out = moe.moe_topk_combine(c2, al["pair_to_row"], tw, t_live=t_live, out=b.get("out"))
    return out, h, y, ids, tw


@pytest.mark.parametrize("tokens", [1, 4, 50, 200])
def test_layer_with_int4_experts(tokens):
    """A run as a decode step or a prompt makes it. FC1's output is rounded to
    BF16 (2**-8 of it) and goes through FC2: the bound carries it along."""
    g = _rng(430, tokens)
    e, hidden, inter, topk = 12, 512, 128, 3
    x, r = _bf16(g.standard_normal((tokens, hidden))), _bf16(g.standard_normal((tokens, hidden)))
    gamma = np.float32(1 + 0.1 * g.standard_normal(hidden))
    router = torch.from_numpy(g.standard_normal((hidden, e)).astype(np.float32)).to(dev())
    t1 = torch.from_numpy(0.05 * g.standard_normal((e, 2 * inter, hidden)).astype(np.float32)).to(dev()).bfloat16()
    t2 = torch.from_numpy(0.05 * g.standard_normal((e, hidden, inter)).astype(np.float32)).to(dev()).bfloat16()
    w1, w2 = moe.moe_int4_quant(t1, 64), moe.moe_int4_quant(t2, 32, symmetric=False, scale_dtype=torch.float16)
    out, h, y, ids, tw = _layer(up(x).view(torch.bfloat16), up(r), up(gamma), router, w1, w2, e, topk)
    want_h, want_y = oracle.rmsnorm(x, gamma.astype(np.float64), 1e-6, r)
    assert np.array_equal(down(h.view(torch.int16)), want_h) and np.array_equal(down(y.view(torch.int16)), want_y)
    yv, iv, wv = oracle.bf16_bits_to_f64(want_y), down(ids), down(tw).astype(np.float64)
    c = [[down(t) if t is not None and t.dtype == torch.uint8 else t for t in w] for w in (w1, w2)]
    s1 = oracle.scale_values(down(w1[1].view(torch.int16)), "bf16")
    s2 = oracle.scale_values(down(w2[1].view(torch.int16)), "fp16")
    ref, bound = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for x_ in range(e):
        t, k = np.nonzero(iv == x_)
        if not t.size:
            continue
        assert t.size <= EXACT_ROWS
        v1, e1 = _reference(yv[t], c[0][0][x_], s1[x_], None, "swiglu", INF)
        e1 = e1 * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(v1)
        v2, e2 = _reference(v1, c[1][0][x_], s2[x_], c[1][2][x_], None, INF)
        through = e1 @ np.abs(oracle.int4_values(c[1][0][x_], s2[x_], c[1][2][x_])).T
        e2 = (e2 + through) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(v2)
        np.add.at(ref, t, wv[t, k][:, None] * v2)
        np.add.at(bound, t, wv[t, k][:, None] * (e2 + (topk + 1) * 2.0 ** -24 * np.abs(v2)))
    _close(down(out), ref, bound)


def test_layer_captured_and_replayed():
    g = _rng(431)
    e, hidden, inter, topk, t = 10, 256, 128, 2, 24
    new = lambda: up(_bf16(g.standard_normal((t, hidden)))).view(torch.bfloat16)  # noqa: E731
    x, r = new(), new()
    gamma = torch.ones(hidden, device=dev())
    router = torch.from_numpy(g.standard_normal((hidden, e)).astype(np.float32)).to(dev())
    w1 = moe.moe_int4_quant(torch.from_numpy(0.1 * g.standard_normal((e, 2 * inter, hidden)).astype(np.float32)).to(dev()), 32)
    w2 = moe.moe_int4_quant(torch.from_numpy(0.1 * g.standard_normal((e, hidden, inter)).astype(np.float32)).to(dev()), 128)
    live = _i32([t])
    bufs = dict(y=torch.zeros_like(x), h=torch.zeros_like(x), out=torch.zeros((t, hidden), dtype=torch.int16, device=dev()))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            _layer(x, r, gamma, router, w1, w2, e, topk, live, bufs)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _layer(x, r, gamma, router, w1, w2, e, topk, live, bufs)
    for n in (t, 1, 0, 13, t):
        x.copy_(new())
        r.copy_(new())
        live.fill_(n)
        for b in bufs.values():
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = _layer(x, r, gamma, router, w1, w2, e, topk, _i32([n]))
        assert torch.equal(bufs["out"][:n], want[0][:n]) and not bufs["out"][n:].any()
        assert torch.equal(bufs["h"][:n], want[1][:n]) and not bufs["h"][n:].any()


def test_two_streams_at_once():
    g = _rng(432)
    codes, bits, _, _ = _weights(g, (), 512, 2048, 128, False, "bf16")
    w, s = up(codes), _scales(bits, "bf16")
    a = [torch.randn((m, 2048), device=dev()).bfloat16() for m in (1, 100, 400)]
    want = [moe.moe_gemm_int4(x, w, s) for x in a]
    streams = [torch.cuda.Stream() for _ in a]
    got = []
    for x, st in zip(a, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(5):
                y = moe.moe_gemm_int4(x, w, s)
            got.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
