"""The 4-bit activation operators on the GPU against the fp64 oracle: routing,
MXFP4 quantization (bit for bit), dequantization, SiLU * up with MXFP4
quantization (bit for bit), the MXFP4 x MXFP4 grouped product and the whole
layer, at sizes and inputs where they can go wrong.

Bounds. Codes, scale bytes, expert ids: equal. A routing weight is one
rounding to float32 of a double (2**-24 relative, and the oracle's double is
within a few 2**-52): 2**-23. A product's BF16 output: half a step of the
value (2**-8) plus the fp32 accumulation of K products, each addition off by
at most one unit in the last place of a running sum of at most the sum of
magnitudes: K * 2**-23 * sum |a w|. The whole layer's inputs are chosen so
that FC1 sums exactly (see _exact_layer); an expert output may then round to
the other side of a BF16 tie, a step of 2**-7, and the weighted sum adds its
own rounding, 2**-8, and top-k fp32 additions: 2**-7 * sum |w y| + 2**-8 * |out|
+ (topk + 1) * 2**-24 * sum |w y|."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
import oracle
from tests.gpu_helpers import POISON_BF16, POISON_I32, POISON_U8, dev, down, say, up

pytestmark = pytest.mark.gpu

INF = float("inf")
ACTS = [("swiglu", INF), ("swiglu_clamp", 1.5), ("swiglu_clamp_after_silu", 1.5)]


def _rng(*key):
    return np.random.default_rng([int(k) for k in key])


def _bf16(a):
    return oracle.bf16_from_f64(np.asarray(a, np.float64))


def _mx(g, rows, cols, lo=118, hi=124):
    return (g.integers(0, 256, (rows, cols // 2), dtype=np.uint8),
            g.integers(lo, hi, (rows, cols // 32)).astype(np.uint8))


def _i32(v):
    return up(np.asarray(v, np.int32))


# ---- routing --------------------------------------------------------------------

def _as(logits, dtype):
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype)
    return t.to(dev()), t.double().numpy()


def _check_route(l, ref_l, topk, bias=None, **kw):
    b = None if bias is None else up(bias.astype(np.float32))
    ids, w = moe.moe_route(l, topk, bias=b, **kw)
    torch.cuda.synchronize()
    ri, rw = oracle.route(ref_l, topk, bias=bias, **kw)
    assert np.array_equal(down(ids), ri)
    err = np.abs(down(w).astype(np.float64) - rw)
    assert np.all(err <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149)


ROUTES = [
    # tokens, experts, topk, options
    (1, 1, 1, {}),
    (1, 288, 8, {}),
    (5, 8, 8, dict(renormalize=False)),
    (3, 63, 5, dict(score="sigmoid")),
    (4, 64, 64, dict(score="sigmoid", renormalize=False, scale=2.5)),
    (7, 65, 3, dict(scale=-0.5)),
    (2, 129, 8, dict(num_groups=3, top_groups=2)),
    (6, 256, 8, dict(num_groups=8, top_groups=4, group_top=2, score="sigmoid")),
    (3, 320, 6, dict(num_groups=64, top_groups=7, group_top=2)),
    (2, 513, 12, dict(num_groups=27, top_groups=1)),
    (2, 1024, 8, dict(num_groups=4, top_groups=4, group_top=2)),
    (9, 12, 4, dict(num_groups=12, top_groups=4, group_top=2)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("ci", range(len(ROUTES)))
def test_route_matches_oracle(ci, biased, dtype):
    t, e, k, kw = ROUTES[ci]
    g = _rng(10, ci, biased)
    say(f"route {ROUTES[ci]} bias={biased} {dtype}")
    l, ref = _as(2.0 * g.standard_normal((t, e)), dtype)
    bias = 0.3 * g.standard_normal(e).astype(np.float32) if biased else None
    _check_route(l, ref, k, bias, **kw)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("tokens", [1, 3, 4, 17])
@pytest.mark.parametrize("experts,topk,kw", [
    (2, 1, {}), (16, 16, dict(score="sigmoid")), (17, 17, {}), (32, 2, dict(renormalize=False)),
    (48, 16, dict(num_groups=16, top_groups=9, group_top=2)), (64, 16, dict(num_groups=4, top_groups=1)),
    (60, 4, dict(num_groups=3, top_groups=2, group_top=2)), (34, 2, dict(num_groups=17, top_groups=3)),
    (62, 7, dict(num_groups=31, top_groups=8, group_top=2, score="sigmoid"))])
def test_route_of_few_experts(experts, topk, kw, tokens, biased):
    g = _rng(15, experts, topk, tokens)
    l, ref_l = _as(g.standard_normal((tokens, experts)) * 3, torch.float32)
    bias = np.float32(g.standard_normal(experts) * 0.3) if biased else None
    _check_route(l, ref_l, topk, bias=bias, **kw)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("capacity,experts,topk,kw", [
    (8192, 65, 8, {}), (8191, 65, 8, {}), (8192, 128, 16, dict(score="sigmoid", num_groups=16, top_groups=5)),
    (8192, 128, 17, {}), (9000, 256, 8, dict(num_groups=8, top_groups=4, group_top=2, score="sigmoid")),
    (8192, 256, 6, dict(renormalize=False)), (8192, 255, 4, dict(num_groups=17, top_groups=2, group_top=2)),
    (8192, 257, 3, {})])
def test_route_of_many_tokens(capacity, experts, topk, kw, biased):
    """Sizes around those at which fewer lanes take a token; the live count
    ends inside a wave and the rest of the rows stay as they were."""
    g = _rng(16, capacity, experts, topk)
    live = 41
    l, ref_l = _as(g.standard_normal((capacity, experts)) * 3, torch.bfloat16)
    bias = np.float32(g.standard_normal(experts) * 0.3) if biased else None
    ids = torch.full((capacity, topk), POISON_I32, dtype=torch.int32, device=dev())
    w = torch.full((capacity, topk), 7.0, device=dev())
    moe.moe_route(l, topk, bias=None if bias is None else up(bias), t_live=_i32([live]), ids=ids, weights=w, **kw)
    ri, rw = oracle.route(ref_l[:live], topk, bias=bias, **kw)
    assert np.array_equal(down(ids)[:live], ri)
    assert np.all(np.abs(down(w)[:live] - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149)
    assert np.all(down(ids)[live:] == POISON_I32) and np.all(down(w)[live:] == 7.0)


@pytest.mark.parametrize("kw", [{}, dict(score="sigmoid"), dict(num_groups=4, top_groups=2, group_top=2),
                                dict(num_groups=4, top_groups=2, renormalize=False)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_ties_and_extremes(biased, kw):
    inf, nan, big = np.inf, np.nan, np.finfo(np.float32).max
    g = _rng(11)
    rows = [np.full(16, -inf), np.full(16, nan), np.zeros(16), np.full(16, inf),
            np.where(np.arange(16) == 9, 1.0, -inf), np.tile([0.0, -0.0], 8),
            np.where(np.arange(16) % 3 == 0, nan, 2.0), np.where(np.arange(16) < 2, inf, big),
            np.full(16, -big), np.where(np.arange(16) > 10, -inf, -800.0),
            np.where(np.arange(16) == 4, -1e-45, 1e-45)]
    for _ in range(6):
        r = g.integers(-2, 3, 16).astype(np.float64)  # many ties
        r[g.integers(0, 16, 5)] = -inf
        rows.append(r)
    l = np.stack(rows).astype(np.float32)
    bias = None
    if biased:
        bias = np.zeros(16, np.float32)
        bias[[2, 5, 7, 11]] = [-inf, nan, inf, 0.25]
    say(f"route extremes {kw} bias={biased}")
    _check_route(up(l), l.astype(np.float64), 6, bias, **kw)


@pytest.mark.parametrize("kw", [{}, dict(score="sigmoid"), dict(num_groups=4, top_groups=2, group_top=2),
                                dict(num_groups=20, top_groups=6, renormalize=False)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_and_ties_of_a_wave_per_token(biased, kw):
    inf, nan, e = np.inf, np.nan, 160
    g, i = _rng(17), np.arange(e)
    rows = [np.full(e, -inf), np.full(e, nan), np.zeros(e), np.where(i == 159, 1.0, -inf),
            np.where(i % 64 == 7, 3.0, -1.0), np.where(i < 130, -inf, 0.5), np.where(i % 3 == 0, nan, 2.0)]
    for _ in range(6):
        r = g.integers(-2, 3, e).astype(np.float64)  # many ties
        r[g.integers(0, e, 70)] = -inf
        rows.append(r)
    l = np.stack(rows).astype(np.float32)
    bias = None
    if biased:
        bias = np.zeros(e, np.float32)
        bias[[2, 65, 70, 131]] = [-inf, nan, inf, 0.25]
    say(f"route of a wave per token, extremes {kw} bias={biased}")
    _check_route(up(l), l.astype(np.float64), 6, bias, **kw)


def test_route_rows_apart_and_past_the_live_count():
    g = _rng(12)
    wide = up(g.standard_normal((9, 100)).astype(np.float32))
    view = wide[:, 3:73]  # 70 experts, rows 100 apart, not 16-byte aligned
    ids = torch.full((9, 4), POISON_I32, dtype=torch.int32, device=dev())
    w = torch.full((9, 4), -7.0, device=dev())
    for live in (-3, 0, 1, 6, 9, 20):
        ids.fill_(POISON_I32)
        w.fill_(-7.0)
        moe.moe_route(view, 4, t_live=_i32([live]), ids=ids, weights=w)
        n = min(max(live, 0), 9)
        ri, rw = oracle.route(down(view.contiguous()), 4)
        assert np.array_equal(down(ids)[:n], ri[:n]) and np.all(down(ids)[n:] == POISON_I32)
        assert np.allclose(down(w)[:n], rw[:n], rtol=2.0 ** -23) and np.all(down(w)[n:] == -7.0)


# ---- quantization -----------------------------------------------------------------

def _quant_inputs(g, rows, cols):
    v = g.standard_normal((rows, cols)) * np.exp2(g.integers(-3, 4, (rows, cols // 32)).repeat(32, 1))
    flat = v.reshape(-1, 32)
    n = len(flat)
    flat[::5] = 0.25 * g.integers(-24, 25, flat[::5].shape)  # the grid and its ties
    if n > 11:
        flat[1] = 0.0
        flat[2] = -0.0
        flat[3] *= 2.0 ** -130  # subnormal BF16
        flat[4] *= 2.0 ** 120
        flat[6, 7] = np.nan
        flat[7, 0] = np.inf
        flat[8, 31] = -np.inf
        flat[9] = np.where(np.arange(32) == 30, 1.0, 2.0 ** -20)
    return _bf16_any(v)


def _bf16_any(v):
    """BF16 bits, NaN and infinities included (the oracle's rounding takes finite values)."""
    with np.errstate(over="ignore"):
        t = torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 128), (1, 4096), (37, 640), (130, 7168)])
def test_quantization_bit_exact(rows, cols, rounding):
    say(f"quant {rows}x{cols} {rounding}")
    x = _quant_inputs(_rng(20, rows, cols), rows, cols)
    live = max(1, rows - 2)
    xq = torch.full((rows, cols // 2), POISON_U8, dtype=torch.uint8, device=dev())
    xs = torch.full((rows, cols // 32), POISON_U8, dtype=torch.uint8, device=dev())
    moe.moe_act_quant(up(x), "mxfp4", t_live=_i32([live]), xq=xq, xs=xs, rounding=rounding)
    codes, scales = oracle.mxfp4_quantize(oracle.bf16_bits_to_f64(x))
    assert np.array_equal(down(xs)[:live], scales[:live])
    assert np.array_equal(down(xq)[:live], codes[:live])
    assert np.all(down(xq)[live:] == POISON_U8) and np.all(down(xs)[live:] == POISON_U8)


def test_quantization_of_every_bf16_value():
    """Every finite BF16 pattern as the largest of its block, with values around the ties of its scale."""
    bits = np.array([b for b in range(1 << 15) if (b >> 7) != 255], np.uint16)
    x = np.zeros((len(bits), 32), np.float64)
    top = oracle.bf16_bits_to_f64(bits)
    x[:, 0] = top
    x[:, 1:17] = top[:, None] * np.arange(1, 17) / 17.0
    x[:, 17:] = -top[:, None] * np.arange(15) / 16.0
    x = _bf16_any(x).reshape(-1, 128)
    xq, xs = moe.moe_act_quant(up(x), "mxfp4")
    codes, scales = oracle.mxfp4_quantize(oracle.bf16_bits_to_f64(x))
    assert np.array_equal(down(xs), scales) and np.array_equal(down(xq), codes)


def test_dequantization_is_exact():
    g = _rng(21)
    codes, scales = _mx(g, 300, 96, 0, 252)
    scales[5, 1] = 255
    out = moe.moe_mxfp4_dequant(up(codes), up(scales))
    got = oracle.bf16_bits_to_f64(down(out.view(torch.int16)))
    want = oracle.mxfp4_dequant(codes, scales)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got)[~np.isnan(want)], np.signbit(want)[~np.isnan(want)])
    # past BF16's range: infinity (6 * 2**126 and more), the rest exact
    codes = np.tile(np.arange(16, dtype=np.uint8) * 17, (1, 2))[:, :16].copy()
    for byte in (252, 253, 254):
        got = oracle.bf16_bits_to_f64(down(moe.moe_mxfp4_dequant(
            up(codes), up(np.array([[byte]], np.uint8))).view(torch.int16)))
        want = oracle.mxfp4_dequant(codes, np.array([[byte]], np.uint8))
        over = np.abs(want) >= 2.0 ** 128
        assert np.all(np.isinf(got[over])) and np.array_equal(got[~over], want[~over])
    # more rows than one pass of the grid, and none
    codes, scales = _mx(g, 20000, 1024, 100, 140)
    got = moe.moe_mxfp4_dequant(up(codes), up(scales)).float().cpu().numpy()
    assert np.array_equal(got, oracle.mxfp4_dequant(codes, scales).astype(np.float32))
    assert moe.moe_mxfp4_dequant(up(codes[:0]), up(scales[:0])).shape == (0, 1024)


def _aligned(counts, align):
    counts = np.asarray(counts, np.int64)
    seg = (counts + align - 1) // align * align
    return counts.astype(np.int32), np.concatenate([[0], np.cumsum(seg)]).astype(np.int32)


@pytest.mark.parametrize("act,lim", ACTS)
@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
@pytest.mark.parametrize("counts,inter,align", [([1], 128, 16), ([3, 0, 17, 1], 384, 16),
                                                ([0, 0], 128, 1), ([700, 0, 301], 2048, 1)])
def test_silu_quantization_bit_exact(counts, inter, align, rounding, act, lim):
    say(f"silu {counts} inter={inter} {rounding} {act}")
    counts, offsets = _aligned(counts, align)
    rows = int(offsets[-1]) + 5
    g = _rng(22, rows, inter)
    gu = 2.0 * g.standard_normal((rows, 2 * inter))
    gu[0, :7] = [0.0, -0.0, 1e-6, 300.0, -300.0, 17.0, 2.0 ** -13]
    gu = _bf16(gu)
    hq = torch.full((rows, inter // 2), POISON_U8, dtype=torch.uint8, device=dev())
    hs = torch.full((rows, inter // 32), POISON_U8, dtype=torch.uint8, device=dev())
    moe.moe_silu_mul_quant(up(gu), up(counts), up(offsets), act, lim, "mxfp4", hq=hq, hs=hs,
                           rounding=rounding)
    v = oracle.bf16_bits_to_f64(gu)
    codes, scales = oracle.mxfp4_quantize(oracle.swiglu(v[:, :inter], v[:, inter:], act, lim, rounding))
    live = np.zeros(rows, bool)
    for e, c in enumerate(counts):
        live[offsets[e]:offsets[e] + c] = True
    assert np.array_equal(down(hs)[live], scales[live]) and np.array_equal(down(hq)[live], codes[live])
    assert np.all(down(hq)[~live] == POISON_U8) and np.all(down(hs)[~live] == POISON_U8)


def test_silu_quantization_masked_layout():
    g = _rng(23)
    cap, inter, masked = 9, 256, np.array([0, 9, 4, 1], np.int32)
    gu = _bf16(g.standard_normal((4 * cap, 2 * inter)))
    hq = torch.full((4 * cap, inter // 2), POISON_U8, dtype=torch.uint8, device=dev())
    hs = torch.full((4 * cap, inter // 32), POISON_U8, dtype=torch.uint8, device=dev())
    moe.moe_silu_mul_quant_masked(up(gu), up(masked), cap, fmt="mxfp4", hq=hq, hs=hs)
    v = oracle.bf16_bits_to_f64(gu)
    codes, scales = oracle.mxfp4_quantize(oracle.swiglu(v[:, :inter], v[:, inter:]))
    live = (np.arange(cap) < masked[:, None]).reshape(-1)
    assert np.array_equal(down(hs)[live], scales[live]) and np.array_equal(down(hq)[live], codes[live])
    assert np.all(down(hq)[~live] == POISON_U8) and np.all(down(hs)[~live] == POISON_U8)


def test_silu_quantization_of_infinities_and_nan():
    gu = np.zeros((1, 256))
    gu[0, :128] = 1.0
    gu[0, 128:] = 2.0
    gu[0, 3] = np.inf      # silu(inf) * 2 = inf
    gu[0, 40] = np.nan
    gu[0, 128 + 70] = -np.inf
    hq, hs = moe.moe_silu_mul_quant(up(_bf16_any(gu)), _i32([1]), _i32([0, 1]), fmt="mxfp4")
    assert down(hs)[0].tolist()[:3] == [255, 255, 255] and down(hs)[0, 3] != 255
    assert not down(hq)[0, :48].any()


# ---- the grouped product -------------------------------------------------------------

GEMMS = [
    # counts per expert, N, K, align
    ([1], 128, 128, 16),
    ([1, 0, 3, 2], 256, 256, 16),
    ([16, 17, 0, 15], 128, 640, 1),
    ([33, 0, 70, 1, 5], 384, 384, 16),
    ([64, 65], 512, 1024, 1),
    ([130, 7, 0, 31, 257], 256, 896, 16),
    ([0, 0, 0], 128, 128, 16),
    ([600, 1, 300], 640, 512, 16),
    ([3] * 40, 128, 2048, 1),
    ([65, 0, 2], 128, 128, 16),
    ([256, 257, 129], 896, 1536, 1),
    ([128, 300], 384, 2176, 16),
]


def _gemm(counts, n, k, align, gather, seed, masked=False, a_scale=None):
    g = _rng(30, seed, gather, masked)
    counts, offsets = _aligned(counts, align)
    e_n = len(counts)
    if masked:
        cap = int(max(counts.max(), 1)) + 3
        offsets = (np.arange(e_n + 1) * cap).astype(np.int32)
        row_cap = e_n * cap
    else:
        row_cap = int(offsets[-1]) + 9
    a_rows = 40 if gather else max(row_cap, 1)
    a, asc = _mx(g, a_rows, k)
    w, ws = zip(*[_mx(g, n, k) for _ in range(e_n)])
    w, ws = np.stack(w), np.stack(ws)
    row_map = None
    if gather:
        row_map = np.full(row_cap, -1, np.int32)
        for e in range(e_n):
            row_map[offsets[e]:offsets[e] + counts[e]] = g.integers(0, a_rows * 4, counts[e])
    return counts, offsets, row_cap, a, asc, w, ws, row_map


def _check_gemm(out, counts, offsets, a, asc, w, ws, row_map, k):
    got = down(out)
    live = np.zeros(len(got), bool)
    for e, c in enumerate(counts):
        rows = np.arange(offsets[e], offsets[e] + c)
        live[rows] = True
        if not c:
            continue
        src = rows if row_map is None else row_map[rows] // 4
        bits, mag = oracle.gemm_rows_mx4(a[src], asc[src], w[e], ws[e])
        want = oracle.mxfp4_dequant(a[src], asc[src]) @ oracle.mxfp4_dequant(w[e], ws[e]).T
        bound = 2.0 ** -8 * np.abs(want) + k * 2.0 ** -23 * mag
        bad = ~(np.abs(oracle.bf16_bits_to_f64(got[rows]) - want) <= bound)
        assert not bad.any(), f"expert {e}: {bad.sum()} outside, first {np.argwhere(bad)[0]}"
    assert np.all(got[~live] == POISON_BF16)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("ci", range(len(GEMMS)))
def test_product_matches_oracle(ci, gather):
    counts, n, k, align = GEMMS[ci]
    say(f"mx4 gemm {counts[:6]} n={n} k={k} gather={gather}")
    counts, offsets, row_cap, a, asc, w, ws, row_map = _gemm(counts, n, k, align, gather, ci)
    for bound in (0, int(max(counts.max(), 1))):
        out = torch.full((row_cap, n), POISON_BF16, dtype=torch.int16, device=dev())
        moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap,
                                   a_row_map=None if row_map is None else up(row_map),
                                   a_row_div=4 if gather else 1, max_rows_per_expert=bound, out=out)
        _check_gemm(out, counts, offsets, a, asc, w, ws, row_map, k)


# Eight experts and 32 column tiles: enough for the product through LDS. The
# mean rows per expert set the height of its row tiles, 64, 128, 192 or 256; in
# each set some end in a whole tile, some in one of at most 64 rows.
TILED = [
    [64, 1, 0, 65, 33, 17, 100, 40],
    [128, 129, 1, 64, 65, 192, 0, 61],
    [192, 193, 256, 257, 1, 0, 150, 151],
    [256, 257, 320, 321, 1, 0, 512, 400],
]


@pytest.mark.parametrize("k", [128, 640, 512, 1536, 1024, 2048])
@pytest.mark.parametrize("ci", range(len(TILED)))
def test_product_through_lds_matches_oracle(ci, k):
    gather, n = bool((ci + k // 128) & 1), 8064 if ci & 1 else 8192
    say(f"mx4 gemm through LDS {TILED[ci]} n={n} k={k} gather={gather}")
    counts, offsets, row_cap, a, asc, w, ws, row_map = _gemm(TILED[ci], n, k, 1, gather, 100 + ci)
    out = torch.full((row_cap, n), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap,
                               a_row_map=None if row_map is None else up(row_map), a_row_div=4 if gather else 1,
                               out=out)
    _check_gemm(out, counts, offsets, a, asc, w, ws, row_map, k)


@pytest.mark.parametrize("ci", [1, 3])
def test_product_through_lds_masked_layout(ci):
    counts, offsets, row_cap, a, asc, w, ws, _ = _gemm(TILED[ci], 8192, 768, 1, False, 110 + ci, masked=True)
    out = torch.full((row_cap, 8192), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), None, row_cap,
                               expert_cap=row_cap // len(counts), out=out)
    _check_gemm(out, counts, offsets, a, asc, w, ws, None, 768)


@pytest.mark.parametrize("k", [640, 1024])
def test_product_through_lds_of_nan_scales_and_sourceless_rows(k):
    counts, offsets, row_cap, a, asc, w, ws, row_map = _gemm(TILED[3], 8192, k, 1, True, 120)
    asc[7, 3] = 255
    ws[1, 5, 2] = 255
    for r, v in ((1, -4), (offsets[1] + 2, 4 * len(a)), (offsets[1] + 3, 4 * 7), (offsets[4], -2 ** 31),
                 (offsets[2] - 1, 2 ** 31 - 1)):
        row_map[r] = v
    out = torch.full((row_cap, 8192), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap,
                               a_row_map=up(row_map), a_row_div=4, out=out)
    got = oracle.bf16_bits_to_f64(down(out))
    for e, c in enumerate(counts):
        for r in range(offsets[e], offsets[e] + c):
            src = row_map[r] // 4 if row_map[r] >= 0 else -1
            nan = np.isnan(got[r])
            if not 0 <= src < len(a):
                assert not got[r].any(), (e, r)
                continue
            want = np.full(8192, src == 7)
            if e == 1:
                want[5] = True
            assert np.array_equal(nan, want), (e, r, src)


@pytest.mark.parametrize("ci", [1, 3, 5])
def test_product_masked_layout(ci):
    counts, n, k, align = GEMMS[ci]
    counts, offsets, row_cap, a, asc, w, ws, _ = _gemm(counts, n, k, align, False, ci, masked=True)
    cap = row_cap // len(counts)
    out = torch.full((row_cap, n), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), expert_cap=cap, out=out)
    _check_gemm(out, counts, offsets, a, asc, w, ws, None, k)


@pytest.mark.parametrize("counts", [[3, 20], [300, 90]])
def test_product_of_nan_scales_and_sourceless_rows(counts):
    """A NaN scale byte reaches exactly its row (of A) or its column (of W);
    a row whose map points outside A gives zeros."""
    counts, offsets, row_cap, a, asc, w, ws, row_map = _gemm(counts, 256, 512, 1, True, 50)
    asc[7, 3] = 255
    ws[1, 5, 2] = 255
    row_map[1] = -4
    row_map[offsets[1] + 2] = 4 * len(a)
    row_map[offsets[1] + 3] = 4 * 7
    out = torch.full((row_cap, 256), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap,
                               a_row_map=up(row_map), a_row_div=4, out=out)
    got = oracle.bf16_bits_to_f64(down(out))
    for e, c in enumerate(counts):
        for r in range(offsets[e], offsets[e] + c):
            src = row_map[r] // 4 if row_map[r] >= 0 else -1
            nan = np.isnan(got[r])
            if not 0 <= src < len(a):
                assert not got[r][~nan].any()
                continue
            want = np.full(256, src == 7)
            if e == 1:
                want[5] = True
            assert np.array_equal(nan, want), (e, r, src)


def test_product_does_not_depend_on_the_other_rows():
    """An expert's rows give the same bits alone and among others (no row's sum
    is taken in an order that the launch's other rows decide), twice the same."""
    counts, offsets, row_cap, a, asc, w, ws, _ = _gemm([40, 200, 3], 512, 1024, 16, False, 60)
    args = (up(w), up(ws), up(counts), up(offsets), row_cap)
    one = moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", *args)
    two = moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", *args)
    for e, c in enumerate(counts):
        r = slice(int(offsets[e]), int(offsets[e]) + int(c))
        assert torch.equal(one[r], two[r])


# ---- the whole layer -----------------------------------------------------------------

def _exact_layer(seed, tokens, experts, hidden, inter, topk):
    """Inputs whose FC1 sums are exact in fp32 in any order: x is E2M1 values
    with a 6 in every block of 32, times 2**-2 or 2**-3, so quantization keeps
    it; weight scales per expert span two binades. Every product is a multiple
    of 2**-2 times the smallest scale product, at most 36 times the largest
    (2**3 apart): sums of K <= 7168 of them stay below 4 * 36 * 8 * 7168 <
    2**23 units."""
    g = _rng(40, seed)
    mags = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    x = mags[g.integers(0, 8, (tokens, hidden // 32, 32))] * g.choice([-1, 1], (tokens, hidden // 32, 32))
    x[:, :, 0] = 6.0
    x *= np.exp2(-g.integers(2, 4, (tokens, hidden // 32)))[:, :, None]
    x = _bf16(x.reshape(tokens, hidden))
    w1 = (g.integers(0, 256, (experts, 2 * inter, hidden // 2), dtype=np.uint8),
          g.integers(118, 121, (experts, 2 * inter, hidden // 32)).astype(np.uint8))
    w2 = (g.integers(0, 256, (experts, hidden, inter // 2), dtype=np.uint8),
          g.integers(118, 121, (experts, hidden, inter // 32)).astype(np.uint8))
    ids = np.stack([g.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)
    w = g.uniform(0.05, 1.0, (tokens, topk)).astype(np.float32)
    return x, ids, w, w1, w2


def _check_layer(got_bits, ref, t_live, topk):
    out, mag = ref
    got = oracle.bf16_bits_to_f64(got_bits[:t_live])
    bound = (2.0 ** -7 + (topk + 1) * 2.0 ** -24) * mag + 2.0 ** -8 * np.abs(out)
    bad = ~(np.abs(got - out) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}"
    assert np.all(got_bits[t_live:] == POISON_BF16)


LAYERS = [
    # tokens, live, experts, hidden, inter, topk, expert_start, (act, lim), rounding
    (1, 1, 4, 128, 128, 1, 0, 0, "divide"),
    (1, 1, 16, 1024, 512, 8, 0, 0, "divide"),
    (4, 3, 24, 640, 384, 8, 0, 1, "reciprocal"),
    (8, 8, 5, 256, 128, 5, 0, 2, "divide"),      # most pairs share experts
    (16, 16, 6, 384, 256, 4, 2, 0, "divide"),    # 64 pairs; experts of another rank dropped
    (32, 31, 40, 512, 640, 2, 0, 0, "reciprocal"),
    (64, 64, 2, 256, 256, 1, 0, 1, "divide"),    # an expert of more than 16 and of more than 32 rows
    (13, 0, 8, 256, 128, 2, 0, 0, "divide"),     # nothing live
    (33, 33, 9, 256, 384, 3, 0, 2, "divide"),    # past the few-token path
    (200, 190, 7, 512, 256, 4, 1, 0, "reciprocal"),
]


def _forward(li, **over):
    t, live, e, h, i, k, start, ai, rounding = LAYERS[li]
    act, lim = ACTS[ai]
    x, ids, w, w1, w2 = _exact_layer(li, t, e, h, i, k)
    out = torch.full((t, h), POISON_BF16, dtype=torch.int16, device=dev())
    # experts [start, e) are this rank's
    own = slice(start, e)
    args = dict(act=act, clamp_limit=lim, t_live=_i32([live]), out=out, rounding=rounding, expert_start=start,
                weight_fmt="mxfp4")
    args.update(over)
    moe.moe_forward(up(x), up(ids), up(w), up(w1[0][own]), up(w1[1][own]), up(w2[0][own]), up(w2[1][own]),
                    "mxfp4", **args)
    ref = oracle.token_forward_mx4(x, ids, w, (w1[0][own], w1[1][own]), (w2[0][own], w2[1][own]), e - start,
                                   live, act, lim, rounding, start)
    return down(args["out"]), ref


@pytest.mark.parametrize("li", range(len(LAYERS)))
def test_layer_matches_oracle(li):
    say(f"mx4 layer {LAYERS[li]}")
    got, ref = _forward(li)
    _check_layer(got, ref, LAYERS[li][1], LAYERS[li][5])


@pytest.mark.parametrize("li", [2, 4, 9])
def test_layer_batched_layout_and_odd_row_alignment(li):
    t, live, e, h, i, k, start, ai, rounding = LAYERS[li]
    got, ref = _forward(li, expert_cap=t)
    _check_layer(got, ref, live, k)
    got, ref = _forward(li, align_rows=5)
    _check_layer(got, ref, live, k)


@pytest.mark.parametrize("t,k,e", [(1, 8, 3), (2, 5, 2), (5, 12, 4), (16, 4, 3), (1, 64, 7), (13, 5, 3)])
def test_layer_of_tokens_that_have_an_expert_more_than_once(t, k, e):
    say(f"mx4 layer of {t} tokens, {k} choices among {e} experts with repetition")
    x, ids, w, w1, w2 = _exact_layer(60 + t, t, max(e, k), 384, 256, k)
    g = _rng(61, t, k)
    ids = g.integers(0, e, (t, k)).astype(np.int32)
    ids[0] = ids[0, 0]
    w1, w2 = (w1[0][:e], w1[1][:e]), (w2[0][:e], w2[1][:e])
    out = torch.full((t, 384), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_forward(*[up(v) for v in (x, ids, w, *w1, *w2)], "mxfp4", weight_fmt="mxfp4", out=out)
    ref = oracle.token_forward_mx4(x, ids, w, w1, w2, e, t)
    _check_layer(down(out), ref, t, k)


@pytest.mark.parametrize("t,k,h,i", [(48, 1, 128, 128), (49, 1, 128, 128), (16, 3, 7168, 128), (17, 2, 7168, 128),
                                     (16, 1, 15360, 128), (16, 1, 16384, 128), (1, 2, 32768, 128),
                                     (8, 1, 30720, 128), (2, 1, 32640, 256),
                                     (4, 2, 128, 8192)])
def test_layer_at_the_limits_of_the_few_token_path(t, k, h, i):
    """48 and 49 pairs; hidden sizes whose tokens do and do not fit the LDS.
    The sums of _exact_layer are exact to K = 7168 and its FC2 sums short; past
    that about one block of 32 in 16 is kept, the rest is zeros."""
    say(f"mx4 layer {t} tokens, top {k}, {h} -> {i}")
    e = 5
    x, ids, w, w1, w2 = _exact_layer(70 + t, t, e, h, i, k)
    g = _rng(71, t, h)
    if h > 7168:
        x = x * np.repeat(g.random((t, h // 32)) < 1 / 16, 32, axis=1).astype(x.dtype)
    if i > 7168:
        w2[0][:] *= np.repeat(g.random((e, h, i // 32)) < 1 / 16, 16, axis=2).astype(np.uint8)
    out = torch.full((t, h), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_forward(*[up(v) for v in (x, ids, w, *w1, *w2)], "mxfp4", weight_fmt="mxfp4", out=out)
    ref = oracle.token_forward_mx4(x, ids, w, w1, w2, e, t)
    _check_layer(down(out), ref, t, k)


@pytest.mark.parametrize("t,i", [(2, 128), (5, 4096), (3, 16384), (60, 512)])
def test_layer_of_tokens_without_an_expert_here(t, i):
    """No id is this rank's: zeros, whatever the weights hold."""
    g = _rng(72, t, i)
    x = _bf16(g.standard_normal((t, 256)))
    ids = g.choice(np.array([-1, -2 ** 31, 3, 7, 2 ** 31 - 1], np.int32), (t, 6))
    w = g.random((t, 6)).astype(np.float32)
    w[0, 0] = np.nan
    codes = [torch.zeros(s, dtype=torch.uint8, device=dev()) for s in ((3, 2 * i, 128), (3, 256, i // 2))]
    scales = [torch.full(s, 255, dtype=torch.uint8, device=dev()) for s in ((3, 2 * i, 8), (3, 256, i // 32))]
    out = torch.full((t, 256), POISON_BF16, dtype=torch.int16, device=dev())
    say(f"mx4 layer without experts, {t} tokens, inter {i}")
    moe.moe_forward(up(x), up(ids), up(w), codes[0], scales[0], codes[1], scales[1], "mxfp4", weight_fmt="mxfp4",
                    out=out)
    assert not down(out).any()


@pytest.mark.parametrize("t,e,k", [(3, 12, 4), (100, 12, 4)])
def test_router_and_layer_captured_and_replayed(t, e, k):
    """Routing and the layer as a user runs them, captured once on a side
    stream and replayed with other inputs in the same buffers and other live
    counts, with eager calls between: the eager results, bit for bit."""
    h, i = 512, 256
    x, ids, w, w1, w2 = _exact_layer(70, t, e, h, i, k)
    g = _rng(71)
    weights = [up(v) for v in (*w1, *w2)]
    sx, sl, live = up(x), up(g.standard_normal((t, e)).astype(np.float32)), _i32([t])
    out = torch.full((t, h), POISON_BF16, dtype=torch.int16, device=dev())
    n = moe.moe_workspace_bytes(e, h, i, k, t, fmt="mxfp4", weight_fmt="mxfp4")
    ws = torch.empty(n, dtype=torch.uint8, device=dev())
    s_ids = torch.empty((t, k), dtype=torch.int32, device=dev())
    s_w = torch.empty((t, k), dtype=torch.float32, device=dev())

    def step(x_, l_, live_, ids_, w_, out_, ws_):
        moe.moe_route(l_, k, t_live=live_, ids=ids_, weights=w_)
        moe.moe_forward(x_, ids_, w_, *weights, "mxfp4", t_live=live_, out=out_, workspace=ws_, weight_fmt="mxfp4")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(sx, sl, live, s_ids, s_w, out, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(sx, sl, live, s_ids, s_w, out, ws)
    for trial in range(4):
        x2 = up(_exact_layer(72 + trial, t, e, h, i, k)[0])
        l2 = up(g.standard_normal((t, e)).astype(np.float32))
        n_live = [t, max(1, t // 2), 0, t][trial]
        sx.copy_(x2)
        sl.copy_(l2)
        live.fill_(n_live)
        out.fill_(POISON_BF16)
        graph.replay()
        e_out = torch.full((t, h), POISON_BF16, dtype=torch.int16, device=dev())
        e_ids, e_w = torch.empty_like(s_ids), torch.empty_like(s_w)
        step(x2, l2, live, e_ids, e_w, e_out, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(out, e_out), trial
        assert torch.equal(s_ids[:n_live], e_ids[:n_live]) and torch.equal(s_w[:n_live], e_w[:n_live])
        ref = oracle.token_forward_mx4(down(x2), down(e_ids), down(e_w), w1, w2, e, n_live)
        _check_layer(down(out), ref, n_live, k)


def test_layers_on_two_streams_at_once():
    """Calls with workspaces of their own on two streams, unordered, give what
    they give alone (the few-token path keeps nothing between calls)."""
    h, i, e, k = 512, 256, 12, 4
    sets = []
    for s in range(2):
        x, ids, w, w1, w2 = _exact_layer(80 + s, 4, e, h, i, k)
        a = [up(v) for v in (x, ids, w, *w1, *w2)]
        alone = moe.moe_forward(*a, "mxfp4", weight_fmt="mxfp4")[0]
        sets.append((a, alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for _ in range(10):
            for a, alone, stream in sets:
                with torch.cuda.stream(stream):
                    outs.append((moe.moe_forward(*a, "mxfp4", weight_fmt="mxfp4"), alone))
        torch.cuda.synchronize()
        assert all(torch.equal(o[0], alone) for o, alone in outs)


def test_layer_noalloc_gives_the_same_bits():
    x, ids, w, w1, w2 = _exact_layer(90, 6, 10, 256, 128, 3)
    a = [up(v) for v in (x, ids, w, *w1, *w2)]
    want = moe.moe_forward(*a, "mxfp4", weight_fmt="mxfp4")[0]
    assert torch.equal(moe.moe_forward_noalloc(*a, "mxfp4", weight_fmt="mxfp4"), want)


def test_weights_quantized_on_the_gpu_serve_the_layer():
    """moe_act_quant makes an expert's MXFP4 weights from BF16 rows; the layer
    takes them as they are."""
    g = _rng(91)
    e, h, i, t = 3, 256, 128, 5
    wb = [_bf16(0.05 * g.standard_normal((e * r, c))) for r, c in ((2 * i, h), (h, i))]
    packed = [moe.moe_act_quant(up(v), "mxfp4") for v in wb]
    host = [oracle.mxfp4_quantize(oracle.bf16_bits_to_f64(v)) for v in wb]
    for (c, s), (hc, hs) in zip(packed, host):
        assert np.array_equal(down(c), hc) and np.array_equal(down(s), hs)
    x, ids, w, _, _ = _exact_layer(92, t, e, h, i, 2)
    shape = [(e, 2 * i, h), (e, h, i)]
    dw = [v.view(a, b, -1) for (a, b, _), (c, s) in zip(shape, packed) for v in (c, s)]
    out = moe.moe_forward(up(x), up(ids), up(w), *dw, "mxfp4", weight_fmt="mxfp4")[0]
    hw = [v.reshape(a, b, -1) for (a, b, _), (c, s) in zip(shape, host) for v in (c, s)]
    ref = oracle.token_forward_mx4(x, ids, w, (hw[0], hw[1]), (hw[2], hw[3]), e, t)
    got = oracle.bf16_bits_to_f64(down(out))
    # C1 sums are not exact here: a C1 value may fall to the other side of a
    # BF16 tie and, rarely, its quantized code with it; in the 2-norm a tenth
    # of the codes' own step is far beyond that.
    assert np.linalg.norm(got - ref[0]) <= 0.01 * np.linalg.norm(ref[0])


# ---- the ranges' ends ------------------------------------------------------------

@pytest.mark.parametrize("t,k", [(5, 3), (40, 4)])
def test_layer_keeps_a_bad_token_to_itself(t, k):
    """An infinity or a NaN in one token makes that token's output NaN and
    leaves the others' bits as they are without it."""
    x, ids, w, w1, w2 = _exact_layer(90 + t, t, 6, 384, 256, k)
    args = [up(v) for v in (ids, w, *w1, *w2)]
    clean = down(moe.moe_forward(up(x), *args, "mxfp4", weight_fmt="mxfp4")[0])
    bad = x.copy()
    bad[1, 200], bad[t - 1, 7] = 0x7F80, 0x7FC0
    got = down(moe.moe_forward(up(bad), *args, "mxfp4", weight_fmt="mxfp4")[0])
    keep = np.ones(t, bool)
    keep[[1, t - 1]] = False
    assert np.array_equal(got[keep], clean[keep])
    assert np.isnan(oracle.bf16_bits_to_f64(got[~keep])).all()


def _big_weights(experts, n, k, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    w = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device=dev(), generator=g)
    return w, torch.randint(118, 121, (experts, n, k // 32), dtype=torch.uint8, device=dev(), generator=g)


@pytest.mark.parametrize("per", [2, 70])
def test_product_of_weights_past_four_gigabytes(per):
    """The last expert's codes lie past 2^32 bytes; few rows go through the
    streaming kernel, more through LDS."""
    e, n, k = 280, 8192, 4096
    say(f"mx4 gemm of {e} x {n} x {k}, {per} rows")
    w, ws = _big_weights(e, n, k, 5)
    counts = np.zeros(e, np.int32)
    counts[[0, e - 1]] = per
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    a, asc = _mx(_rng(130, per), 2 * per, k)
    out = moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", w, ws, up(counts), up(offsets), 2 * per)
    for x, r in ((0, slice(0, per)), (e - 1, slice(per, 2 * per))):
        wv = oracle.mxfp4_dequant(down(w[x]), down(ws[x]))
        av = oracle.mxfp4_dequant(a[r], asc[r])
        want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
        err = np.abs(oracle.bf16_bits_to_f64(down(out[r])) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + k * 2.0 ** -23 * mag)


def test_layer_of_weights_past_four_gigabytes():
    """Two tokens whose experts are the first and the last of 520: both weight
    tensors are past 2^32 bytes. The same pair of experts alone, as experts 0
    and 1, gives the same bits."""
    e, h, i = 520, 4096, 4096
    w1, w1s = _big_weights(e, 2 * i, h, 6)
    w2, w2s = _big_weights(e, h, i, 7)
    g = _rng(131)
    x = up(_bf16(g.standard_normal((2, h))))
    tw = up(g.random((2, 2)).astype(np.float32))
    got = moe.moe_forward(x, _i32([[0, e - 1], [e - 1, 0]]), tw, w1, w1s, w2, w2s, "mxfp4", weight_fmt="mxfp4")[0]
    two = [v[[0, e - 1]].contiguous() for v in (w1, w1s, w2, w2s)]
    alone = moe.moe_forward(x, _i32([[0, 1], [1, 0]]), tw, *two, "mxfp4", weight_fmt="mxfp4")[0]
    assert torch.equal(got, alone) and down(got).any()


def test_dequantization_past_two_to_the_32_values():
    rows, cols = 1 << 20, 4224
    codes = torch.zeros((rows, cols // 2), dtype=torch.uint8, device=dev())
    scales = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device=dev())
    codes[-1] = 0x72
    codes[rows // 2, 3] = 0x0F
    out = moe.moe_mxfp4_dequant(codes, scales)
    assert out[-1, 0::2].eq(1.0).all() and out[-1, 1::2].eq(6.0).all()
    assert out[rows // 2, 6].item() == -6.0 and not out[:rows // 2].any() and not out[rows // 2 + 1:-1].any()


def test_route_of_rows_past_two_to_the_31_elements():
    t, e, ld = 3000, 40, 800000
    wide = torch.empty((t, ld), dtype=torch.bfloat16, device=dev())
    view = wide[:, 5:5 + e]
    view.copy_(torch.randn((t, e), device=dev()))
    ids, w = moe.moe_route(view, 4)
    ids2, w2 = moe.moe_route(view.contiguous(), 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_calls_on_a_device_that_is_not_current(monkeypatch):
    """With another device current the binding switches to the tensors' (one
    GPU stands in for two: the binding is told that another is current)."""
    from block_fp8_mixture_amd import _binding
    l = torch.randn((3, 40), device=dev())
    ids, w = moe.moe_route(l, 4)
    monkeypatch.setattr(_binding, "_current_device", lambda: -1)
    ids2, w2 = moe.moe_route(l, 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_route_and_layer_follow_the_current_stream():
    """Work enqueued under a side stream stays behind what that stream holds."""
    h, i, e, k, t = 512, 256, 12, 4, 4
    x, _, _, w1, w2 = _exact_layer(95, t, e, h, i, k)
    weights = [up(v) for v in (*w1, *w2)]
    xs, logits = up(x), up(_rng(132).standard_normal((t, e)).astype(np.float32))
    ids, w = moe.moe_route(logits, k)
    want = moe.moe_forward(xs, ids, w, *weights, "mxfp4", weight_fmt="mxfp4")[0]
    side = torch.cuda.Stream()
    late = torch.zeros_like(logits)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            late.zero_()
        late.copy_(logits)
        ids, w = moe.moe_route(late, k)
        got = moe.moe_forward(xs, ids, w, *weights, "mxfp4", weight_fmt="mxfp4")[0]
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("t,k,e,start", [(3, 1, 1, 0), (80, 1, 1, 0), (2, 8, 1024, 0), (12, 4, 1024, 0), (1, 48, 60, 0),
                                         (1, 64, 70, 0), (6, 8, 1030, 6), (7, 3, 5, 4)])
def test_layer_of_one_and_of_many_experts(t, k, e, start):
    say(f"mx4 layer {t} tokens, top {k} of {e} experts from {start}")
    x, ids, w, w1, w2 = _exact_layer(140 + t, t, e, 128, 128, k)
    own = slice(start, e)
    w1, w2 = (w1[0][own], w1[1][own]), (w2[0][own], w2[1][own])
    out = torch.full((t, 128), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_forward(*[up(v) for v in (x, ids, w, *w1, *w2)], "mxfp4", weight_fmt="mxfp4", out=out, expert_start=start)
    ref = oracle.token_forward_mx4(x, ids, w, w1, w2, e - start, t, expert_start=start)
    _check_layer(down(out), ref, t, k)


def test_misaligned_quantization_is_refused():
    """Views one element into a buffer: refused before any launch; scale bytes
    may lie anywhere."""
    x = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device=dev())
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant(x[1:1 + 1024].view(4, 256), "mxfp4")
    codes = torch.zeros(4 * 128 + 4, dtype=torch.uint8, device=dev())
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant(x[:1024].view(4, 256), "mxfp4", xq=codes[1:513].view(4, 128))
    scales = torch.full((33,), POISON_U8, dtype=torch.uint8, device=dev())
    v = up(_bf16(_rng(150).standard_normal((4, 256))))
    xq, xs = moe.moe_act_quant(v, "mxfp4", xs=scales[1:].view(4, 8))
    xq2, xs2 = moe.moe_act_quant(v, "mxfp4")
    assert torch.equal(xq, xq2) and torch.equal(xs, xs2) and scales[0].item() == POISON_U8
