"""What the 4-bit activation operators do at the edges of their documentation.
Expectations are exact (codes, scale bytes, zeros, NaN) or the bounds of
tests/test_gpu_mx4.py."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
import oracle
from tests.gpu_helpers import POISON_U8, dev, down, say, up
from tests.test_gpu_mx4 import ACTS, _aligned, _bf16, _bf16_any, _exact_layer, _rng

pytestmark = pytest.mark.gpu


def _quantized(gu_bits, inter, act, lim, rounding):
    """Codes and scale bytes of SiLU(gate) * up, NaN and infinities included."""
    v = oracle.bf16_bits_to_f64(gu_bits)
    with np.errstate(all="ignore"):
        y = oracle.swiglu(v[:, :inter], v[:, inter:], act, lim)
    if rounding == "reciprocal":
        y = oracle.bf16_bits_to_f64(_bf16_any(y))
    return oracle.mxfp4_quantize(y)


# Block: what is planted in its gate and in its up.
PLANTED = [(np.nan, None), (None, np.nan), (np.nan, np.nan), (np.inf, None), (-np.inf, None), (None, np.inf),
           (None, -np.inf), (np.inf, 0.0), (-np.nan, 2.0), (100.0, -np.nan), (np.inf, np.nan)]


@pytest.mark.parametrize("act,lim", ACTS)
@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
@pytest.mark.parametrize("rows,inter", [(1, 384), (5, 384), (2048, 4096)])
def test_silu_quantization_keeps_nan_and_infinities(rows, inter, rounding, act, lim):
    """One bad value per block, in SiLU by formula (few rows) and by table
    (2048 rows of 4096 are 65536 groups of 128, 128 for each of 512 workgroups)."""
    say(f"silu with NaN, {rows} x {inter} {rounding} {act}")
    g = _rng(200, rows, inter)
    gu = g.standard_normal((rows, 2 * inter)).astype(np.float32)
    planted = sorted({0, rows // 2, rows - 1})
    for r in planted:
        for b, (gate, upv) in enumerate(PLANTED):
            at = 32 * b + (7 * b + r) % 32
            if gate is not None:
                gu[r, at] = gate
            if upv is not None:
                gu[r, inter + at] = upv
    gu = _bf16_any(gu)
    counts, offsets = _aligned([rows], 1)
    hq, hs = moe.moe_silu_mul_quant(up(gu), up(counts), up(offsets), act, lim, "mxfp4", rounding=rounding)
    mq, ms = moe.moe_silu_mul_quant_masked(up(gu), up(counts), rows, act, lim, "mxfp4", rounding=rounding)
    codes, scales = _quantized(gu[planted], inter, act, lim, rounding)
    # A NaN, whatever the clamp; the others as the formula has them.
    assert np.all(scales[:, [0, 1, 2, 8, 9, 10]] == 255)
    for q, s in ((hq, hs), (mq, ms)):
        assert np.array_equal(down(s)[planted], scales) and np.array_equal(down(q)[planted], codes)


@pytest.mark.parametrize("act,lim", ACTS)
@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
@pytest.mark.parametrize("t,k,cap", [(1, 8, 0), (5, 3, 0), (40, 4, 0), (40, 4, 40)])
def test_layer_keeps_a_bad_token_to_itself_under_every_activation(t, k, cap, rounding, act, lim):
    """An infinity or a NaN in one token makes that token's output NaN and
    leaves the others' bits as they are without it: the few-token layer, the
    general path and the batched layout."""
    say(f"mx4 layer with bad tokens, t={t} k={k} cap={cap} {rounding} {act}")
    x, ids, w, w1, w2 = _exact_layer(210 + t, t, 9, 384, 256, k)
    args = [up(v) for v in (ids, w, *w1, *w2)]
    kw = dict(act=act, clamp_limit=lim, rounding=rounding, expert_cap=cap, weight_fmt="mxfp4")
    clean = down(moe.moe_forward(up(x), *args, "mxfp4", **kw)[0])
    bad = x.copy()
    bad[t // 2, 200], bad[t - 1, 7] = 0xFF80, 0x7FC0
    got = down(moe.moe_forward(up(bad), *args, "mxfp4", **kw)[0])
    keep = np.ones(t, bool)
    keep[[t // 2, t - 1]] = False
    assert np.array_equal(got[keep], clean[keep])
    assert np.isnan(oracle.bf16_bits_to_f64(got[~keep])).all()


@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
def test_silu_quantization_of_subnormal_products(rounding):
    """Products down to float32's smallest: blocks of scale byte 0 and around."""
    g = _rng(240)
    rows, inter = 40, 256
    gate = np.exp2(-g.integers(60, 100, (rows, inter // 32))).repeat(32, 1) * g.uniform(1, 2, (rows, inter))
    upv = np.exp2(-g.integers(20, 52, (rows, inter // 32))).repeat(32, 1) * g.standard_normal((rows, inter))
    gu = _bf16(np.concatenate([gate, upv], 1))
    counts, offsets = _aligned([rows], 1)
    hq = torch.full((rows, inter // 2), POISON_U8, dtype=torch.uint8, device=dev())
    hq, hs = moe.moe_silu_mul_quant(up(gu), up(counts), up(offsets), fmt="mxfp4", rounding=rounding, hq=hq)
    codes, scales = _quantized(gu, inter, "swiglu", np.inf, rounding)
    assert (scales == 0).any() and (scales > 0).any()
    assert np.array_equal(down(hs), scales) and np.array_equal(down(hq), codes)
