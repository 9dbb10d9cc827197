"""The norm's codes beside those of moe_act_quant(y) where y is not finite: the same
scales, the same codes but for NaN, which is kept."""

import pytest
import torch

import block_fp8_mixture_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
@pytest.mark.parametrize("fmt", ["fp32", "pow2", "ue8m0", "mxfp4"])
def test_codes_of_rows_that_are_not_finite(fmt, rounding):
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    rows, hidden = 6, 640
    x = torch.randn((rows, hidden), generator=g, device="cuda").bfloat16()
    gamma = torch.randn(hidden, generator=g, device="cuda")
    gamma[300], gamma[301] = 3e38, -3e38    # infinite in y where |x| is above 1.1 or so
    x[:, 300], x[:, 301] = 4.0, 0.5
    x[1, 17], x[2, 500], x[3, 3], x[3, 639] = float("nan"), float("inf"), float("-inf"), float("inf")
    x[4] = 0.0
    y, xq, xs, _ = moe.moe_rmsnorm_quant(x, gamma, 0.0 if rounding == "divide" else 1e-6, fmt, rounding=rounding)
    assert y[1].isnan().all() and y[0, 300].isinf() and y[0, 301].isfinite() and y[2, 500].isnan()
    assert bool(y[4].isnan().all()) == (rounding == "divide")  # 0 / 0 without eps
    want_q, want_s = moe.moe_act_quant(y, fmt, rounding=rounding)
    assert torch.equal(xs.view(torch.uint8), want_s.view(torch.uint8))
    if fmt == "mxfp4":
        assert torch.equal(xq, want_q)
        return
    kept = xq.view(torch.float8_e4m3fn).float().isnan()
    assert torch.equal(xq[~kept], want_q[~kept])
    # (a group with an infinity has an infinite scale: its codes stand for no finite value)
    lost = y.isinf().reshape(rows, -1, 128).any(2).repeat_interleave(128, 1)
    assert not bool((kept & y.isfinite() & ~lost).any()) and bool(kept[y.isnan()].all())
