"""moe_rmsnorm_quant on the GPU against the fp64 oracle, bit for bit.

The mean, the root and the products are in 64 bits on both sides, rounded to
float32 and to BF16: the sides may differ where the 64-bit value is within a few
2**-52 of a float32 rounding border, one value in some 2**26; the inputs here
(seeded, under 2**22 values) hold none. Codes and scales are those of the y that
was returned, by the oracle's quantizers and by moe_act_quant."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
import oracle
import synth
from tests.gpu_helpers import (POISON_BF16, POISON_U8, assert_bf16_close, dev, device_weights, down,
                               host_weights, say, up)

pytestmark = pytest.mark.gpu

FMTS = [None, "fp32", "pow2", "ue8m0", "mxfp4"]


def _rng(*key):
    return np.random.default_rng([int(k) for k in key])


def _bits(g, rows, cols, scale=1.0):
    return oracle.bf16_from_f64(scale * g.standard_normal((rows, cols)))


def _poison(rows, hidden, fmt):
    xq = xs = None
    if fmt is not None:
        cols = hidden // 2 if fmt == "mxfp4" else hidden
        xq = torch.full((rows, cols), POISON_U8, dtype=torch.uint8, device=dev())
        shape = (rows, hidden // 32) if fmt == "mxfp4" else (hidden // 128, rows)
        kind = torch.uint8 if fmt in ("ue8m0", "mxfp4") else torch.float32
        xs = torch.full(shape, POISON_U8, dtype=kind, device=dev())
    return xq, xs


def _codes(y_bits, fmt, rounding="divide"):
    v = oracle.bf16_bits_to_f64(y_bits)
    if fmt == "mxfp4":
        return oracle.mxfp4_quantize(v)
    return oracle.quantize_groups(v.astype(np.float32), fmt, rounding)


def _check(x, w, r=None, eps=1e-6, fmt=None, live=None, rounding="divide", dx=None):
    rows, hidden = x.shape
    n = rows if live is None else live
    weight = up(w) if w.dtype == np.float32 else up(w)
    wv = w.astype(np.float64) if w.dtype == np.float32 else oracle.bf16_bits_to_f64(w)
    if w.dtype != np.float32:
        weight = weight.view(torch.bfloat16)
    y = torch.full((rows, hidden), POISON_BF16, dtype=torch.int16, device=dev())
    h = None if r is None else torch.full_like(y, POISON_BF16)
    xq, xs = _poison(rows, hidden, fmt)
    t_live = None if live is None else up(np.array([live], np.int32))
    got = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16) if dx is None else dx, weight, eps, fmt,
                                residual=None if r is None else up(r), t_live=t_live, residual_out=h, y=y,
                                xq=xq, xs=xs, rounding=rounding)
    assert got[0] is y and got[1] is xq and got[2] is xs and got[3] is h
    want_h, want_y = oracle.rmsnorm(x[:n], wv, eps, None if r is None else r[:n])
    assert np.array_equal(down(y)[:n], want_y)
    assert (down(y)[n:] == POISON_BF16).all()
    if r is not None:
        assert np.array_equal(down(h)[:n], want_h) and (down(h)[n:] == POISON_BF16).all()
    if fmt is not None:
        codes, scales = _codes(want_y, fmt, rounding)
        assert np.array_equal(down(xq)[:n], codes) and (down(xq)[n:] == POISON_U8).all()
        s = down(xs) if fmt == "mxfp4" else down(xs).T
        assert np.array_equal(s[:n], scales if fmt == "mxfp4" else scales.T) and (s[n:] == POISON_U8).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hidden", [128, 512, 640, 2048, 2176, 4096, 6144, 7168, 8320, 16384, 16512, 32768])
def test_norm_matches_oracle(hidden, fmt):
    g = _rng(300, hidden)
    for rows, residual, f32 in ((1, True, False), (3, False, True), (18, True, True)):
        say(f"norm {rows} x {hidden} {fmt} residual={residual} f32={f32}")
        x = _bits(g, rows, hidden, 2.0)
        r = _bits(g, rows, hidden, 5.0) if residual else None
        w = 1 + 0.3 * g.standard_normal(hidden)
        _check(x, w.astype(np.float32) if f32 else oracle.bf16_from_f64(w), r, fmt=fmt)


@pytest.mark.parametrize("fmt", FMTS[1:])
@pytest.mark.parametrize("rounding", ["divide", "reciprocal"])
def test_codes_are_those_of_the_two_passes(rounding, fmt):
    g = _rng(301)
    x, r = _bits(g, 37, 1024), _bits(g, 37, 1024)
    x[5] = 0
    r[5] = 0
    w = oracle.bf16_from_f64(1 + 0.1 * g.standard_normal(1024))
    _check(x, w, r, fmt=fmt, rounding=rounding)
    y, xq, xs, h = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16), up(w).view(torch.bfloat16), 1e-5, fmt,
                                         residual=up(r), rounding=rounding)
    assert torch.equal(h, up(x).view(torch.bfloat16) + up(r).view(torch.bfloat16))
    q, s = moe.moe_act_quant(y, fmt, rounding=rounding)
    assert torch.equal(q, xq) and torch.equal(s, xs)
    none, xq2, xs2, _ = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16), up(w).view(torch.bfloat16), 1e-5, fmt,
                                              residual=up(r), rounding=rounding, y=False)
    assert none is None and torch.equal(xq2, xq) and torch.equal(xs2, xs)


@pytest.mark.parametrize("fmt", ["fp32", "mxfp4"])
@pytest.mark.parametrize("live", [0, 1, 6, 7])
def test_rows_past_the_live_count_stay(live, fmt):
    g = _rng(302, live)
    w = np.ones(384, np.float32)
    _check(_bits(g, 7, 384), w, _bits(g, 7, 384), fmt=fmt, live=live)
    # The count is clamped to the capacity.
    x = _bits(g, 7, 384)
    y = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16), up(w), fmt=None,
                              t_live=up(np.array([99], np.int32)))[0]
    assert np.array_equal(down(y.view(torch.int16)), oracle.rmsnorm(x, w.astype(np.float64), 1e-6)[1])


def test_no_rows():
    y, xq, xs, h = moe.moe_rmsnorm_quant(torch.empty((0, 256), dtype=torch.bfloat16, device=dev()),
                                         torch.ones(256, device=dev()), fmt="fp32")
    assert y.shape == (0, 256) and xq.shape == (0, 256) and xs.shape == (2, 0) and h is None


def test_strided_rows():
    g = _rng(303)
    wide = _bits(g, 9, 1024 + 256 + 8)
    d = up(wide).view(torch.bfloat16)
    w = np.float32(1 + 0.1 * g.standard_normal(256))
    for at in (0, 8, 1024):
        _check(np.ascontiguousarray(wide[:, at:at + 256]), w, _bits(g, 9, 256), fmt="ue8m0",
               dx=d[:, at:at + 256])
    with pytest.raises(moe.MoeError, match="invalid"):  # a start off 16 bytes
        moe.moe_rmsnorm_quant(d[:, 4:260], up(w))
    with pytest.raises(moe.MoeError, match="invalid"):  # rows off 16 bytes
        moe.moe_rmsnorm_quant(torch.zeros((4, 260), dtype=torch.bfloat16, device=dev())[:, :256], up(w))


def test_in_place():
    g = _rng(304)
    x, r, w = _bits(g, 20, 896), _bits(g, 20, 896), np.ones(896, np.float32)
    h, y = oracle.rmsnorm(x, w.astype(np.float64), 1e-6, r)
    for where in ("residual", "x", "y in x", "y in residual"):
        dx, dr = up(x).view(torch.bfloat16), up(r).view(torch.bfloat16)
        kw = {"residual": dict(residual_out=dr), "x": dict(residual_out=dx),
              "y in x": dict(residual_out=dr, y=dx), "y in residual": dict(residual_out=dx, y=dr)}[where]
        gy, _, _, gh = moe.moe_rmsnorm_quant(dx, up(w), residual=dr, **kw)
        assert np.array_equal(down(gh.view(torch.int16)), h), where
        assert np.array_equal(down(gy.view(torch.int16)), y), where
    dx = up(x).view(torch.bfloat16)
    gy = moe.moe_rmsnorm_quant(dx, up(w), fmt=None, y=dx)[0]
    assert np.array_equal(down(gy.view(torch.int16)), oracle.rmsnorm(x, w.astype(np.float64), 1e-6)[1])


def test_rows_that_are_not_ordinary():
    """Zeros, subnormals, the largest values, and a residual that cancels."""
    g = _rng(305)
    x, r = _bits(g, 6, 256), _bits(g, 6, 256)
    x[0] = r[0] = 0
    x[1] = g.integers(1, 0x80, 256)  # BF16 subnormals
    r[1] = 0
    x[2] = np.where(g.integers(0, 2, 256), 0x7F00, 0xFF00)  # +-2^127
    r[2] = 0
    r[3] = x[3] ^ 0x8000
    w = np.float32(1 + 0.1 * g.standard_normal(256))
    for fmt in FMTS:
        _check(x, w, r, fmt=fmt)
    for eps in (1e-5, 1e-12, 0.25):
        _check(x, w, r, eps=eps, fmt="fp32")
    _check(x[4:], w, r[4:], eps=0.0, fmt="fp32")


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_and_infinity_reach_the_outputs(fmt):
    g = _rng(306)
    x = _bits(g, 4, 512)
    x[1, 200] = 0x7FC0  # NaN
    x[2, 77] = 0xFF80   # -infinity
    w = np.ones(512, np.float32)
    y, xq, xs, _ = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16), up(w), 1e-6, fmt)
    yv = y.double().cpu().numpy()
    assert np.isnan(yv[1]).all() and np.isnan(yv[2, 77]) and (np.delete(yv[2], 77) == 0).all()
    assert np.isfinite(yv[[0, 3]]).all()
    if fmt == "mxfp4":
        s = down(xs)
        assert (s[1] == 255).all() and s[2, 77 // 32] == 255 and (s[[0, 3]] < 255).all()
    elif fmt is not None:
        q = oracle.e4m3_decode(down(xq))
        assert np.isnan(q[1]).all() and np.isnan(q[2, 77]) and np.isfinite(np.delete(q[2], 77)).all()
        assert np.isfinite(q[[0, 3]]).all()


def test_captured_and_replayed_beside_eager_calls():
    g = _rng(307)
    rows, hidden = 12, 4096
    x, r = up(_bits(g, rows, hidden)).view(torch.bfloat16), up(_bits(g, rows, hidden)).view(torch.bfloat16)
    w = torch.ones(hidden, device=dev())
    live = up(np.array([rows], np.int32))
    y, h = torch.zeros_like(x), torch.zeros_like(x)
    xq, xs = torch.zeros((rows, hidden), dtype=torch.uint8, device=dev()), torch.zeros((32, rows), device=dev())
    moe.moe_rmsnorm_quant(x, w, residual=r, residual_out=h, y=y, xq=xq, xs=xs, t_live=live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_rmsnorm_quant(x, w, residual=r, residual_out=h, y=y, xq=xq, xs=xs, t_live=live)
    for i, n in enumerate((rows, 5, 0, rows)):
        x.copy_(up(_bits(g, rows, hidden)).view(torch.bfloat16))
        live.fill_(n)
        for t in (y, h, xq, xs):
            t.zero_()
        graph.replay()
        want = moe.moe_rmsnorm_quant(x, w, residual=r)
        torch.cuda.synchronize()
        for a, b in zip((y, xq, h), (want[0], want[1], want[3])):
            assert torch.equal(a[:n], b[:n]) and not a[n:].any(), i
        assert torch.equal(xs[:, :n], want[2][:, :n]) and not xs[:, n:].any()


def test_on_a_stream_of_its_own():
    g = _rng(308)
    x = up(_bits(g, 64, 2048)).view(torch.bfloat16)
    w = torch.ones(2048, device=dev())
    want = moe.moe_rmsnorm_quant(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.moe_rmsnorm_quant(x, w)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))


def test_feeds_the_layer():
    """The staged layer on the norm's codes is the layer on its BF16 output."""
    cfg = synth.get("tiny")
    x, ids, tw = synth.make_workload(cfg, 8)
    w1q, w1s, w2q, w2s = device_weights("tiny")
    e, inter, hidden = cfg.num_experts, cfg.inter, cfg.hidden
    gamma = torch.ones(hidden, device=dev())
    for fmt in ("fp32", "ue8m0"):
        y, xq, xs, _ = moe.moe_rmsnorm_quant(up(x).view(torch.bfloat16), gamma, fmt=fmt, residual=up(x))
        al = moe.moe_align(up(ids), e, cfg.align_rows, cfg.row_cap)
        c1 = moe.moe_grouped_gemm_fp8(xq, xs, fmt, w1q, w1s, al["counts"], al["offsets"], cfg.row_cap,
                                      a_row_map=al["row_to_pair"], a_row_div=cfg.topk)
        hq, hs = moe.moe_silu_mul_quant(c1, al["counts"], al["offsets"], fmt=fmt)
        c2 = moe.moe_grouped_gemm_fp8(hq, hs, fmt, w2q, w2s, al["counts"], al["offsets"], cfg.row_cap)
        out = moe.moe_topk_combine(c2, al["pair_to_row"], up(tw))
        q2, s2 = moe.moe_act_quant(y, fmt)
        assert torch.equal(q2, xq) and torch.equal(s2, xs)
        c1b = moe.moe_grouped_gemm_fp8(q2, s2, fmt, w1q, w1s, al["counts"], al["offsets"], cfg.row_cap,
                                       a_row_map=al["row_to_pair"], a_row_div=cfg.topk)
        live = al["row_to_pair"][:int(al["offsets"][-1])] >= 0
        assert torch.equal(c1[:live.numel()][live], c1b[:live.numel()][live])
        ref = oracle.forward(down(y.view(torch.int16)), ids, tw, *host_weights("tiny"), 8, cfg.align_rows, fmt)
        assert_bf16_close(down(out), ref["out"], "layer after the norm")

