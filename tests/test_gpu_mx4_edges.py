"""What the 4-bit activation operators do at the edges of their documentation.
Expectations are exact (codes, scale bytes, zeros, NaN) or the bounds of
tests/test_gpu_mx4.py."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
import oracle
from block_fp8_mixture_amd import _binding
from tests.gpu_helpers import POISON_BF16, POISON_U8, dev, down, say, up
from tests.test_gpu_mx4 import (ACTS, TILED, _aligned, _bf16, _bf16_any, _check_gemm, _exact_layer, _gemm,
                                _rng)

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


@pytest.mark.parametrize("counts,n", [([3, 20], 256), ([300, 90], 256), (TILED[0], 8192), (TILED[3], 8192)])
def test_rows_whose_map_entry_is_negative_or_past_the_end_are_zero(counts, n):
    """-1 .. -(div - 1) divide to 0 in C; they have no source all the same
    (-1 is how an alignment marks a row without a pair)."""
    say(f"mx4 gemm, negative map entries, {counts} n={n}")
    counts, offsets, row_cap, a, asc, w, ws, row_map = _gemm(counts, n, 512, 1, True, 220)
    live = np.flatnonzero(row_map >= 0)
    bad = {int(live[i]): v for i, v in ((0, -1), (2, -3), (5, -2), (7, -4), (9, -2 ** 31), (-1, -1),
                                        (-2, 4 * len(a)), (-4, 2 ** 31 - 1))}
    for r, v in bad.items():
        row_map[r] = v
    out = torch.full((row_cap, n), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap,
                               a_row_map=up(row_map), a_row_div=4, out=out)
    got = down(out)
    for r in bad:
        assert not (got[r] & 0x7FFF).any(), (r, bad[r])
    for e, c in enumerate(counts):  # the rest of the rows keep theirs
        rows = np.array([r for r in range(offsets[e], offsets[e] + c) if r not in bad], np.int64)
        if len(rows):
            src = row_map[rows] // 4
            av, wv = oracle.mxfp4_dequant(a[src], asc[src]), oracle.mxfp4_dequant(w[e], ws[e])
            want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
            err = np.abs(oracle.bf16_bits_to_f64(got[rows]) - want)
            assert np.all(err <= 2.0 ** -8 * np.abs(want) + 512 * 2.0 ** -23 * mag), e


@pytest.mark.parametrize("counts,align,bounds", [([40, 200, 3, 64], 16, (0, 200, 256, 1024)),
                                                  ([16, 15, 3, 16], 128, (0, 16, 64, 1024))])
def test_product_alone_among_others_and_under_other_bounds(counts, align, bounds):
    """An expert's rows alone, among other experts' and under other host
    bounds: within the bound of the product each time (the order of a row's sum
    follows the launch), and the same bits when the same call is made again.
    Scales 2**50 apart, so that the sums do round."""
    n, k = 8192, 1024
    counts, offsets, _, a, asc, w, ws, _ = _gemm(counts, n, k, align, False, 230)
    g = _rng(231)
    asc, ws = (g.integers(100, 150, v.shape).astype(np.uint8) for v in (asc, ws))
    dw, dws = up(w), up(ws)
    calls = [(slice(0, 4), b) for b in bounds]
    calls += [(slice(e, e + 1), b) for e in range(4) for b in (0, int(counts[e]))]
    for own, bound in calls:
        say(f"mx4 gemm of experts {own.start}..{own.stop - 1} under bound {bound}")
        c, first = counts[own], int(offsets[own.start])
        o = offsets[own.start:own.stop + 1] - np.int32(first)
        cap = int(o[-1])
        av, asv = a[first:first + cap], asc[first:first + cap]
        bits = []
        for _ in range(2):
            out = torch.full((cap, n), POISON_BF16, dtype=torch.int16, device=dev())
            moe.moe_grouped_gemm_mxfp4(up(av), up(asv), "mxfp4", dw[own], dws[own], up(c), up(o), cap,
                                       max_rows_per_expert=bound, out=out)
            bits.append(out)
        assert torch.equal(*bits)
        _check_gemm(bits[0], c, o, av, asv, w[own], ws[own], None, k)


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


@pytest.mark.parametrize("tokens,experts,topk,kw", [
    ((1 << 28) + 48, 2, 1, {}),  # 16 lanes per token
    ((1 << 26) + 12, 17, 1, dict(num_groups=17, top_groups=17, renormalize=False)),  # 64
])
def test_route_past_two_to_the_32_threads(tokens, experts, topk, kw):
    """More lanes than one dimension of a grid holds: every token is routed,
    and none past the last."""
    say(f"route of {tokens} tokens, {experts} experts")
    l = torch.zeros((tokens, experts), dtype=torch.bfloat16, device=dev())
    # The picked expert and its logit vary along the tokens.
    t = torch.arange(tokens, device=dev())
    pick = (t * 40503 >> 7) % experts
    l.scatter_(1, pick[:, None], 1.0)
    l[0::5] *= 2
    del t
    ids = torch.full((tokens + 8, topk), -9, dtype=torch.int32, device=dev())
    w = torch.full((tokens + 8, topk), -9.0, device=dev())
    moe.moe_route(l, topk, ids=ids[:tokens], weights=w[:tokens], **kw)
    assert torch.equal(ids[:tokens, 0], pick.int())
    best = torch.where(torch.arange(tokens, device=dev()) % 5 == 0, 2.0, 1.0)
    want = 1.0 if kw == {} else None  # a renormalized single pick weighs one
    if want is None:
        two, one = (np.exp(v) / (np.exp(v) + experts - 1) for v in (2.0, 1.0))
        want = torch.where(best == 2.0, two, one).float()
    # A double rounded once, on both sides of the double's own error.
    assert (w[:tokens, 0] - want).abs().max().item() <= 2.0 ** -24
    assert ids[tokens:].eq(-9).all() and w[tokens:].eq(-9.0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "ue8m0"])
def test_quantization_past_two_to_the_32_threads(fmt):
    """2^28 groups of 128 and a few rows more (64 GiB of BF16, as a tensor of
    weights quantized at once may be): the first and last rows and the bytes
    about the 2^32-thread border are those of a short call."""
    cols, rows = 1 << 15, (1 << 20) + 3
    say(f"quantization of {rows} x {cols} {fmt}")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev())
    probe = [0, 1, 4097, (1 << 19) + 5, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, rows - 1]
    g = torch.Generator(device=dev()).manual_seed(9)
    part = torch.randn((len(probe), cols), generator=g, device=dev()).bfloat16()
    x[probe] = part
    want_q, want_s = moe.moe_act_quant(part, fmt)
    xq, xs = moe.moe_act_quant(x, fmt, xq=torch.full((rows, want_q.shape[1]), POISON_U8, dtype=torch.uint8, device=dev()))
    assert torch.equal(xq[probe], want_q)
    assert torch.equal(xs[probe] if fmt == "mxfp4" else xs[:, probe], want_s)
    rest = torch.ones(rows, dtype=torch.bool, device=dev())
    rest[probe] = False
    for lo in range(0, rows, 1 << 17):  # zeros everywhere else
        assert not xq[lo:lo + (1 << 17)][rest[lo:lo + (1 << 17)]].any(), lo
    del x, xq, xs
    torch.cuda.empty_cache()


def test_combine_past_two_to_the_32_threads():
    """2^25 workgroups of 128 threads and a few more, as the last step of a
    layer of that many tokens: every token has its row, rows behind the last stay."""
    tokens, hidden, rows = (1 << 25) + 21, 128, 1000
    say(f"combine of {tokens} tokens of {hidden}")
    y = torch.randn((rows, hidden), device=dev()).bfloat16()
    pair_to_row = ((torch.arange(tokens, device=dev()) * 40503 >> 3) % (rows + 1) - 1).int()  # -1: none
    w = torch.ones((tokens, 1), device=dev())
    out = torch.full((tokens + 4, hidden), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_topk_combine(y, pair_to_row, w, out=out[:tokens])
    want = torch.cat([y.view(torch.int16), torch.zeros((1, hidden), dtype=torch.int16, device=dev())])
    for lo in range(0, tokens, 1 << 22):
        assert torch.equal(out[lo:min(lo + (1 << 22), tokens)], want[pair_to_row[lo:lo + (1 << 22)].long()]), lo
    assert out[tokens:].eq(POISON_BF16).all()


def test_every_entry_point_is_given_the_current_stream(monkeypatch):
    """The handle each call passes to the library, under a side stream and
    outside it."""
    handles = {}

    class Library:
        def __getattr__(self, name):
            fn = getattr(real, name)

            def call(*args):
                handles[name] = args[-1]
                return fn(*args)
            return call

    real = moe.load_library()
    monkeypatch.setattr(_binding, "_lib", Library())
    e, h, i, k, t = 3, 256, 128, 2, 5
    x, _, _, w1, w2 = _exact_layer(250, t, e, h, i, k)
    xs, weights = up(x), [up(v) for v in (*w1, *w2)]
    logits = torch.randn((t, e), device=dev())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls():
        ids, tw = moe.moe_route(logits, k)
        al = moe.moe_align(ids, e)
        xq, sc = moe.moe_act_quant(xs, "mxfp4")
        moe.moe_mxfp4_dequant(xq, sc)
        rows = al["row_to_pair"].numel()
        c1 = moe.moe_grouped_gemm_mxfp4(xq, sc, "mxfp4", *weights[:2], al["counts"], al["offsets"], rows,
                                        a_row_map=al["row_to_pair"], a_row_div=k)
        hq, hs = moe.moe_silu_mul_quant(c1, al["counts"], al["offsets"], fmt="mxfp4")
        y = moe.moe_grouped_gemm_mxfp4(hq, hs, "mxfp4", *weights[2:], al["counts"], al["offsets"], rows)
        out = moe.moe_topk_combine(y, al["pair_to_row"], tw)
        full = moe.moe_forward(xs, ids, tw, *weights, "mxfp4", weight_fmt="mxfp4")[0]
        moe.moe_forward_noalloc(xs, ids, tw, *weights, "mxfp4", weight_fmt="mxfp4")
        al2 = moe.moe_align_batched(ids, e, t)
        moe.moe_silu_mul_quant_masked(torch.zeros((e * t, 2 * i), dtype=torch.bfloat16, device=dev()), al2["masked_m"], t,
                                      fmt="mxfp4")
        return out, full

    names = {"moe_route", "moe_align", "moe_align_batched", "moe_act_quant", "moe_mxfp4_dequant",
             "moe_grouped_gemm_mxfp4", "moe_silu_mul_quant", "moe_silu_mul_quant_masked", "moe_topk_combine",
             "moe_forward", "moe_forward_noalloc"}
    with torch.cuda.stream(side):
        a = calls()
    side.synchronize()
    assert {n: handles[n] for n in names} == dict.fromkeys(names, side.cuda_stream)
    handles.clear()
    b = calls()
    torch.cuda.synchronize()
    assert {n: handles[n] for n in names} == dict.fromkeys(names, torch.cuda.current_stream().cuda_stream)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("t,h", [(16, 15360), (48, 128)])
def test_few_token_layer_captured_at_its_limits(t, h):
    """The most tokens, and the most LDS a workgroup of theirs takes (128 KB of
    codes): every replay as the eager call, with other work between."""
    say(f"mx4 layer of {t} x {h}, captured")
    x, ids, w, w1, w2 = _exact_layer(260 + t, t, 5, h, 128, 1)
    args = [up(v) for v in (ids, w, *w1, *w2)]
    xs, out = up(x), torch.empty((t, h), dtype=torch.int16, device=dev())
    ws = torch.empty(moe.moe_workspace_bytes(5, h, 128, 1, t, fmt="mxfp4", weight_fmt="mxfp4"), dtype=torch.uint8,
                     device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        moe.moe_forward(xs, *args, "mxfp4", weight_fmt="mxfp4", out=out, workspace=ws)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_forward(xs, *args, "mxfp4", weight_fmt="mxfp4", out=out, workspace=ws)
    for trial in range(3):
        xs.copy_(up(x).roll(trial, 0))
        out.fill_(POISON_BF16)
        graph.replay()
        eager = moe.moe_forward(up(x).roll(trial, 0), *args, "mxfp4", weight_fmt="mxfp4")[0]
        torch.cuda.synchronize()
        assert torch.equal(out, eager), trial


@pytest.mark.parametrize("counts,n,k", [([3, 40], 128, 32640), ([300], 128, 32768), ([1], 1 << 20, 128),
                                        ([70], 1 << 18, 256)])
def test_product_of_the_longest_rows_and_the_most_columns(counts, n, k):
    """K up to 32768, past which a call is refused, and N far past K."""
    say(f"mx4 gemm {counts} n={n} k={k}")
    counts, offsets, row_cap, a, asc, w, ws, _ = _gemm(counts, n, k, 16, False, 270)
    out = torch.full((row_cap, n), POISON_BF16, dtype=torch.int16, device=dev())
    moe.moe_grouped_gemm_mxfp4(up(a), up(asc), "mxfp4", up(w), up(ws), up(counts), up(offsets), row_cap, out=out)
    _check_gemm(out, counts, offsets, a, asc, w, ws, None, k)
