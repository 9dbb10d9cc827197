"""4-bit integer products of many rows, per expert too, on shapes that reach every
form: sums that are exact in fp32 in any order, so that a plain product is compared
bit for bit, whatever kernel and tile computes it.

Rows of A hold -1, 0 and 1, weights s (q - z) with scales of full mantissas (BF16: 128
.. 255, FP16: 1024 .. 2047, times a power of two) and either sign. A sum of K <= 1024
such terms, |q - z| <= 15, has a standard deviation below 32 * 15 * 2 scales, so all
partial sums are far below 2**13 of them, and multiples of a scale's last bit: 13 + 10
bits. (A weight rounded to BF16 is off by up to 2**-9 of itself, and sums of such
weights show it.) Gated, the sums are exact, and SiLU's exponential, quotient and
product take 2**-19 of the result, the output's rounding 2**-8.

Which kernel a shape takes is seen from outside: a group's sum is a difference in the
streamed form, so an infinity in a row makes all of the row NaN there; in tiles it
stays an infinity where the weight is not zero."""

import numpy as np
import pytest
import torch

import block_fp8_mixture_amd as moe
from tests.gpu_helpers import POISON_BF16, dev, say

pytestmark = pytest.mark.gpu

ACTS = ["swiglu", "swiglu_clamp", "swiglu_clamp_after_silu"]
LIM = 1.5
UNIT = 2.0 ** -7  # of the scales: sums of a few units


def _gen(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(np.random.SeedSequence([int(k) for k in key]).generate_state(1)[0]))
    return g


def _rand(g, lo, hi, shape, dtype):
    return torch.randint(lo, hi, shape, generator=g, device="cuda").to(dtype)


def _rows(g, m, k):
    return _rand(g, -1, 2, (m, k), torch.bfloat16)


def _weights(g, lead, n, k, group, zeros, kind):
    codes = _rand(g, 0, 256, lead + (n, k // 2), torch.uint8)
    one = 128 if kind == torch.bfloat16 else 1024
    s = _rand(g, one, 2 * one, lead + (n, k // group), torch.float32) * (UNIT / one)
    s = s * (1 - 2 * _rand(g, 0, 2, s.shape, torch.float32))
    z = _rand(g, 0, 16, lead + (n, k // group), torch.uint8) if zeros else None
    return codes, s.to(kind), z


def _values(codes, s, z):
    """float64 [n, k] of one matrix."""
    q = torch.stack([codes & 15, codes >> 4], -1).double().reshape(s.shape + (-1,))
    zero = 8.0 if z is None else z.double()[..., None]
    return ((q - zero) * s.double()[..., None]).reshape(codes.shape[0], -1)


def _act(c, act):
    if act is None:
        return c
    g, u = c.chunk(2, 1)
    if act == "swiglu_clamp":
        g = g.clamp(max=LIM)
    g = g / (1 + torch.exp(-g))
    if act == "swiglu_clamp_after_silu":
        g = g.clamp(max=LIM)
    return g * (u if act == "swiglu" else u.clamp(-LIM, LIM))


def _compare(out, sums, act, what):
    """out BF16 of the exact sums."""
    ref = _act(sums, act)
    if act is None:
        ok = out.double() == ref.float().bfloat16().double()
    else:
        ok = (out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -19) * ref.abs()
    assert bool(ok.all()), (what, int((~ok).sum()), (~ok).nonzero()[:3].tolist(), out[~ok][:3], ref[~ok][:3])


def _poison(m, n):
    return torch.full((m, n), POISON_BF16, dtype=torch.int16, device="cuda").view(torch.bfloat16)


def _untouched(t):
    assert bool((t.view(torch.int16) == POISON_BF16).all())


def _linear(g, rows, k, n, group, zeros, kind, act, live=None, tiles=None):
    a = _rows(g, rows, k)
    codes, s, z = _weights(g, (), n, k, group, zeros, kind)
    out = _poison(rows, n if act is None else n // 2)
    t_live = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    moe.moe_gemm_int4(a, codes, s, z, act=act, clamp_limit=LIM, t_live=t_live, out=out)
    m = rows if live is None else live
    _compare(out[:m], a[:m].double() @ _values(codes, s, z).t(), act, (rows, k, n, group, zeros, kind, act, live))
    _untouched(out[m:])
    if tiles is not None and m > 64:
        a[m - 1, k - 1] = float("inf")
        assert bool(moe.moe_gemm_int4(a, codes, s, z, t_live=t_live)[m - 1].isinf().any()) == tiles


LINEAR = [
    # rows, k, n, whether in tiles
    (64, 832, 1000, False), (66, 544, 1000, False),
    (300, 832, 4096, True), (257, 352, 7170, True), (2048, 608, 4098, True),   # of 64 rows
    (700, 992, 8192, True), (1030, 800, 6150, True), (2048, 352, 16384, True),  # of 128 rows
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,k,n,tiles", LINEAR)
def test_linear_sums_are_exact(rows, k, n, tiles, group):
    k = k // group * group
    for i in range(4):
        kind = (torch.bfloat16, torch.float16)[i % 2]
        say(f"int4 linear {rows} x {k} -> {n} group {group} {kind} zeros {i >= 2}")
        g = _gen(500, rows, k, n, group, i)
        _linear(g, rows, k, n, group, i >= 2, kind, None, tiles=tiles)
        _linear(g, rows, k, n + n % 2, group, i % 2 == 1, kind, ACTS[(i + rows) % 3])


@pytest.mark.parametrize("live", [0, 1, 16, 17, 64, 65, 128, 699])
def test_live_rows_of_many(live):
    """The device's count decides between the launches for few rows and the tiles."""
    for i, group in enumerate((32, 64, 128)):
        _linear(_gen(501, live, i), 700, 384, 4096, group, i == 0, torch.bfloat16, None, live=live)
        _linear(_gen(502, live, i), 700, 384, 4096, group, i == 1, torch.float16, ACTS[i], live=live)


def _grouped(g, counts, k, n, group, zeros, kind, act=None, align=16, cap=0, gather=0, bound=0, slack=0, tiles=None):
    e = len(counts)
    if cap:
        ends, row_cap = [x * cap for x in range(e + 1)], e * cap
    else:
        ends = [0] + np.cumsum([(c + align - 1) // align * align for c in counts]).tolist()
        row_cap = ends[-1] + slack
    codes, s, z = _weights(g, (e,), n, k, group, zeros, kind)
    a = _rows(g, max(3, row_cap // 2) if gather else row_cap, k)
    src = torch.arange(row_cap, device="cuda")
    row_map = None
    if gather:
        row_map = _rand(g, 0, a.shape[0] * gather, (row_cap,), torch.int32)
        # every seventh row without a source: negative, past the end
        row_map[::28], row_map[7::28], row_map[14::28], row_map[21::28] = -1, -gather, a.shape[0] * gather, 2 ** 31 - 1
        src = torch.where(row_map >= 0, row_map.long() // gather, -1)
        src = torch.where(src < a.shape[0], src, -1)
    out = _poison(row_cap, n if act is None else n // 2)

    def run(x, to, how):
        return moe.moe_grouped_gemm_int4(
            x, codes, s, torch.tensor(counts, dtype=torch.int32, device="cuda"),
            None if cap else torch.tensor(ends, dtype=torch.int32, device="cuda"), row_cap, w_zeros=z, a_row_map=row_map,
            a_row_div=max(gather, 1), expert_cap=cap, max_rows_per_expert=bound, act=how, clamp_limit=LIM, out=to)
    run(a, out, act)
    live = torch.zeros(row_cap, dtype=torch.bool, device="cuda")
    for x in range(e):
        m = min(counts[x], ends[x + 1] - ends[x])
        if not m:
            continue
        at = slice(ends[x], ends[x] + m)
        live[at] = True
        rows = torch.where((src[at] >= 0)[:, None], a[src[at].clamp(min=0)], 0).double()
        _compare(out[at], rows @ _values(codes[x], s[x], None if z is None else z[x]).t(), act,
                 (x, counts[x], k, n, group, zeros, kind, act, cap, gather))
    _untouched(out[~live])
    if tiles is not None:
        x = max(range(e), key=lambda i: counts[i])
        at = ends[x] + 1  # (no multiple of seven: it has a source)
        while at % 7 == 0:
            at += 1
        a[src[at], 0] = float("inf")
        assert bool(run(a, torch.zeros((row_cap, n), dtype=torch.bfloat16, device="cuda"), None)[at].isinf().any()) == tiles


SEGMENTS = [65, 1, 0, 600, 128, 129, 33, 300, 16, 192, 0, 161]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", [None] + ACTS)
def test_tiles_per_expert(act, group):
    """Aligned segments and masked batches, gathered through a map with rows that
    have no source; six steps of K and a part of one (where the group divides it)."""
    k = 832 // group * group
    for i, (align, cap, gather, n) in enumerate(((16, 0, 3, 4096), (1, 0, 0, 3082), (1, 300, 2, 4096), (1, 608, 0, 2600))):
        for zeros in (False, True):
            say(f"int4 tiles per expert {act} group {group} align {align} cap {cap} gather {gather} zeros {zeros}")
            _grouped(_gen(503, group, i, zeros), SEGMENTS, k, n, group, zeros, (torch.bfloat16, torch.float16)[i % 2], act,
                     align, cap, gather, slack=0 if cap else 40 * (i % 2), tiles=True if act is None else None)


@pytest.mark.parametrize("tail", [1, 31, 32, 33, 63, 64, 65, 96, 97, 127])
def test_last_tiles_of_any_rows(tail):
    """Of 64 and of 128 rows, half of them or more empty."""
    _grouped(_gen(504, tail), [128 + tail, 256 + tail, 64 + tail], 384, 4096, 128, False, torch.bfloat16, tiles=True)
    _grouped(_gen(505, tail), [1024 + tail] * 4, 512, 16384, 64, True, torch.bfloat16, gather=2, tiles=True)


@pytest.mark.parametrize("most", [3, 4, 16, 20, 64])
@pytest.mark.parametrize("group", [32, 128])
def test_streamed_workgroups_take_several_experts(most, group):
    """More units than the workgroups that stay: the next one's rows and sums take the
    LDS of the one before."""
    g = np.random.default_rng(most)
    counts = g.integers(0, most + 1, 100).tolist()
    counts[7], counts[99] = most, most
    for i in range(2):
        _grouped(_gen(506, most, group, i), counts, 384, 2048, group, i == 1, torch.bfloat16, (None, "swiglu")[i],
                 gather=2 * i, bound=most)


@pytest.mark.parametrize("e", [600, 1024])
def test_experts_past_one_scan(e):
    """A wave scans 512 experts at a time: live ones on both sides, streamed and tiled."""
    counts = [0] * e
    for x, c in ((0, 3), (510, 9), (511, 20), (512, 17), (513, 1), (e - 2, 64), (e - 1, 5)):
        counts[x] = c
    for bound in (4, 16, 64):
        _grouped(_gen(507, e, bound), counts, 256, 96, 128, False, torch.bfloat16, bound=bound)
    for x, c in ((3, 130), (511, 70), (512, 300), (e - 1, 65)):
        counts[x] = c
    _grouped(_gen(508, e), counts, 128, 2048, 32, True, torch.bfloat16, tiles=True)


@pytest.mark.parametrize("rows", [300, 700])
@pytest.mark.parametrize("zeros", [False, True])
def test_infinities_and_nan_in_tiles(zeros, rows):
    """An infinity is one where its weight is not zero (and a NaN where it is), also at
    a row's start where K is no whole step; NaN stays in its row or column."""
    k, n = 352, 8192
    g = _gen(509, rows, zeros)
    a = _rows(g, rows, k)
    codes, s, z = _weights(g, (), n, k, 32, zeros, torch.bfloat16)
    clean = moe.moe_gemm_int4(a, codes, s, z)
    bad = a.clone()
    bad[1, 17], bad[2, 0], bad[rows - 1, k - 1] = float("nan"), float("inf"), float("-inf")
    out = moe.moe_gemm_int4(bad, codes, s, z)
    assert bool(out[1].isnan().all())
    w = _values(codes, s, z)
    for r, col, sign in ((2, 0, 1.0), (rows - 1, k - 1, -1.0)):
        want = sign * float("inf") * w[:, col]
        assert torch.equal(out[r].isnan(), want.isnan()) and torch.equal(out[r].double().nan_to_num(7.0, 1.0, -1.0),
                                                                         want.nan_to_num(7.0, 1.0, -1.0))
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[1, 2, rows - 1]] = False
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    for value in (float("nan"), float("inf")):
        s2 = s.clone()
        s2[5, 10], s2[n - 1, 0] = value, value
        out = moe.moe_gemm_int4(a, codes, s2, z)
        assert not bool(out[:, [5, n - 1]].isfinite().any())
        assert torch.equal(out[:, 6:n - 1].view(torch.int16), clean[:, 6:n - 1].view(torch.int16))


@pytest.mark.parametrize("act", [None, "swiglu_clamp", "swiglu_clamp_after_silu"])
def test_nan_passes_the_clamps_in_tiles(act):
    a = _rows(_gen(510), 700, 256)
    codes, s, z = _weights(_gen(511), (), 8192, 256, 64, False, torch.bfloat16)
    a[699, 255] = float("nan")
    s[4096 + 3, 1] = float("nan")
    out = moe.moe_gemm_int4(a, codes, s, z, act=act, clamp_limit=LIM)
    col = 4096 + 3 if act is None else 3
    assert bool(out[699].isnan().all()) and bool(out[:, col].isnan().all())
    keep = [c for c in range(out.shape[1]) if c != col]
    assert bool(out[:699][:, keep].isfinite().all())


@pytest.mark.parametrize("rows", [40, 300, 700])
@pytest.mark.parametrize("zeros", [False, True])
def test_scales_at_the_ends_of_their_range(zeros, rows):
    """What the quantizer makes and the dequantization gives back finite is used as such:
    scales up to 2**126 and down to BF16's least, with rows that bring the sums back."""
    n, k, group = 4096, 256, 64
    for e in (126, 119, -126, -133):
        a = _rows(_gen(512, rows, e + 200), rows, k) * 2.0 ** (-60 if e > 0 else 60)
        codes, s, z = _weights(_gen(513, rows, e + 200), (), n, k, group, zeros, torch.bfloat16)
        s = torch.full_like(s, 2.0 ** e)
        assert bool(moe.moe_int4_dequant(codes[:8], s[:8], None if z is None else z[:8]).isfinite().all()) or e == 126
        out = moe.moe_gemm_int4(a, codes, s, z)
        _compare(out, a.double() @ _values(codes, s, z).t(), None, (rows, e))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [300, 700])
def test_gates_of_any_size_in_tiles(act, rows):
    """SiLU from its overflow to its underflow: sums of one value. The exponential's
    argument is off by 2**-24 of itself at most; below -128 ln 2 it is infinite in fp32,
    and SiLU zero instead of at most 2**-121."""
    values = [0.0, 1e-30, 1.0, 20.0, 87.0, 88.5, 89.0, 100.0, 104.0, 127.0, 128.0, 150.0, 1e4, 1e15]
    values = torch.tensor([x for v in values for x in (v, -v)], device="cuda").bfloat16()
    k, n, lim = 64, 8192, 1e3
    a = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    r = torch.arange(rows, device="cuda")
    a[r, r * 7 % k] = values[r % values.numel()]
    codes = torch.full((n, k // 2), 0x99, dtype=torch.uint8, device="cuda")
    out = moe.moe_gemm_int4(a, codes, torch.ones((n, 2), dtype=torch.bfloat16, device="cuda"), act=act, clamp_limit=lim)
    x = a.double().sum(1, keepdim=True)
    gate = x.clamp(max=lim) if act == "swiglu_clamp" else x
    ref = gate / (1 + torch.exp(-gate))
    if act == "swiglu_clamp_after_silu":
        ref = ref.clamp(max=lim)
    u = x if act == "swiglu" else x.clamp(-lim, lim)
    ref = ref * u
    bound = ref.abs() * (2.0 ** -8 + 2.0 ** -20 + 2.0 ** -23 * gate.abs().clamp(max=200)) + 2.0 ** -126
    bound = bound + torch.where(gate < -88.7, 2.0 ** -121 * u.abs(), 0.0)
    assert bool(((out.double() - ref).abs() <= bound).all())


def test_tiles_twice_and_at_once():
    """The same call gives the same bits, alone, on two streams at once and replayed."""
    counts = [300, 65, 0, 129]
    ends = torch.tensor([0, 304, 384, 384, 528], dtype=torch.int32, device="cuda")
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    g = _gen(514)
    a = torch.randn((528, 1024), generator=g, device="cuda").bfloat16()
    codes, s, z = _weights(g, (4,), 4096, 1024, 32, True, torch.float16)

    def run(out):
        return moe.moe_grouped_gemm_int4(a, codes, s, c, ends, 528, w_zeros=z, act="swiglu", out=out)
    new = lambda: torch.zeros((528, 2048), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want = run(new())
    outs = [new() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, o in zip(streams, outs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs[2])
    for _ in range(3):
        outs[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.int16), want.view(torch.int16)) for o in outs)
        run(outs[0])
