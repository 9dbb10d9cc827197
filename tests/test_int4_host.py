"""Host-only checks of the norm and of the 4-bit integer weights: the C ABI's and
the binding's refusals come before any HIP call."""

import ctypes

import pytest
import torch

import block_fp8_mixture_amd as moe
from block_fp8_mixture_amd import _binding as B

OK, INVALID, UNSUPPORTED = 0, 1, 2
NULL = None
BASE = 1 << 30


def _p(v):
    """Never dereferenced: validation fails first."""
    return None if v is None else ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def _norm(lib, **over):
    p = dict(x=BASE, ld=256, r=2 * BASE, w=3 * BASE, wt=1, eps=1e-6, t=4, live=None, hidden=256, fmt=0, rnd=0,
             ro=2 * BASE, y=4 * BASE, xq=5 * BASE, xs=6 * BASE)
    p.update(over)
    return lib.moe_rmsnorm_quant(_p(p["x"]), p["ld"], _p(p["r"]), _p(p["w"]), p["wt"], p["eps"], p["t"],
                                 _p(p["live"]), p["hidden"], p["fmt"], p["rnd"], _p(p["ro"]), _p(p["y"]),
                                 _p(p["xq"]), _p(p["xs"]), NULL)


@pytest.mark.parametrize("over", [
    dict(t=-1), dict(hidden=0), dict(hidden=200), dict(hidden=-128), dict(ld=255), dict(ld=260), dict(ld=1 << 62),
    dict(wt=2), dict(wt=3), dict(wt=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(fmt=3), dict(fmt=5), dict(rnd=2), dict(x=None), dict(w=None), dict(r=None), dict(ro=None),
    dict(xq=None), dict(xs=None), dict(y=None, xq=None, xs=None), dict(x=BASE + 2), dict(r=BASE + 8, ro=BASE + 8),
    dict(w=BASE + 4), dict(ro=BASE * 7 + 8), dict(y=BASE * 4 + 8), dict(xq=BASE * 5 + 4), dict(fmt=4, xq=BASE * 5 + 2),
    dict(xs=BASE * 6 + 2),
])
def test_norm_refusals(lib, over):
    assert _norm(lib, **over) == INVALID


@pytest.mark.parametrize("over", [
    dict(ro=BASE + 16), dict(ro=BASE, ld=512), dict(ro=2 * BASE - 16), dict(y=BASE + 512), dict(y=BASE, ld=512),
    dict(y=2 * BASE), dict(y=2 * BASE + 512, ro=7 * BASE), dict(y=3 * BASE), dict(y=3 * BASE - 2032),
    dict(xq=BASE), dict(xq=2 * BASE), dict(xq=3 * BASE), dict(xq=4 * BASE), dict(xs=BASE + 16), dict(xs=2 * BASE),
    dict(xs=3 * BASE), dict(xs=4 * BASE), dict(xs=5 * BASE), dict(live=2 * BASE + 8), dict(live=4 * BASE),
    dict(live=5 * BASE), dict(live=6 * BASE), dict(x=BASE, ld=4096, y=BASE + 2 * 4096),
])
def test_norm_refuses_overlaps(lib, over):
    assert _norm(lib, **over) == INVALID


def test_norm_limits(lib):
    assert _norm(lib, hidden=32768 + 128, ld=32768 + 128) == UNSUPPORTED
    assert _norm(lib, t=0, x=None, w=None, r=None, ro=None, xq=None, xs=None, y=None) == OK
    assert _norm(lib, t=(1 << 31) - 1) == INVALID  # more groups than 31 bits count


def test_int4_quant_validation(lib):
    f = lib.moe_int4_quant
    odd = _p(2 * BASE + 2)

    def call(w=_p(BASE), type=1, rows=4, cols=256, group=64, st=1, codes=_p(2 * BASE), scales=_p(3 * BASE), zeros=None):
        return f(w, type, rows, cols, group, st, codes, scales, zeros, NULL)
    for bad in (dict(type=3), dict(type=-1), dict(rows=-1), dict(cols=0), dict(cols=96), dict(group=16),
                dict(group=256), dict(group=0), dict(st=0), dict(st=3), dict(w=None), dict(codes=None),
                dict(scales=None), dict(w=_p(BASE + 8)), dict(codes=odd), dict(scales=_p(3 * BASE + 1)),
                dict(rows=1 << 62), dict(codes=_p(BASE + 2044)), dict(w=_p(2 * BASE), type=0),
                dict(scales=_p(BASE)), dict(zeros=_p(BASE)), dict(zeros=_p(2 * BASE + 511)), dict(zeros=_p(3 * BASE + 31)),
                dict(scales=_p(2 * BASE + 510)), dict(codes=_p(BASE + 4092), type=0)):
        assert call(**bad) == INVALID, bad
    assert call(rows=0, w=None, codes=None, scales=None) == OK


def test_int4_dequant_validation(lib):
    f = lib.moe_int4_dequant
    def call(codes=_p(BASE), scales=_p(2 * BASE), st=1, zeros=None, rows=4, cols=256, group=64, out=_p(3 * BASE)):
        return f(codes, scales, st, zeros, rows, cols, group, out, NULL)
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=96), dict(group=48), dict(st=0), dict(codes=None),
                dict(scales=None), dict(out=None), dict(codes=_p(BASE + 4)), dict(out=_p(3 * BASE + 8)),
                dict(scales=_p(2 * BASE + 1)), dict(rows=1 << 62), dict(out=_p(BASE)), dict(codes=_p(3 * BASE + 2040)),
                dict(scales=_p(3 * BASE + 2046)), dict(zeros=_p(3 * BASE + 2047))):
        assert call(**bad) == INVALID, bad
    assert call(rows=0, codes=None, scales=None, out=None) == OK


def _weights(codes=BASE, scales=2 * BASE, zeros=None, st=1, group=64, e=1, n=64, k=256):
    return B._Int4Weights(codes, scales, zeros, st, group, e, n, k)


WEIGHTS_INVALID = [dict(codes=None), dict(scales=None), dict(codes=BASE + 8), dict(scales=2 * BASE + 1), dict(st=0),
                   dict(group=16), dict(group=96), dict(n=0), dict(k=0), dict(k=96), dict(e=0)]


def test_gemm_validation(lib):
    def call(a=_p(3 * BASE), rows=4, act=-1, lim=1.0, c=_p(4 * BASE), w=None, **over):
        return lib.moe_gemm_int4(a, rows, NULL, ctypes.byref(w or _weights(**over)), act, lim, c, NULL)
    for bad in WEIGHTS_INVALID + [dict(a=None), dict(c=None), dict(a=_p(3 * BASE + 8)), dict(c=_p(4 * BASE + 1)), dict(rows=-1),
                                  dict(act=3), dict(act=-2), dict(act=0, n=63), dict(act=1, lim=0.0),
                                  dict(act=2, lim=float("nan")), dict(act=1, lim=-1.0), dict(e=2),
                                  dict(rows=(1 << 31) - 1), dict(c=_p(3 * BASE + 2046)), dict(c=_p(BASE)),
                                  dict(c=_p(2 * BASE + 510)), dict(zeros=4 * BASE + 511)]:
        assert call(**bad) == INVALID, bad
    assert call(k=131072 + 64) == UNSUPPORTED
    assert call(k=131072, n=32768) == UNSUPPORTED
    assert call(k=64, n=(1 << 25) + 1) == UNSUPPORTED
    assert call(k=131072, rows=1 << 20) == UNSUPPORTED
    assert call(rows=0, a=None, c=None) == OK
    assert lib.moe_gemm_int4(_p(BASE), 4, NULL, None, -1, 1.0, _p(BASE), NULL) == INVALID


def test_grouped_gemm_validation(lib):
    def call(a=_p(3 * BASE), ar=64, div=1, counts=_p(5 * BASE), offsets=_p(6 * BASE), ec=0, rc=64, mr=0, act=-1, lim=1.0,
             c=_p(4 * BASE), e=4, **over):
        return lib.moe_grouped_gemm_int4(a, ar, NULL, div, ctypes.byref(_weights(e=e, **over)), counts, offsets, ec,
                                         rc, mr, act, lim, c, NULL)
    for bad in WEIGHTS_INVALID + [dict(a=None), dict(c=None), dict(ar=-1), dict(ar=0), dict(div=0), dict(counts=None),
                                  dict(offsets=None), dict(ec=-1), dict(ec=8), dict(rc=-1), dict(mr=-1), dict(act=7),
                                  dict(act=0, n=63), dict(act=1, lim=0.0), dict(rc=(1 << 31) - 1), dict(c=_p(3 * BASE)),
                                  dict(c=_p(5 * BASE + 14)), dict(c=_p(6 * BASE + 18)), dict(c=_p(BASE + 32766))]:
        assert call(**bad) == INVALID, bad
    assert call(e=1025) == UNSUPPORTED
    assert call(k=131072, ar=1 << 20) == UNSUPPORTED
    assert call(rc=0, a=None, c=None) == OK
    assert call(ec=0, rc=0) == OK
    # moe_act's extra value is a product's alone
    p = B._Problem(4, 256, 128, 2, 8, 16, 0, 0, -1, float("inf"), 0, 0, 0, 0)
    assert lib.moe_workspace_plan(ctypes.byref(p), ctypes.byref(B._Layout())) == INVALID


# ---- the binding --------------------------------------------------------------

BF, U8 = torch.bfloat16, torch.uint8


def test_norm_binding_refusals():
    x, w = torch.zeros((4, 256), dtype=BF), torch.ones(256)
    f = moe.moe_rmsnorm_quant
    with pytest.raises(TypeError, match="tensor"):
        f([[0.0]], w)
    with pytest.raises(TypeError, match="x must be"):
        f(x.half(), w)
    with pytest.raises(ValueError, match="hidden"):
        f(x[0], w)
    with pytest.raises(ValueError, match="contiguous"):
        f(x.t(), w)
    with pytest.raises(ValueError, match="contiguous"):
        f(x[:1].expand(4, 256), w)
    with pytest.raises(TypeError, match="weight"):
        f(x, w.half())
    with pytest.raises(ValueError, match="weight"):
        f(x, w[:128])
    with pytest.raises(ValueError, match="eps"):
        f(x, w, -1.0)
    with pytest.raises(ValueError, match="eps"):
        f(x, w, float("nan"))
    with pytest.raises(ValueError, match="scale format"):
        f(x, w, fmt="e5m2")
    with pytest.raises(ValueError, match="residual"):
        f(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="residual"):
        f(x, w, residual_out=x)
    with pytest.raises(ValueError, match="residual_out"):
        f(x, w, residual=x, residual_out=x[:3])
    with pytest.raises(TypeError, match="residual"):
        f(x, w, residual=x.float())
    with pytest.raises(ValueError, match="y must"):
        f(x, w, y=x[:3])
    with pytest.raises(ValueError, match="fmt"):
        f(x, w, fmt=None, xq=torch.zeros((4, 256), dtype=U8))
    with pytest.raises(ValueError, match="fmt"):
        f(x, w, fmt=None, y=False)
    with pytest.raises(ValueError, match="xq"):
        f(x, w, xq=torch.zeros((4, 128), dtype=U8))
    with pytest.raises(ValueError, match="xs"):
        f(x, w, xs=torch.zeros((4, 2)))
    with pytest.raises(TypeError, match="xs"):
        f(x, w, fmt="ue8m0", xs=torch.zeros((2, 4)))
    with pytest.raises(ValueError, match="GPU"):
        f(x, w)


def test_int4_binding_refusals():
    w = torch.zeros((8, 256), dtype=BF)
    q = moe.moe_int4_quant
    with pytest.raises(TypeError, match="w must"):
        q(w.double())
    with pytest.raises(ValueError, match="contiguous"):
        q(w.t())
    with pytest.raises(ValueError, match="group"):
        q(w, 16)
    with pytest.raises(ValueError, match="group"):
        q(w[:, :96].contiguous(), 64)
    with pytest.raises(TypeError, match="scales"):
        q(w, scale_dtype=torch.float32)
    with pytest.raises(ValueError, match="zero points"):
        q(w, zeros=torch.zeros((8, 2), dtype=U8))
    with pytest.raises(ValueError, match="codes"):
        q(w, codes=torch.zeros((8, 256), dtype=U8))
    with pytest.raises(ValueError, match="scales"):
        q(w, scales=torch.zeros((8, 4), dtype=BF))
    with pytest.raises(ValueError, match="zeros"):
        q(w, symmetric=False, zeros=torch.zeros((8, 4), dtype=U8))
    with pytest.raises(ValueError, match="GPU"):
        q(w)
    d = moe.moe_int4_dequant
    codes, scales = torch.zeros((8, 128), dtype=U8), torch.zeros((8, 4), dtype=BF)
    with pytest.raises(TypeError, match="scales"):
        d(codes, scales.float())
    with pytest.raises(ValueError, match="32, 64 or 128"):
        d(codes, torch.zeros((8, 1), dtype=BF))
    with pytest.raises(ValueError, match="32, 64 or 128"):
        d(codes, torch.zeros((8, 3), dtype=BF))
    with pytest.raises(ValueError, match="scales"):
        d(codes, torch.zeros((7, 4), dtype=BF))
    with pytest.raises(ValueError, match="zeros"):
        d(codes, scales, torch.zeros((8, 2), dtype=U8))
    with pytest.raises(ValueError, match="out"):
        d(codes, scales, out=torch.zeros((8, 128), dtype=BF))
    with pytest.raises(ValueError, match="GPU"):
        d(codes, scales)


def test_gemm_int4_binding_refusals():
    x, w, s = torch.zeros((4, 256), dtype=BF), torch.zeros((64, 128), dtype=U8), torch.zeros((64, 2), dtype=BF)
    f = moe.moe_gemm_int4
    for bad, match in ((dict(x=x[0]), "x must"), (dict(x=x[:, :128].contiguous()), "K"), (dict(w_scales=s[:32]), "w_scales"),
                       (dict(w_scales=torch.zeros((64, 5), dtype=BF)), "32, 64 or 128"),
                       (dict(w_zeros=torch.zeros((64, 4), dtype=U8)), "w_zeros"), (dict(act="gelu"), "act"),
                       (dict(w=w[:63], w_scales=s[:63], act="swiglu"), "even"), (dict(out=x), "out"),
                       (dict(act="swiglu", out=torch.zeros((4, 64), dtype=BF)), "out"),
                       (dict(t_live=torch.zeros(2, dtype=torch.int32)), "t_live"), ({}, "GPU")):
        with pytest.raises(ValueError, match=match):
            f(**{**dict(x=x, w=w, w_scales=s), **bad})
    for bad, match in ((dict(x=x.half()), "x must"), (dict(w=w.int()), "w must"), (dict(w_scales=s.float()), "w_scales"),
                       (dict(w_zeros=s), "w_zeros")):
        with pytest.raises(TypeError, match=match):
            f(**{**dict(x=x, w=w, w_scales=s), **bad})
    counts, offsets = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    a, we, se = torch.zeros((32, 256), dtype=BF), torch.zeros((2, 64, 128), dtype=U8), torch.zeros((2, 64, 2), dtype=BF)
    base = dict(a=a, w=we, w_scales=se, counts=counts, offsets=offsets, row_cap=32)
    g = moe.moe_grouped_gemm_int4
    for bad, match in ((dict(a=a[:16]), "row_cap"), (dict(counts=counts[:1]), "counts"), (dict(offsets=counts), "offsets"),
                       (dict(offsets=None), "aligned"), (dict(row_cap=None), "aligned"), (dict(w_scales=se[:1]), "w_scales"),
                       (dict(a_row_map=counts), "a_row_map"), (dict(out=torch.zeros((31, 64), dtype=BF)), "out"),
                       (dict(act="swiglu", out=torch.zeros((32, 64), dtype=BF)), "out"),
                       (dict(max_rows_per_expert=1 << 31), "2\\*\\*31"), ({}, "GPU")):
        with pytest.raises(ValueError, match=match):
            g(**{**base, **bad})
