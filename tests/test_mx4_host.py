"""Host-only checks of the 4-bit activation format and the router: the C ABI's
and the binding's refusals come before any HIP call, and the workspace of a
layer with MXFP4 activations has their sizes."""

import ctypes

import pytest
import torch

import block_fp8_mixture_amd as moe
from block_fp8_mixture_amd import _binding as B

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3
NULL = None
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1002)
EIGHT = ctypes.c_void_p(0x1008)  # every MXFP4 operand is at a multiple of 16
MX = 4


@pytest.fixture(scope="module")
def lib():
    return moe.load_library()


def test_route_validation(lib):
    def call(e=8, k=2, score=0, renorm=1, scale=1.0, g=1, tg=1, gt=1, logits=FAKE, type=0, ld=None, t=4,
             ids=FAKE, w=FAKE, r=True):
        router = B._Router(e, k, score, renorm, scale, g, tg, gt)
        return lib.moe_route(ctypes.byref(router) if r else None, logits, type, e if ld is None else ld, NULL,
                             t, NULL, ids, w, NULL)
    assert call(r=False) == INVALID
    for bad in (dict(e=0), dict(k=0), dict(score=2), dict(g=0), dict(tg=0), dict(g=2, tg=3), dict(gt=0),
                dict(gt=3), dict(t=-1), dict(type=3), dict(ld=7), dict(logits=NULL), dict(ids=NULL),
                dict(w=NULL), dict(scale=float("inf")), dict(scale=float("nan")), dict(k=9),
                dict(g=3), dict(e=8, g=4, tg=1, k=3), dict(ld=1 << 62), dict(t=1 << 30, k=2)):
        assert call(**bad) == INVALID, bad
    assert call(e=1025) == UNSUPPORTED
    assert call(e=512, k=65) == UNSUPPORTED
    assert call(e=130, g=65, tg=65) == UNSUPPORTED
    assert call(t=0, logits=NULL, ids=NULL, w=NULL) == OK


def test_dequant_validation(lib):
    f = lib.moe_mxfp4_dequant
    assert f(FAKE, FAKE, -1, 32, FAKE, NULL) == INVALID
    assert f(FAKE, FAKE, 1, 0, FAKE, NULL) == INVALID
    assert f(FAKE, FAKE, 1, 48, FAKE, NULL) == INVALID
    assert f(NULL, FAKE, 1, 32, FAKE, NULL) == INVALID
    assert f(FAKE, NULL, 1, 32, FAKE, NULL) == INVALID
    assert f(FAKE, FAKE, 1, 32, NULL, NULL) == INVALID
    assert f(ODD, FAKE, 1, 32, FAKE, NULL) == INVALID
    assert f(FAKE, FAKE, 1, 32, ODD, NULL) == INVALID
    assert f(FAKE, FAKE, 1 << 62, 32, FAKE, NULL) == INVALID
    assert f(NULL, NULL, 0, 32, NULL, NULL) == OK


def test_mxfp4_format_of_the_stages(lib):
    q = lib.moe_act_quant
    assert q(FAKE, 4, NULL, 200, MX, 0, FAKE, FAKE, NULL) == INVALID
    assert q(NULL, 4, NULL, 256, MX, 0, FAKE, FAKE, NULL) == INVALID
    assert q(NULL, 0, NULL, 256, MX, 0, NULL, NULL, NULL) == OK
    s = lib.moe_silu_mul_quant
    assert s(FAKE, 200, FAKE, FAKE, 4, 64, 0, 7.0, MX, 0, FAKE, FAKE, NULL) == INVALID
    assert s(NULL, 256, FAKE, FAKE, 4, 64, 0, 7.0, MX, 0, FAKE, FAKE, NULL) == INVALID
    assert s(NULL, 256, FAKE, FAKE, 4, 0, 0, 7.0, MX, 0, NULL, NULL, NULL) == OK
    # FP8 weights take FP8 activations
    f = lib.moe_grouped_gemm_fp8
    assert f(FAKE, FAKE, MX, 64, NULL, 1, FAKE, FAKE, FAKE, FAKE, 4, 64, 0, 256, 256, FAKE, NULL, NULL) == UNSUPPORTED
    f = lib.moe_grouped_gemm_fp8_masked
    assert f(FAKE, FAKE, MX, 64, NULL, 1, FAKE, FAKE, FAKE, 4, 16, 256, 256, FAKE, NULL, NULL) == UNSUPPORTED


def test_mxfp4_quantization_alignment(lib):
    q, s, m = lib.moe_act_quant, lib.moe_silu_mul_quant, lib.moe_silu_mul_quant_masked
    for x, c in ((EIGHT, FAKE), (ODD, FAKE), (FAKE, ODD)):
        assert q(x, 4, NULL, 256, MX, 0, c, FAKE, NULL) == INVALID
        assert s(x, 256, FAKE, FAKE, 4, 64, 0, 7.0, MX, 0, c, FAKE, NULL) == INVALID
        assert m(x, 256, FAKE, 4, 16, 0, 7.0, MX, 0, c, FAKE, NULL) == INVALID


def test_mxfp4_gemm_alignment(lib):
    f = lib.moe_grouped_gemm_mxfp4

    def call(a=FAKE, asc=FAKE, w=FAKE, ws=FAKE, c=FAKE, n=256, k=256, rc=64):
        return f(a, asc, MX, 64, NULL, 1, w, ws, FAKE, FAKE, 0, 4, rc, 0, n, k, c, NULL)
    for bad in (dict(a=ODD), dict(w=ODD), dict(c=ODD), dict(asc=ODD), dict(ws=ODD), dict(asc=NULL),
                dict(a=EIGHT), dict(w=EIGHT), dict(c=EIGHT), dict(asc=EIGHT), dict(ws=EIGHT), dict(n=200), dict(k=64)):
        assert call(**bad) == INVALID, bad
    assert call(rc=0) == OK


def _problem(**over):
    p = dict(num_experts=4, hidden=256, inter=128, topk=2, t_cap=8, align_rows=16, row_cap=0, scale_fmt=MX,
             act=0, clamp_limit=float("inf"), rounding=0, expert_start=0, expert_cap=0, weight_fmt=1)
    p.update(over)
    return B._Problem(*p.values())


def test_workspace_of_mxfp4_activations(lib):
    lay = B._Layout()
    assert lib.moe_workspace_plan(ctypes.byref(_problem(weight_fmt=0)), ctypes.byref(lay)) == UNSUPPORTED
    assert lib.moe_workspace_plan(ctypes.byref(_problem(scale_fmt=3)), ctypes.byref(lay)) == INVALID
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for over in (dict(t_cap=100), dict(t_cap=100, expert_cap=32), dict(t_cap=8)):
        p = _problem(**over)
        assert lib.moe_workspace_plan(ctypes.byref(p), ctypes.byref(lay)) == OK
        t, h, i, r = p.t_cap, p.hidden, p.inter, lay.row_cap
        assert lay.xs - lay.xq == up(t * h // 2)
        assert lay.c1 - lay.xs == up(t * h // 32)
        assert lay.hs - lay.hq == up(r * i // 2)
        assert lay.y - lay.hs == up(r * i // 32)


def test_forward_refuses_misaligned_tensors(lib):
    p = _problem(t_cap=100)
    n = lib.moe_workspace_bytes(ctypes.byref(p))
    names = [f for f, _ in B._Tensors._fields_]
    for name, value in (("x", ODD), ("w1", ODD), ("w2", ODD), ("out", ODD), ("w1_scales", ODD), ("w2_scales", ODD)):
        t = B._Tensors(*[value.value if f == name else (None if f == "t_live_dev" else FAKE.value) for f in names])
        assert lib.moe_forward(ctypes.byref(p), ctypes.byref(t), FAKE, n, NULL) == INVALID, name
    t = B._Tensors(*[None if f == "t_live_dev" else FAKE.value for f in names])
    assert lib.moe_forward(ctypes.byref(p), ctypes.byref(t), ODD, n, NULL) == INVALID
    assert lib.moe_forward(ctypes.byref(p), ctypes.byref(t), FAKE, n - 1, NULL) == CAPACITY


# ---- the binding --------------------------------------------------------------

@pytest.mark.parametrize("name", ["x", "w1", "w2", "out", "w1_scales", "w2_scales"])
def test_forward_refuses_tensors_at_odd_multiples_of_eight(lib, name):
    p = _problem(t_cap=4)
    n = lib.moe_workspace_bytes(ctypes.byref(p))
    names = [f for f, _ in B._Tensors._fields_]
    t = B._Tensors(*[EIGHT.value if f == name else (None if f == "t_live_dev" else FAKE.value) for f in names])
    assert lib.moe_forward(ctypes.byref(p), ctypes.byref(t), FAKE, n, NULL) == INVALID


def test_route_binding_refusals():
    l = torch.zeros((4, 8))
    with pytest.raises(TypeError, match="tensor"):
        moe.moe_route([[0.0]], 1)
    with pytest.raises(TypeError, match="logits"):
        moe.moe_route(l.double(), 2)
    with pytest.raises(ValueError, match="num_experts"):
        moe.moe_route(l[0], 2)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_route(l.t(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_route(l[:1].expand(4, 8), 2)  # rows on top of each other
    with pytest.raises(ValueError, match="score"):
        moe.moe_route(l, 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        moe.moe_route(l, 2, bias=torch.zeros(7))
    with pytest.raises(TypeError, match="bias"):
        moe.moe_route(l, 2, bias=torch.zeros(8).half())
    with pytest.raises(ValueError, match="ids"):
        moe.moe_route(l, 2, ids=torch.zeros((4, 3), dtype=torch.int32))
    with pytest.raises(ValueError, match="weights"):
        moe.moe_route(l, 2, weights=torch.zeros((3, 2)))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_route(l, 2)


def test_mxfp4_binding_refusals():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    u8 = torch.uint8
    with pytest.raises(ValueError, match="xq"):
        moe.moe_act_quant(x, "mxfp4", xq=torch.zeros((4, 256), dtype=u8))
    with pytest.raises(ValueError, match="xs"):
        moe.moe_act_quant(x, "mxfp4", xs=torch.zeros((2, 4), dtype=u8))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_act_quant(x, "mxfp4")
    with pytest.raises(ValueError, match="codes"):
        moe.moe_mxfp4_dequant(torch.zeros((4, 24), dtype=u8), torch.zeros((4, 1), dtype=u8))
    with pytest.raises(ValueError, match="scales"):
        moe.moe_mxfp4_dequant(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 1), dtype=u8))
    with pytest.raises(ValueError, match="out"):
        moe.moe_mxfp4_dequant(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 2), dtype=u8),
                              out=torch.zeros((4, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_mxfp4_dequant(torch.zeros((4, 32), dtype=u8), torch.zeros((4, 2), dtype=u8))
    counts, offsets = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros((2, 128, 128), dtype=u8), torch.zeros((2, 128, 8), dtype=u8)
    a, asc = torch.zeros((16, 128), dtype=u8), torch.zeros((16, 8), dtype=u8)
    with pytest.raises(ValueError, match="K"):
        moe.moe_grouped_gemm_mxfp4(torch.zeros((16, 256), dtype=u8), asc, "mxfp4", w, ws, counts, offsets, 16)
    with pytest.raises(ValueError, match="a_scales"):
        moe.moe_grouped_gemm_mxfp4(a, torch.zeros((2, 16), dtype=u8), "mxfp4", w, ws, counts, offsets, 16)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_grouped_gemm_mxfp4(a, asc, "mxfp4", w, ws, counts, offsets, 16)
    gu = torch.zeros((16, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="hq"):
        moe.moe_silu_mul_quant(gu, counts, offsets, fmt="mxfp4", hq=torch.zeros((16, 128), dtype=u8))
    with pytest.raises(ValueError, match="hs"):
        moe.moe_silu_mul_quant_masked(gu, counts, 8, fmt="mxfp4", hs=torch.zeros((1, 16), dtype=u8))
    with pytest.raises(ValueError, match="scale format"):
        moe.moe_workspace_bytes(4, 256, 128, 2, 8, fmt="fp4")
    with pytest.raises(moe.MoeError, match="unsupported"):
        moe.moe_workspace_plan(4, 256, 128, 2, 8, fmt="mxfp4")
    assert moe.moe_workspace_bytes(4, 256, 128, 2, 8, fmt="mxfp4", weight_fmt="mxfp4") > 0
