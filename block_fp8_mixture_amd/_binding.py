"""ctypes marshalling for libmoefp8.so. No arithmetic of the layer lives here."""

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmoefp8.so"

SCALE_FMTS = {"fp32": 0, "pow2": 1, "ue8m0": 2, "mxfp4": 4}
ROUNDINGS = {"divide": 0, "reciprocal": 1}
# Types of norm weights and of 4-bit weights before their quantization, and of their scales.
ELEM_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
INT4_GROUPS = (32, 64, 128)
ACTS = {"swiglu": 0, "swiglu_clamp": 1, "swiglu_clamp_after_silu": 2}
WEIGHT_FMTS = {"e4m3": 0, "mxfp4": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
# Row-tile geometry of the grouped GEMM (mirrors the header's macros), used to
# interpret the tiles_visited counter.
GEMM_TILES = {"stream_tile_m": 16, "stream_max_rows": 64, "tiled_tile_m": 256, "col_tile": 128}
# Limits of moe_forward's decode path and of its one-launch form (mirrors the
# header's MOE_DECODE_* macros).
DECODE_LIMITS = {"max_pairs": 64, "fc2_row_bytes": 24576, "fc2_max_scales": 256,
                 "layer_token_bytes": 61440, "layer_max_scales": 512}


def decode_layer_applies(t_cap, topk, hidden, inter, weight_fmt="e4m3"):
    """Whether moe_forward runs this problem (aligned layout, FP8 activations) as
    its one-launch decode layer; with MXFP4 weights H and I must also be multiples of 256."""
    d, p = DECODE_LIMITS, t_cap * topk
    if _weight_fmt(weight_fmt) == 1 and (hidden % 256 or inter % 256):
        return False
    return (1 <= p <= d["max_pairs"] and p * (inter + 16) <= d["fc2_row_bytes"]
            and p * (inter // 128) <= d["fc2_max_scales"] and hidden % 16 == 0
            and t_cap * (hidden + 16) <= d["layer_token_bytes"]
            and t_cap * (hidden // 128) <= d["layer_max_scales"])

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "capacity too small",
           4: "HIP runtime error"}

# ctypes keeps the low 32 bits of a larger int32 argument without a word.
_PAST_INT32 = "sizes must be below 2**31"

_lock = threading.Lock()
_lib = None

_i32 = ctypes.c_int32
_vp = ctypes.c_void_p
_f32 = ctypes.c_float


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)} ({status})")


class _Problem(ctypes.Structure):
    _fields_ = [("num_experts", _i32), ("hidden", _i32), ("inter", _i32), ("topk", _i32),
                ("t_cap", _i32), ("align_rows", _i32), ("row_cap", _i32),
                ("scale_fmt", ctypes.c_int), ("act", ctypes.c_int), ("clamp_limit", _f32),
                ("rounding", ctypes.c_int), ("expert_start", _i32), ("expert_cap", _i32),
                ("weight_fmt", ctypes.c_int)]


class _Tensors(ctypes.Structure):
    _fields_ = [("x", _vp), ("topk_ids", _vp), ("topk_w", _vp), ("t_live_dev", _vp),
                ("w1", _vp), ("w1_scales", _vp), ("w2", _vp), ("w2_scales", _vp),
                ("out", _vp)]


class _Router(ctypes.Structure):
    _fields_ = [("num_experts", _i32), ("topk", _i32), ("score", ctypes.c_int), ("renormalize", _i32),
                ("scale", _f32), ("num_groups", _i32), ("top_groups", _i32), ("group_top", _i32)]


class _Int4Weights(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("zeros", _vp), ("scale_type", ctypes.c_int),
                ("group", _i32), ("num_experts", _i32), ("n", _i32), ("k", _i32)]


class _Layout(ctypes.Structure):
    _fields_ = [("expert_counts", ctypes.c_size_t), ("expert_offsets", ctypes.c_size_t),
                ("row_to_pair", ctypes.c_size_t), ("pair_to_row", ctypes.c_size_t),
                ("xq", ctypes.c_size_t), ("xs", ctypes.c_size_t), ("c1", ctypes.c_size_t),
                ("hq", ctypes.c_size_t), ("hs", ctypes.c_size_t), ("y", ctypes.c_size_t),
                ("act", ctypes.c_size_t), ("status", ctypes.c_size_t),
                ("overflow", ctypes.c_size_t), ("total", ctypes.c_size_t), ("row_cap", _i32)]


_SIGNATURES = {
    "moe_min_row_cap": (_i32, [_i32, _i32, _i32, _i32]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_route": (ctypes.c_int, [ctypes.POINTER(_Router), _vp, ctypes.c_int, ctypes.c_int64, _vp, _i32,
                                 _vp, _vp, _vp, _vp]),
    "moe_mxfp4_dequant": (ctypes.c_int, [_vp, _vp, ctypes.c_int64, _i32, _vp, _vp]),
    "moe_rmsnorm_quant": (ctypes.c_int, [_vp, ctypes.c_int64, _vp, _vp, ctypes.c_int, ctypes.c_double, _i32,
                                         _vp, _i32, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _vp]),
    "moe_int4_quant": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int64, _i32, _i32, ctypes.c_int, _vp, _vp,
                                      _vp, _vp]),
    "moe_int4_dequant": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, ctypes.c_int64, _i32, _i32, _vp, _vp]),
    "moe_gemm_int4": (ctypes.c_int, [_vp, _i32, _vp, ctypes.POINTER(_Int4Weights), ctypes.c_int, _f32, _vp,
                                     _vp]),
    "moe_grouped_gemm_int4": (ctypes.c_int, [_vp, _i32, _vp, _i32, ctypes.POINTER(_Int4Weights), _vp, _vp,
                                             _i32, _i32, _i32, ctypes.c_int, _f32, _vp, _vp]),
    "moe_align": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                 _vp]),
    "moe_align_batched": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                         _vp, _vp]),
    "moe_grouped_gemm_mxfp4": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i32, _vp, _i32, _vp, _vp,
                                              _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp,
                                              _vp]),
    "moe_grouped_gemm_fp8_masked": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i32, _vp, _i32, _vp,
                                                   _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                                   _vp]),
    "moe_silu_mul_quant_masked": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i32, ctypes.c_int, _f32,
                                                 ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "moe_act_quant": (ctypes.c_int, [_vp, _i32, _vp, _i32, ctypes.c_int, ctypes.c_int, _vp, _vp,
                                     _vp]),
    "moe_grouped_gemm_fp8": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i32, _vp, _i32, _vp, _vp,
                                            _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                                            _vp]),
    "moe_silu_mul_quant": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _i32, ctypes.c_int, _f32,
                                          ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]),
    "moe_topk_combine": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _vp]),
    "moe_workspace_plan": (ctypes.c_int, [ctypes.POINTER(_Problem), ctypes.POINTER(_Layout)]),
    "moe_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(_Problem)]),
    "moe_forward": (ctypes.c_int, [ctypes.POINTER(_Problem), ctypes.POINTER(_Tensors), _vp,
                                   ctypes.c_size_t, _vp]),
    "moe_fc1_decode": (ctypes.c_int, [ctypes.POINTER(_Problem), ctypes.POINTER(_Tensors), _vp,
                                      ctypes.c_size_t, _vp]),
    "moe_forward_noalloc": (ctypes.c_int, [ctypes.POINTER(_Problem), ctypes.POINTER(_Tensors), _vp]),
    "moe_barrier_timeouts": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32)]),
    "moe_barrier_spin_limit": (_i32, [_i32]),
}


def library_path():
    return os.path.join(_HERE, _LIB_NAME)


def load_library():
    """Load libmoefp8.so from the package directory (raises if it is not built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise ImportError(f"{path} is not built; run python -m block_fp8_mixture_amd.build")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(fn, status):
    if status != 0:
        raise MoeError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The handle of a device's current stream (torch.cuda.current_stream builds a
# Stream object around it: 3 us per call against 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # without its checks


def _stream(index):
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream


def _enqueue(name, device, *args):
    """Calls library function `name` on the current stream of `device`, where the
    tensors live (made the current device if it is another)."""
    fn = getattr(_lib, name)
    if device.index == _current_device():
        status = fn(*args, _stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(device.index))
    if status != 0:
        raise MoeError(name, status)


def _need(t, name, dtype, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t


def _shape(t, name, shape):
    """Raises ValueError unless tensor ``t`` has exactly ``shape``."""
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _exact(t, name, dtype, shape):
    """_need and _shape (a tuple), at once where they hold."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    return _shape(_need(t, name, dtype), name, shape)


def _min_numel(t, name, n):
    if t.numel() < n:
        raise ValueError(f"{name} needs at least {n} elements, has {t.numel()}")
    return t


def _same_device(*tensors):
    """All given tensors on one GPU (checked after every shape, so shape errors
    are reported first). Returns the device."""
    first, index = None, -1
    for t in tensors:
        if t is None:
            continue
        if first is None:
            first, index = t, t.get_device()  # -1 off the GPUs; cheaper than t.device
        elif t.get_device() != index:
            devs = {t.device for t in tensors if t is not None}
            raise ValueError(f"tensors live on different devices: {sorted(map(str, devs))}")
    if index < 0:
        raise ValueError("tensors must be GPU tensors")
    return first.device


def _fmt(fmt):
    if fmt not in SCALE_FMTS:
        raise ValueError(f"scale format must be one of {list(SCALE_FMTS)}")
    return SCALE_FMTS[fmt]


def _rounding(rounding):
    if rounding not in ROUNDINGS:
        raise ValueError(f"rounding must be one of {list(ROUNDINGS)}")
    return ROUNDINGS[rounding]


def _scale_dtype(fmt):
    return torch.uint8 if fmt in ("ue8m0", "mxfp4") else torch.float32


def _code_cols(cols, fmt):
    """Bytes of a row of codes (MXFP4: two columns per byte)."""
    return cols // 2 if fmt == "mxfp4" else cols


def _scale_shape(rows, cols, fmt):
    """Shape of the scales of [rows, cols]: group-major per 128 columns, or
    MXFP4's row-major bytes per 32."""
    return (rows, cols // 32) if fmt == "mxfp4" else (cols // 128, rows)


def _live(t_live):
    if t_live is None:
        return None
    _need(t_live, "t_live", torch.int32)
    if t_live.numel() != 1 or not t_live.is_cuda:
        raise ValueError("t_live must be a one-element int32 GPU tensor")
    return _ptr(t_live)


def _bf16(t, name):
    """BF16 values or their bits (int16); only the address is used."""
    return _need(t, name, torch.bfloat16 if t.dtype == torch.bfloat16 else torch.int16)


def _bf16_exact(t, name, shape):
    """_bf16 and _shape (a tuple), at once where they hold."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.shape == shape and t.is_contiguous():
        return t
    return _shape(_bf16(t, name), name, shape)


def moe_min_row_cap(t_cap, topk, num_experts, align_rows):
    return int(load_library().moe_min_row_cap(t_cap, topk, num_experts, align_rows))


def moe_status_string(status):
    return load_library().moe_status_string(status).decode()


def moe_route(logits, topk, score="softmax", bias=None, renormalize=True, scale=1.0, num_groups=1,
              top_groups=1, group_top=1, t_live=None, ids=None, weights=None):
    """Top-k routing from router logits [t_cap, E] (float32, bfloat16 or float16,
    columns contiguous, any row stride). Returns (ids int32 [t_cap, topk],
    weights float32 [t_cap, topk]), what moe_align and moe_forward take."""
    lib = load_library()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor")
    if logits.dtype not in LOGIT_TYPES:
        raise TypeError(f"logits must be one of {list(LOGIT_TYPES)}, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [t_cap, num_experts]")
    t_cap, num_experts = logits.shape
    ld = logits.stride(0) if t_cap > 1 else num_experts
    if (num_experts > 1 and logits.stride(1) != 1) or ld < num_experts:
        raise ValueError("the columns of logits must be contiguous and its rows apart")
    if score not in SCORES:
        raise ValueError(f"score must be one of {list(SCORES)}")
    num_groups, top_groups, group_top = int(num_groups), int(top_groups), int(group_top)
    if (t_cap | num_experts | topk | num_groups | top_groups | group_top) >> 31 not in (0, -1):
        raise ValueError(_PAST_INT32)
    if bias is not None:
        _exact(bias, "bias", torch.float32, (num_experts,))
    if ids is None:
        ids = torch.empty((t_cap, topk), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((t_cap, topk), dtype=torch.float32, device=logits.device)
    _exact(ids, "ids", torch.int32, (t_cap, topk))
    _exact(weights, "weights", torch.float32, (t_cap, topk))
    dev = _same_device(logits, bias, ids, weights, t_live)
    router = _Router(num_experts, topk, SCORES[score], int(bool(renormalize)), float(scale),
                     num_groups, top_groups, group_top)
    _enqueue("moe_route", dev, ctypes.byref(router), _ptr(logits), LOGIT_TYPES[logits.dtype], ld,
             _ptr(bias), t_cap, _live(t_live), _ptr(ids), _ptr(weights))
    return ids, weights


def moe_mxfp4_dequant(codes, scales, out=None):
    """BF16 values of an MXFP4 tensor: codes uint8 [..., cols/2], scales uint8
    [..., cols/32]. Returns BF16 [..., cols] (or ``out``)."""
    lib = load_library()
    shape = tuple(_need(codes, "codes", torch.uint8).shape)
    if not shape or shape[-1] < 16 or shape[-1] % 16:
        raise ValueError("codes must be [..., cols / 2] with cols a multiple of 32")
    lead, cols = shape[:-1], 2 * shape[-1]
    if cols >> 31:
        raise ValueError(_PAST_INT32)
    _exact(scales, "scales", torch.uint8, lead + (cols // 32,))
    if out is None:
        out = torch.empty(lead + (cols,), dtype=torch.bfloat16, device=codes.device)
    ob = _shape(_bf16(out, "out"), "out", lead + (cols,))
    dev = _same_device(codes, scales, ob)
    _enqueue("moe_mxfp4_dequant", dev, _ptr(codes), _ptr(scales), codes.numel() * 2 // cols, cols,
             _ptr(ob))
    return out


def moe_rmsnorm_quant(x, weight, eps=1e-6, fmt="fp32", residual=None, t_live=None, residual_out=None,
                      y=None, xq=None, xs=None, rounding="divide"):
    """RMS norm of x [t_cap, H] BF16 (columns contiguous, rows a multiple of 8
    elements apart) with the residual's addition and the quantization of its
    output. Returns (y BF16 [t_cap, H], xq, xs, residual_out): xq and xs as
    moe_act_quant(y, fmt) (None with ``fmt=None``; FP8 codes keep a NaN here),
    residual_out BF16 x + residual (None without a residual). ``y=False``: no BF16
    output (None). residual_out may be ``residual`` itself."""
    lib = load_library()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a tensor")
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.int16:
        raise TypeError(f"x must be {torch.bfloat16}, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must be [t_cap, hidden]")
    shape = t_cap, hidden = tuple(x.shape)
    if (t_cap | hidden) >> 31:
        raise ValueError(_PAST_INT32)
    ld, step = x.stride()
    if t_cap <= 1:
        ld = hidden
    if (hidden > 1 and step != 1) or ld < hidden:
        raise ValueError("the columns of x must be contiguous and its rows apart")
    weight_type = weight.dtype if isinstance(weight, torch.Tensor) else None
    if weight_type is not torch.bfloat16 and weight_type is not torch.float32:
        raise TypeError("weight must be a float32 or bfloat16 tensor")
    _exact(weight, "weight", weight_type, (hidden,))
    eps = float(eps)
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps must be finite and not negative")
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if residual is not None:
        _bf16_exact(residual, "residual", shape)
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        _bf16_exact(residual_out, "residual_out", shape)
    if y is None:
        y = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    elif y is False:
        y = None
    if y is not None:
        _bf16_exact(y, "y", shape)
    if fmt is None:
        if xq is not None or xs is not None:
            raise ValueError("xq and xs need a fmt")
        if y is None:
            raise ValueError("without y there must be a fmt")
    else:
        _fmt(fmt)
        codes, scales, scale_type = (t_cap, _code_cols(hidden, fmt)), _scale_shape(t_cap, hidden, fmt), _scale_dtype(fmt)
        if xq is None:
            xq = torch.empty(codes, dtype=torch.uint8, device=x.device)
        if xs is None:
            xs = torch.empty(scales, dtype=scale_type, device=x.device)
        _exact(xq, "xq", torch.uint8, codes)
        _exact(xs, "xs", scale_type, scales)
    dev = _same_device(x, weight, residual, residual_out, y, xq, xs, t_live)
    _enqueue("moe_rmsnorm_quant", dev, _ptr(x), ld, _ptr(residual), _ptr(weight), ELEM_TYPES[weight_type],
             eps, t_cap, _live(t_live), hidden, _fmt(fmt or "fp32"), _rounding(rounding),
             _ptr(residual_out), _ptr(y), _ptr(xq), _ptr(xs))
    return y, xq, xs, residual_out


def _int4_group(cols, groups, name):
    """Columns per group of ``groups`` scales in a row of ``cols`` columns."""
    group = cols // groups if groups else 0
    if group not in INT4_GROUPS or group * groups != cols:
        raise ValueError(f"{name} must have a scale per 32, 64 or 128 columns ({cols} columns, {groups} scales)")
    return group


def _int4_scale_type(scales, name):
    dtype = scales.dtype if isinstance(scales, torch.Tensor) else None
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"{name} must be a bfloat16 or float16 tensor")
    return ELEM_TYPES[dtype]


def moe_int4_quant(w, group=128, symmetric=True, scale_dtype=torch.bfloat16, codes=None, scales=None,
                   zeros=None):
    """4-bit integer weights of w [..., K] (float32, bfloat16 or float16), a scale
    (bfloat16 or float16) per ``group`` (32, 64 or 128) columns and, if not
    ``symmetric``, a zero point. Returns (codes uint8 [..., K/2], scales [...,
    K/group], zeros uint8 [..., K/group] or None)."""
    lib = load_library()
    if not isinstance(w, torch.Tensor) or w.dtype not in ELEM_TYPES:
        raise TypeError(f"w must be a tensor of one of {list(ELEM_TYPES)}")
    _need(w, "w", w.dtype)
    if group not in INT4_GROUPS:
        raise ValueError(f"group must be one of {INT4_GROUPS}")
    if w.dim() < 1 or w.shape[-1] < group or w.shape[-1] % group:
        raise ValueError("w must be [..., K] with K a multiple of the group")
    lead, cols = tuple(w.shape[:-1]), w.shape[-1]
    if cols >> 31:
        raise ValueError(_PAST_INT32)
    if codes is None:
        codes = torch.empty(lead + (cols // 2,), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(lead + (cols // group,), dtype=scale_dtype, device=w.device)
    if symmetric and zeros is not None:
        raise ValueError("symmetric weights have no zero points")
    if not symmetric and zeros is None:
        zeros = torch.empty(lead + (cols // group,), dtype=torch.uint8, device=w.device)
    _exact(codes, "codes", torch.uint8, lead + (cols // 2,))
    scale_type = _int4_scale_type(scales, "scales")
    _exact(scales, "scales", scales.dtype, lead + (cols // group,))
    if zeros is not None:
        _exact(zeros, "zeros", torch.uint8, lead + (cols // group,))
    dev = _same_device(w, codes, scales, zeros)
    _enqueue("moe_int4_quant", dev, _ptr(w), ELEM_TYPES[w.dtype], w.numel() // cols, cols, int(group),
             scale_type, _ptr(codes), _ptr(scales), _ptr(zeros))
    return codes, scales, zeros


def moe_int4_dequant(codes, scales, zeros=None, out=None):
    """BF16 values of 4-bit integer weights: codes uint8 [..., K/2], scales
    (bfloat16 or float16) and zeros (uint8 or None: 8) [..., K/group]. Returns
    BF16 [..., K] (or ``out``)."""
    lib = load_library()
    shape = tuple(_need(codes, "codes", torch.uint8).shape)
    scale_type = _int4_scale_type(scales, "scales")
    if not shape or scales.dim() != len(shape):
        raise ValueError("codes must be [..., K / 2] and scales [..., K / group]")
    lead, cols = shape[:-1], 2 * shape[-1]
    if cols >> 31:
        raise ValueError(_PAST_INT32)
    group = _int4_group(cols, scales.shape[-1], "codes")
    _exact(scales, "scales", scales.dtype, lead + (cols // group,))
    if zeros is not None:
        _exact(zeros, "zeros", torch.uint8, lead + (cols // group,))
    if out is None:
        out = torch.empty(lead + (cols,), dtype=torch.bfloat16, device=codes.device)
    ob = _shape(_bf16(out, "out"), "out", lead + (cols,))
    dev = _same_device(codes, scales, zeros, ob)
    _enqueue("moe_int4_dequant", dev, _ptr(codes), _ptr(scales), scale_type, _ptr(zeros),
             codes.numel() * 2 // cols, cols, group, _ptr(ob))
    return out


def _int4_weights(w, scales, zeros, num_experts, n, shape):
    """The C structure of checked weights whose shape is ``shape`` (a tuple)."""
    k = 2 * shape[-1]
    scale_type = _int4_scale_type(scales, "w_scales")
    got = tuple(scales.shape)
    if len(got) != len(shape):
        raise ValueError("w_scales must be [..., N, K / group]")
    group = _int4_group(k, got[-1], "w")
    want = shape[:-1] + got[-1:]
    if got != want or not scales.is_contiguous():
        _exact(scales, "w_scales", scales.dtype, want)
    if zeros is not None:
        _exact(zeros, "w_zeros", torch.uint8, want)
    if (n | k) >> 31:
        raise ValueError(_PAST_INT32)
    return _Int4Weights(_ptr(w), _ptr(scales), _ptr(zeros), scale_type, group, num_experts, n, k)


def _gate(act, n):
    """(value of moe_act, columns of the output)."""
    if act is None:
        return -1, n
    if act not in ACTS:
        raise ValueError(f"act must be None or one of {list(ACTS)}")
    if n % 2:
        raise ValueError("a gated product needs an even N")
    return ACTS[act], n // 2


def moe_gemm_int4(x, w, w_scales, w_zeros=None, act=None, clamp_limit=float("inf"), t_live=None, out=None):
    """Product of BF16 rows x [T, K] with 4-bit integer weights: w uint8 [N, K/2],
    w_scales (bfloat16 or float16) and w_zeros (uint8 or None) [N, K/group], from
    a single row (a matrix-vector product) to many. With ``act`` rows [0, N/2) of
    w are gates and [N/2, N) ups, and the result is the activation's. Returns BF16
    [T, N] (gated [T, N/2]), rows past ``t_live`` untouched."""
    lib = load_library()
    xb = _bf16(x, "x")
    if xb.dim() != 2:
        raise ValueError("x must be [T, K]")
    _need(w, "w", torch.uint8, ndim=2)
    rows, k = xb.shape
    n, k2 = shape = tuple(w.shape)
    if 2 * k2 != k:
        raise ValueError("x and w disagree on K")
    if rows >> 31:
        raise ValueError(_PAST_INT32)
    weights = _int4_weights(w, w_scales, w_zeros, 1, n, shape)
    act_value, out_n = _gate(act, n)
    if out is None:
        out = torch.empty((rows, out_n), dtype=torch.bfloat16, device=xb.device)
    ob = _bf16_exact(out, "out", (rows, out_n))
    if t_live is not None:
        _exact(t_live, "t_live", torch.int32, (1,))
    dev = _same_device(xb, w, w_scales, w_zeros, ob, t_live)
    _enqueue("moe_gemm_int4", dev, _ptr(xb), rows, _live(t_live), ctypes.byref(weights), act_value,
             float(clamp_limit), _ptr(ob))
    return out


def moe_grouped_gemm_int4(a, w, w_scales, counts, offsets=None, row_cap=None, w_zeros=None, a_row_map=None,
                          a_row_div=1, expert_cap=0, max_rows_per_expert=0, act=None,
                          clamp_limit=float("inf"), out=None):
    """Product of BF16 rows with every expert's 4-bit integer weights over its
    live rows: a [a_rows, K], w uint8 [E, N, K/2], w_scales and w_zeros [E, N,
    K/group], counts, offsets and row_cap as moe_align makes them (with
    ``expert_cap`` > 0 the batched layout: counts = masked_m, no offsets).
    Gated as moe_gemm_int4. Returns BF16 [row_cap, N] (gated [row_cap, N/2]),
    rows that are not live untouched."""
    lib = load_library()
    ab = _bf16(a, "a")
    if ab.dim() != 2:
        raise ValueError("a must be [a_rows, K]")
    _need(w, "w", torch.uint8, ndim=3)
    num_experts, n, k2 = shape = tuple(w.shape)
    a_rows, k = ab.shape
    if k != 2 * k2:
        raise ValueError("a and w disagree on K")
    weights = _int4_weights(w, w_scales, w_zeros, num_experts, n, shape)
    act_value, out_n = _gate(act, n)
    _exact(counts, "counts", torch.int32, (num_experts,))
    expert_cap, a_row_div, max_rows = int(expert_cap), int(a_row_div), int(max_rows_per_expert)
    if expert_cap > 0:
        row_cap = num_experts * expert_cap if row_cap is None else row_cap
        offsets = None
    else:
        if offsets is None or row_cap is None:
            raise ValueError("the aligned layout needs offsets and row_cap")
        _exact(offsets, "offsets", torch.int32, (num_experts + 1,))
    if (a_rows | row_cap | expert_cap | a_row_div | max_rows) >> 31 not in (0, -1):
        raise ValueError(_PAST_INT32)
    if out is None:
        out = torch.empty((max(row_cap, 1), out_n), dtype=torch.bfloat16, device=ab.device)
    ob = _bf16(out, "out")
    if ob.dim() != 2 or ob.shape[1] != out_n or ob.shape[0] < row_cap:
        raise ValueError(f"out must be [>= {row_cap}, {out_n}], got {tuple(ob.shape)}")
    if a_row_map is not None:
        _min_numel(_need(a_row_map, "a_row_map", torch.int32), "a_row_map", row_cap)
    elif a_rows < row_cap:
        raise ValueError("without a row map, a needs row_cap rows")
    dev = _same_device(ab, w, w_scales, w_zeros, counts, offsets, ob, a_row_map)
    _enqueue("moe_grouped_gemm_int4", dev, _ptr(ab), a_rows, _ptr(a_row_map), a_row_div,
             ctypes.byref(weights), _ptr(counts), _ptr(offsets), expert_cap, row_cap, max_rows, act_value,
             float(clamp_limit), _ptr(ob))
    return out


def moe_align(topk_ids, num_experts, align_rows=16, row_cap=None, t_live=None, out=None,
              expert_start=0):
    """Routing alignment. Returns dict(counts, offsets, row_to_pair, pair_to_row).
    Local expert ids are ``topk_ids - expert_start``."""
    lib = load_library()
    ids = _need(topk_ids, "topk_ids", torch.int32, ndim=2)
    t_cap, topk = ids.shape
    if row_cap is None:
        row_cap = moe_min_row_cap(t_cap, topk, num_experts, align_rows)
    dev = ids.device
    if out is None:
        out = {
            "counts": torch.empty(num_experts, dtype=torch.int32, device=dev),
            "offsets": torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
            "row_to_pair": torch.empty(max(row_cap, 1), dtype=torch.int32, device=dev),
            "pair_to_row": torch.empty(max(t_cap * topk, 1), dtype=torch.int32, device=dev),
        }
    for k, n in (("counts", num_experts), ("offsets", num_experts + 1),
                 ("row_to_pair", row_cap), ("pair_to_row", t_cap * topk)):
        _min_numel(_need(out[k], k, torch.int32), k, n)
    dev = _same_device(ids, *out.values())
    _enqueue("moe_align", dev, _ptr(ids), t_cap, _live(t_live), topk, num_experts, expert_start,
             align_rows, row_cap, _ptr(out["counts"]), _ptr(out["offsets"]),
             _ptr(out["row_to_pair"]), _ptr(out["pair_to_row"]))
    return out


def moe_align_batched(topk_ids, num_experts, expert_cap, t_live=None, out=None, expert_start=0):
    """Routing into the batched masked-M layout ([E, expert_cap] rows). Returns
    dict(masked_m, row_to_pair, pair_to_row, overflow)."""
    lib = load_library()
    ids = _need(topk_ids, "topk_ids", torch.int32, ndim=2)
    t_cap, topk = ids.shape
    dev = ids.device
    if out is None:
        out = {
            "masked_m": torch.empty(num_experts, dtype=torch.int32, device=dev),
            "row_to_pair": torch.empty(max(num_experts * expert_cap, 1), dtype=torch.int32, device=dev),
            "pair_to_row": torch.empty(max(t_cap * topk, 1), dtype=torch.int32, device=dev),
            "overflow": torch.empty(1, dtype=torch.int32, device=dev),
        }
    for k, n in (("masked_m", num_experts), ("row_to_pair", num_experts * expert_cap),
                 ("pair_to_row", t_cap * topk), ("overflow", 1)):
        _min_numel(_need(out[k], k, torch.int32), k, n)
    dev = _same_device(ids, *out.values())
    _enqueue("moe_align_batched", dev, _ptr(ids), t_cap, _live(t_live), topk, num_experts,
             expert_start, expert_cap, _ptr(out["masked_m"]), _ptr(out["row_to_pair"]),
             _ptr(out["pair_to_row"]), _ptr(out["overflow"]))
    return out


def moe_act_quant(x, fmt="fp32", t_live=None, xq=None, xs=None, rounding="divide"):
    """Per-token 1x128 quantization. Returns (xq uint8 [t_cap, H], xs [H/128, t_cap]);
    with ``fmt="mxfp4"`` (xq uint8 [t_cap, H/2], xs uint8 [t_cap, H/32])."""
    lib = load_library()
    xb = _bf16(x, "x")
    if xb.dim() != 2:
        raise ValueError("x must be [t_cap, hidden]")
    t_cap, hidden = xb.shape
    if xq is None:
        xq = torch.empty((t_cap, _code_cols(hidden, fmt)), dtype=torch.uint8, device=xb.device)
    if xs is None:
        xs = torch.empty(_scale_shape(t_cap, hidden, fmt), dtype=_scale_dtype(fmt), device=xb.device)
    _exact(xq, "xq", torch.uint8, (t_cap, _code_cols(hidden, fmt)))
    _exact(xs, "xs", _scale_dtype(fmt), _scale_shape(t_cap, hidden, fmt))
    dev = _same_device(xb, xq, xs, t_live)
    _enqueue("moe_act_quant", dev, _ptr(xb), t_cap, _live(t_live), hidden, _fmt(fmt),
             _rounding(rounding), _ptr(xq), _ptr(xs))
    return xq, xs


def moe_grouped_gemm_fp8(a, a_scales, fmt, w, w_scales, counts, offsets, row_cap,
                         a_row_map=None, a_row_div=1, max_rows_per_expert=0, out=None,
                         tiles_visited=None):
    """Grouped FP8 GEMM over live rows. ``w`` is uint8 [E, N, K]; returns BF16 bits
    (int16) [row_cap, N]."""
    lib = load_library()
    _need(a, "a", torch.uint8, ndim=2)
    _need(a_scales, "a_scales", _scale_dtype(fmt), ndim=2)
    _need(w, "w", torch.uint8, ndim=3)
    _need(w_scales, "w_scales", torch.float32, ndim=3)
    num_experts, n, k = w.shape
    a_rows = a.shape[0]
    if a.shape[1] != k:
        raise ValueError("a and w disagree on K")
    _shape(a_scales, "a_scales", (k // 128, a_rows))
    _shape(w_scales, "w_scales", (num_experts, n // 128, k // 128))
    _exact(counts, "counts", torch.int32, (num_experts,))
    _exact(offsets, "offsets", torch.int32, (num_experts + 1,))
    if out is None:
        out = torch.empty((max(row_cap, 1), n), dtype=torch.int16, device=a.device)
    ob = _bf16(out, "out")
    if ob.dim() != 2 or ob.shape[1] != n or ob.shape[0] < row_cap:
        raise ValueError(f"out must be [>= {row_cap}, {n}], got {tuple(ob.shape)}")
    if a_row_map is not None:
        _min_numel(_need(a_row_map, "a_row_map", torch.int32), "a_row_map", row_cap)
    elif a_rows < row_cap:
        raise ValueError("without a row map, a needs row_cap rows")
    if tiles_visited is not None:
        _min_numel(_need(tiles_visited, "tiles_visited", torch.int32), "tiles_visited", 1)
    dev = _same_device(a, a_scales, w, w_scales, counts, offsets, ob, a_row_map, tiles_visited)
    _enqueue("moe_grouped_gemm_fp8", dev, _ptr(a), _ptr(a_scales), _fmt(fmt), a_rows,
             _ptr(a_row_map), a_row_div, _ptr(w), _ptr(w_scales), _ptr(counts), _ptr(offsets),
             num_experts, row_cap, max_rows_per_expert, n, k, _ptr(ob), _ptr(tiles_visited))
    return out


def moe_grouped_gemm_mxfp4(a, a_scales, fmt, w, w_scales, counts, offsets=None, row_cap=None,
                           a_row_map=None, a_row_div=1, expert_cap=0, max_rows_per_expert=0,
                           out=None):
    """Grouped GEMM with MXFP4 weights over live rows. ``w`` is uint8 [E, N, K/2]
    packed E2M1 codes, ``w_scales`` uint8 [E, N, K/32] E8M0 bytes. With
    ``fmt="mxfp4"`` A is MXFP4 too (uint8 [a_rows, K/2] and [a_rows, K/32]). With
    ``expert_cap`` > 0 the batched layout (``counts`` = masked_m, no offsets,
    row_cap = E * expert_cap). Returns BF16 bits (int16) [row_cap, N]."""
    lib = load_library()
    _need(a, "a", torch.uint8, ndim=2)
    _need(a_scales, "a_scales", _scale_dtype(fmt), ndim=2)
    _need(w, "w", torch.uint8, ndim=3)
    _need(w_scales, "w_scales", torch.uint8, ndim=3)
    num_experts, n, k2 = w.shape
    k = 2 * k2
    a_rows = a.shape[0]
    if a.shape[1] != _code_cols(k, fmt):
        raise ValueError("a and w disagree on K")
    _shape(a_scales, "a_scales", _scale_shape(a_rows, k, fmt))
    _shape(w_scales, "w_scales", (num_experts, n, k // 32))
    _exact(counts, "counts", torch.int32, (num_experts,))
    if expert_cap > 0:
        row_cap = num_experts * expert_cap if row_cap is None else row_cap
        offsets = None
    else:
        if offsets is None or row_cap is None:
            raise ValueError("the aligned layout needs offsets and row_cap")
        _exact(offsets, "offsets", torch.int32, (num_experts + 1,))
    if out is None:
        out = torch.empty((max(row_cap, 1), n), dtype=torch.int16, device=a.device)
    ob = _bf16(out, "out")
    if ob.dim() != 2 or ob.shape[1] != n or ob.shape[0] < row_cap:
        raise ValueError(f"out must be [>= {row_cap}, {n}], got {tuple(ob.shape)}")
    if a_row_map is not None:
        _min_numel(_need(a_row_map, "a_row_map", torch.int32), "a_row_map", row_cap)
    elif a_rows < row_cap:
        raise ValueError("without a row map, a needs row_cap rows")
    dev = _same_device(a, a_scales, w, w_scales, counts, offsets, ob, a_row_map)
    _enqueue("moe_grouped_gemm_mxfp4", dev, _ptr(a), _ptr(a_scales), _fmt(fmt), a_rows,
             _ptr(a_row_map), a_row_div, _ptr(w), _ptr(w_scales), _ptr(counts), _ptr(offsets),
             int(expert_cap), num_experts, row_cap, int(max_rows_per_expert), n, k, _ptr(ob))
    return out


def moe_grouped_gemm_fp8_masked(a, a_scales, fmt, w, w_scales, masked_m, expert_cap,
                                a_row_map=None, a_row_div=1, out=None, tiles_visited=None):
    """Grouped FP8 GEMM on the batched masked-M layout: expert e's live rows are
    [e*cap, e*cap + masked_m[e]). Returns BF16 bits (int16) [E*cap, N]."""
    lib = load_library()
    _need(a, "a", torch.uint8, ndim=2)
    _need(a_scales, "a_scales", _scale_dtype(fmt), ndim=2)
    _need(w, "w", torch.uint8, ndim=3)
    _need(w_scales, "w_scales", torch.float32, ndim=3)
    num_experts, n, k = w.shape
    rows = num_experts * expert_cap
    a_rows = a.shape[0]
    if a.shape[1] != k:
        raise ValueError("a and w disagree on K")
    _shape(a_scales, "a_scales", (k // 128, a_rows))
    _shape(w_scales, "w_scales", (num_experts, n // 128, k // 128))
    _exact(masked_m, "masked_m", torch.int32, (num_experts,))
    if out is None:
        out = torch.empty((max(rows, 1), n), dtype=torch.int16, device=a.device)
    ob = _bf16(out, "out")
    if ob.dim() != 2 or ob.shape[1] != n or ob.shape[0] < rows:
        raise ValueError(f"out must be [>= {rows}, {n}], got {tuple(ob.shape)}")
    if a_row_map is not None:
        _min_numel(_need(a_row_map, "a_row_map", torch.int32), "a_row_map", rows)
    elif a_rows < rows:
        raise ValueError("without a row map, a needs num_experts * expert_cap rows")
    if tiles_visited is not None:
        _min_numel(_need(tiles_visited, "tiles_visited", torch.int32), "tiles_visited", 1)
    dev = _same_device(a, a_scales, w, w_scales, masked_m, ob, a_row_map, tiles_visited)
    _enqueue("moe_grouped_gemm_fp8_masked", dev, _ptr(a), _ptr(a_scales), _fmt(fmt), a_rows,
             _ptr(a_row_map), a_row_div, _ptr(w), _ptr(w_scales), _ptr(masked_m), num_experts,
             expert_cap, n, k, _ptr(ob), _ptr(tiles_visited))
    return out


def moe_silu_mul_quant_masked(gate_up, masked_m, expert_cap, act="swiglu",
                              clamp_limit=float("inf"), fmt="fp32", hq=None, hs=None,
                              rounding="divide"):
    """SiLU(gate)*up + 1x128 FP8 quantization on the batched masked-M layout.
    Returns (hq uint8 [E*cap, I], hs [I/128, E*cap]); with ``fmt="mxfp4"`` (hq
    [E*cap, I/2], hs uint8 [E*cap, I/32])."""
    lib = load_library()
    gu = _bf16(gate_up, "gate_up")
    _need(masked_m, "masked_m", torch.int32, ndim=1)
    num_experts = masked_m.shape[0]
    rows = num_experts * expert_cap
    if gu.dim() != 2 or gu.shape[1] % 2 or gu.shape[0] != rows:
        raise ValueError(f"gate_up must be [{rows}, 2 * inter], got {tuple(gu.shape)}")
    inter = gu.shape[1] // 2
    if hq is None:
        hq = torch.empty((rows, _code_cols(inter, fmt)), dtype=torch.uint8, device=gu.device)
    if hs is None:
        hs = torch.empty(_scale_shape(rows, inter, fmt), dtype=_scale_dtype(fmt), device=gu.device)
    _exact(hq, "hq", torch.uint8, (rows, _code_cols(inter, fmt)))
    _exact(hs, "hs", _scale_dtype(fmt), _scale_shape(rows, inter, fmt))
    dev = _same_device(gu, masked_m, hq, hs)
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}")
    _enqueue("moe_silu_mul_quant_masked", dev, _ptr(gu), inter, _ptr(masked_m), num_experts,
             expert_cap, ACTS[act], float(clamp_limit), _fmt(fmt), _rounding(rounding), _ptr(hq),
             _ptr(hs))
    return hq, hs


def moe_silu_mul_quant(gate_up, counts, offsets, act="swiglu", clamp_limit=float("inf"),
                       fmt="fp32", hq=None, hs=None, rounding="divide"):
    """SiLU(gate)*up + 1x128 FP8 quantization of live rows.
    Returns (hq uint8 [row_cap, I], hs [I/128, row_cap]); with ``fmt="mxfp4"``
    (hq [row_cap, I/2], hs uint8 [row_cap, I/32])."""
    lib = load_library()
    gu = _bf16(gate_up, "gate_up")
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError("gate_up must be [row_cap, 2 * inter]")
    row_cap, two_i = gu.shape
    inter = two_i // 2
    _need(counts, "counts", torch.int32, ndim=1)
    num_experts = counts.shape[0]
    _exact(offsets, "offsets", torch.int32, (num_experts + 1,))
    if hq is None:
        hq = torch.empty((row_cap, _code_cols(inter, fmt)), dtype=torch.uint8, device=gu.device)
    if hs is None:
        hs = torch.empty(_scale_shape(row_cap, inter, fmt), dtype=_scale_dtype(fmt), device=gu.device)
    _exact(hq, "hq", torch.uint8, (row_cap, _code_cols(inter, fmt)))
    _exact(hs, "hs", _scale_dtype(fmt), _scale_shape(row_cap, inter, fmt))
    dev = _same_device(gu, counts, offsets, hq, hs)
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}")
    _enqueue("moe_silu_mul_quant", dev, _ptr(gu), inter, _ptr(counts), _ptr(offsets), num_experts,
             row_cap, ACTS[act], float(clamp_limit), _fmt(fmt), _rounding(rounding), _ptr(hq),
             _ptr(hs))
    return hq, hs


def moe_topk_combine(y, pair_to_row, topk_w, t_live=None, out=None):
    """Top-k weighted sum of expert rows. Returns BF16 bits (int16) [t_cap, H]."""
    lib = load_library()
    yb = _bf16(y, "y")
    if yb.dim() != 2:
        raise ValueError("y must be [row_cap, hidden]")
    row_cap, hidden = yb.shape
    w = _need(topk_w, "topk_w", torch.float32, ndim=2)
    t_cap, topk = w.shape
    _min_numel(_need(pair_to_row, "pair_to_row", torch.int32), "pair_to_row", t_cap * topk)
    if out is None:
        out = torch.empty((t_cap, hidden), dtype=torch.int16, device=yb.device)
    ob = _shape(_bf16(out, "out"), "out", (t_cap, hidden))
    dev = _same_device(yb, pair_to_row, w, ob)
    _enqueue("moe_topk_combine", dev, _ptr(yb), row_cap, _ptr(pair_to_row), _ptr(w), t_cap,
             _live(t_live), topk, hidden, _ptr(ob))
    return out


def _weight_fmt(weight_fmt):
    if weight_fmt not in WEIGHT_FMTS:
        raise ValueError(f"weight_fmt must be one of {list(WEIGHT_FMTS)}")
    return WEIGHT_FMTS[weight_fmt]


def _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap, fmt, act, clamp_limit,
             rounding="divide", expert_start=0, expert_cap=0, weight_fmt="e4m3"):
    if act not in ACTS:
        raise ValueError(f"act must be one of {list(ACTS)}")
    return _Problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap or 0, _fmt(fmt),
                    ACTS[act], float(clamp_limit), _rounding(rounding), int(expert_start),
                    int(expert_cap), _weight_fmt(weight_fmt))


def moe_workspace_plan(num_experts, hidden, inter, topk, t_cap, align_rows=16, row_cap=0,
                       fmt="fp32", act="swiglu", clamp_limit=float("inf"), rounding="divide",
                       expert_start=0, expert_cap=0, weight_fmt="e4m3"):
    """Byte offsets of every intermediate in the forward workspace (dict)."""
    lib = load_library()
    prob = _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap, fmt, act,
                    clamp_limit, rounding, expert_start, expert_cap, weight_fmt)
    lay = _Layout()
    _check("moe_workspace_plan", lib.moe_workspace_plan(ctypes.byref(prob), ctypes.byref(lay)))
    return {name: getattr(lay, name) for name, _ in _Layout._fields_}


def moe_workspace_bytes(num_experts, hidden, inter, topk, t_cap, align_rows=16, row_cap=0,
                        fmt="fp32", act="swiglu", clamp_limit=float("inf"), rounding="divide",
                        expert_start=0, expert_cap=0, weight_fmt="e4m3"):
    lib = load_library()
    prob = _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap, fmt, act,
                    clamp_limit, rounding, expert_start, expert_cap, weight_fmt)
    return int(lib.moe_workspace_bytes(ctypes.byref(prob)))


def _check_layer_tensors(xb, topk_ids, w1, w1_scales, w2=None, w2_scales=None, weight_fmt="e4m3"):
    """Shapes and devices of the layer's inputs; returns (num_experts, inter, topk)."""
    t_cap, hidden = xb.shape
    _weight_fmt(weight_fmt)
    mx = weight_fmt == "mxfp4"
    _need(topk_ids, "topk_ids", torch.int32, ndim=2)
    if topk_ids.shape[0] != t_cap:
        raise ValueError(f"topk_ids has {topk_ids.shape[0]} rows, x has {t_cap}")
    _need(w1, "w1", torch.uint8, ndim=3)
    num_experts, two_i, h1 = w1.shape
    if h1 != (hidden // 2 if mx else hidden) or two_i % 256:
        raise ValueError(f"w1 must be [E, 2*inter, {hidden // 2 if mx else hidden}], got {tuple(w1.shape)}")
    inter = two_i // 2
    if mx:
        _exact(w1_scales, "w1_scales", torch.uint8, (num_experts, two_i, hidden // 32))
    else:
        _exact(w1_scales, "w1_scales", torch.float32,
               (num_experts, two_i // 128, hidden // 128))
    if w2 is not None:
        if mx:
            _exact(w2, "w2", torch.uint8, (num_experts, hidden, inter // 2))
            _exact(w2_scales, "w2_scales", torch.uint8,
                   (num_experts, hidden, inter // 32))
        else:
            _exact(w2, "w2", torch.uint8, (num_experts, hidden, inter))
            _exact(w2_scales, "w2_scales", torch.float32,
                   (num_experts, hidden // 128, inter // 128))
    return num_experts, inter, topk_ids.shape[1]


def moe_forward(x, topk_ids, topk_w, w1, w1_scales, w2, w2_scales, fmt="fp32", act="swiglu",
                clamp_limit=float("inf"), align_rows=16, row_cap=0, t_live=None, out=None,
                workspace=None, rounding="divide", expert_start=0, expert_cap=0,
                weight_fmt="e4m3"):
    """The whole expert layer. Returns (out BF16 bits int16 [t_cap, H], workspace uint8).
    ``topk_w=None`` weights every routed pair by one. ``weight_fmt="mxfp4"``:
    w1/w2 are packed E2M1 codes [E, rows, cols/2] with E8M0 scale bytes
    [E, rows, cols/32]; with it ``fmt="mxfp4"`` quantizes both activations to
    MXFP4."""
    lib = load_library()
    xb = _bf16(x, "x")
    if xb.dim() != 2:
        raise ValueError("x must be [t_cap, hidden]")
    t_cap, hidden = xb.shape
    num_experts, inter, topk = _check_layer_tensors(xb, topk_ids, w1, w1_scales, w2, w2_scales,
                                                    weight_fmt)
    if topk_w is None:
        topk_w = torch.ones((t_cap, topk), dtype=torch.float32, device=xb.device)
    _exact(topk_w, "topk_w", torch.float32, (t_cap, topk))
    prob = _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap, fmt, act,
                    clamp_limit, rounding, expert_start, expert_cap, weight_fmt)
    need = int(lib.moe_workspace_bytes(ctypes.byref(prob)))
    if need == 0:
        lay = _Layout()
        _check("moe_workspace_plan", lib.moe_workspace_plan(ctypes.byref(prob), ctypes.byref(lay)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=xb.device)
    _need(workspace, "workspace", torch.uint8)
    if out is None:
        out = torch.empty((t_cap, hidden), dtype=torch.int16, device=xb.device)
    ob = _shape(_bf16(out, "out"), "out", (t_cap, hidden))
    if t_live is not None:
        _exact(t_live, "t_live", torch.int32, (1,))
    dev = _same_device(xb, topk_ids, topk_w, w1, w1_scales, w2, w2_scales, ob, workspace, t_live)
    tens = _Tensors(_ptr(xb), _ptr(topk_ids), _ptr(topk_w), _live(t_live), _ptr(w1),
                    _ptr(w1_scales), _ptr(w2), _ptr(w2_scales), _ptr(ob))
    _enqueue("moe_forward", dev, ctypes.byref(prob), ctypes.byref(tens), _ptr(workspace),
             workspace.numel())
    return out, workspace


# Bytes of the library's static workspace behind moe_forward_noalloc (mirrors
# the header's MOE_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_forward_noalloc(x, topk_ids, topk_w, w1, w1_scales, w2, w2_scales, fmt="fp32",
                        act="swiglu", clamp_limit=float("inf"), align_rows=16, row_cap=0,
                        t_live=None, out=None, rounding="divide", expert_start=0, expert_cap=0,
                        weight_fmt="e4m3"):
    """moe_forward with the library's static per-device workspace instead of a
    caller buffer (for callers that cannot allocate; the call allocates nothing
    when ``out`` and ``topk_w`` are given). Calls on one device must not overlap.
    Returns out (BF16 bits int16 [t_cap, H])."""
    lib = load_library()
    xb = _bf16(x, "x")
    if xb.dim() != 2:
        raise ValueError("x must be [t_cap, hidden]")
    t_cap, hidden = xb.shape
    num_experts, inter, topk = _check_layer_tensors(xb, topk_ids, w1, w1_scales, w2, w2_scales,
                                                    weight_fmt)
    if topk_w is None:
        topk_w = torch.ones((t_cap, topk), dtype=torch.float32, device=xb.device)
    _exact(topk_w, "topk_w", torch.float32, (t_cap, topk))
    if out is None:
        out = torch.empty((t_cap, hidden), dtype=torch.int16, device=xb.device)
    ob = _shape(_bf16(out, "out"), "out", (t_cap, hidden))
    if t_live is not None:
        _exact(t_live, "t_live", torch.int32, (1,))
    dev = _same_device(xb, topk_ids, topk_w, w1, w1_scales, w2, w2_scales, ob, t_live)
    prob = _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap, fmt, act,
                    clamp_limit, rounding, expert_start, expert_cap, weight_fmt)
    tens = _Tensors(_ptr(xb), _ptr(topk_ids), _ptr(topk_w), _live(t_live), _ptr(w1),
                    _ptr(w1_scales), _ptr(w2), _ptr(w2_scales), _ptr(ob))
    _enqueue("moe_forward_noalloc", dev, ctypes.byref(prob), ctypes.byref(tens))
    return out


def moe_fc1_decode(x, topk_ids, w1, w1_scales, inter, fmt="fp32", act="swiglu",
                   clamp_limit=float("inf"), align_rows=16, row_cap=0, t_live=None,
                   workspace=None, rounding="divide", expert_start=0):
    """The decode path's first launch alone (routing, activation quantization and
    FC1 with SiLU(gate)*up), writing moe_forward's workspace. Returns the workspace."""
    lib = load_library()
    xb = _bf16(x, "x")
    if xb.dim() != 2:
        raise ValueError("x must be [t_cap, hidden]")
    t_cap, hidden = xb.shape
    num_experts, w_inter, topk = _check_layer_tensors(xb, topk_ids, w1, w1_scales)
    if w_inter != inter:
        raise ValueError("w1 shape disagrees with inter")
    prob = _problem(num_experts, hidden, inter, topk, t_cap, align_rows, row_cap,
                    fmt, act, clamp_limit, rounding, expert_start)
    need = int(lib.moe_workspace_bytes(ctypes.byref(prob)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=xb.device)
    _need(workspace, "workspace", torch.uint8)
    if t_live is not None:
        _exact(t_live, "t_live", torch.int32, (1,))
    dev = _same_device(xb, topk_ids, w1, w1_scales, workspace, t_live)
    tens = _Tensors(_ptr(xb), _ptr(topk_ids), None, _live(t_live), _ptr(w1), _ptr(w1_scales),
                    None, None, None)
    _enqueue("moe_fc1_decode", dev, ctypes.byref(prob), ctypes.byref(tens), _ptr(workspace),
             workspace.numel())
    return workspace


def moe_barrier_timeouts():
    """Waits at the one-launch decode layer's grid barrier that gave up on the
    current device (sticky count; nonzero means some launch's outputs are unreliable)."""
    lib = load_library()
    n = ctypes.c_uint32(0)
    _check("moe_barrier_timeouts", lib.moe_barrier_timeouts(ctypes.byref(n)))
    return int(n.value)


def moe_barrier_spin_limit(polls):
    """Sets the polls per wait of the one-launch decode layer's grid barrier for
    later launches (negative: every wait gives up at once); returns the old value."""
    return int(load_library().moe_barrier_spin_limit(int(polls)))
