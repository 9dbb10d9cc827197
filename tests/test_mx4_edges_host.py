"""Host-only checks of the routing and 4-bit entry points at the edges of their
arguments. Meta tensors have a shape and no memory; the GPU check comes last."""

import pytest
import torch

import block_fp8_mixture_amd as moe


def _meta(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_int32_are_refused():
    """The C ABI takes int32 sizes: 2**32 + n is not n."""
    u8 = torch.uint8
    for half in (1 << 30, (1 << 31) + 16):  # bytes of a row of codes
        with pytest.raises(ValueError, match="2\\*\\*31"):
            moe.moe_mxfp4_dequant(_meta((1, half), u8), _meta((1, half // 16), u8))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_mxfp4_dequant(_meta((1, (1 << 30) - 16), u8), _meta((1, (1 << 26) - 1), u8))
    for tokens in (1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            moe.moe_route(_meta((tokens, 1), torch.float32), 1)
    l = _meta((3, 8), torch.float32)
    with pytest.raises(ValueError, match="2\\*\\*31"):
        moe.moe_route(l, (1 << 32) + 2)
    for name in ("num_groups", "top_groups", "group_top"):
        for v in ((1 << 31), (1 << 32) + 1, 1 - (1 << 32)):
            with pytest.raises(ValueError, match="2\\*\\*31"):
                moe.moe_route(l, 2, **{name: v})
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_route(l, 2)
