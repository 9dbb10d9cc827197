"""Host-only checks of the routing and 4-bit entry points at the edges of their
arguments. Meta tensors have a shape and no memory; the GPU check comes last."""

import types

import pytest
import torch

import block_fp8_mixture_amd as moe
from block_fp8_mixture_amd import _binding as B


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


@pytest.mark.parametrize("current", [0, 1])
def test_calls_switch_to_the_tensors_device_and_take_its_stream(monkeypatch, current):
    """With the tensors on device 1: entered if another device is current, for
    the call alone, and the stream is device 1's."""
    entered, state = [], {"current": current}

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)
            self.before, state["current"] = state["current"], self.device.index

        def __exit__(self, *_):
            state["current"] = self.before

    seen = []
    lib = types.SimpleNamespace(f=lambda *args: seen.append((args, state["current"])) or 0)
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_current_device", lambda: state["current"])
    monkeypatch.setattr(B, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", Device)
    device = torch.device("cuda", 1)
    B._enqueue("f", device, 7, 8)
    assert seen == [((7, 8, 1001), 1)]
    assert entered == ([] if current == 1 else [device]) and state["current"] == current


def test_a_failed_call_leaves_the_current_device(monkeypatch):
    """A refusal on another device raises and the device is as before."""
    left = []

    class Device:
        def __init__(self, device):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *_):
            left.append(True)

    monkeypatch.setattr(B, "_lib", types.SimpleNamespace(f=lambda *args: 1))
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    with pytest.raises(moe.MoeError, match="invalid argument"):
        B._enqueue("f", torch.device("cuda", 1))
    assert left == [True]


def test_product_of_rows_past_32768_is_refused():
    lib, fake = moe.load_library(), 0x1000  # never dereferenced: the refusal comes first
    for k, status in ((32768, 0), (32896, 2)):
        assert lib.moe_grouped_gemm_mxfp4(fake, fake, 4, 64, None, 1, fake, fake, fake, fake, 0, 4, 0, 0, 128, k, fake,
                                          None) == status
