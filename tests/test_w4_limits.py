"""Refusals of the 4-bit products and of the helpers that make their weights: answered on the
host, before anything is launched."""
import types

import pytest
import torch

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe

bf = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load()


class OnDevice(torch.Tensor):
    """A host tensor that passes for a device tensor as long as nothing is launched."""
    is_cuda = property(lambda self: True)


def on_device(*size, dtype=bf):
    return torch.zeros(*size, dtype=dtype).as_subclass(OnDevice)


def test_packed_weights_are_checked_like_other_operands(lib, monkeypatch):
    """Their memory is the device's, and as much as the products read of it."""
    s = moe.Shape(4, 128, 8, 2, 1, 64)
    lay = moe.Layout.__new__(moe.Layout)
    lay.shape, lay.c = s, moe.MoeLayout()
    st = types.SimpleNamespace(cuda_stream=0)
    ws = on_device(256, dtype=torch.uint8)
    calls = []
    fake = types.SimpleNamespace(moe_w4_gemm=lambda *a: calls.append(a) or 0,
                                 moe_w4_gated_gemm=lambda *a: calls.append(a) or 0,
                                 moe_w4_packed_bytes=lib.moe_w4_packed_bytes)

    for gated in (False, True):
        w4 = moe.W4Matrices(8, 64, 128, 64, gated, device="cpu")
        size = w4.data.numel()
        x, y = on_device(8, 128), on_device(8, 64)

        def product():
            with monkeypatch.context() as m:
                m.setattr(moe, "load", lambda: fake)
                if gated:
                    moe.moe_w4_gated_gemm(x, lay, s, w4, None, y, ws, st)
                else:
                    moe.moe_w4_gemm(x, lay, s, w4, y, ws, st)

        with pytest.raises(ValueError, match="device tensors"):
            product()
        for data in (on_device(size - 1, dtype=torch.uint8), on_device(size, dtype=torch.int8),
                     on_device(2 * size, dtype=torch.uint8)[::2]):
            w4.data = data
            with pytest.raises(ValueError, match="w4: expected|contiguous"):
                product()
        assert not calls
        w4.data = on_device(size, dtype=torch.uint8)
        product()
        assert calls.pop()
