"""Refusals of the 4-bit products and of the helpers that make their weights: answered on the
host, before anything is launched."""
import ctypes
import types

import pytest
import torch

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
OK16 = ctypes.c_void_p(0x10000)  # never dereferenced on the host
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


@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("C_out,C_in", [
    (1 << 30, 32), ((1 << 28) + 8, 128), (2 ** 31 - 8, 64), (8, (1 << 28) + 128),
    (8, 2 ** 31 - 128), (1 << 28, 1 << 28), (1 << 27, 1 << 24),
])
def test_sides_past_those_that_are_counted_in_32_bits(lib, C_out, C_in, gated):
    """Twice C_out from 2^30 on is negative, and so are the rows of a last slab and the weights of
    a last chunk near 2^31: the largest sides are refused, as is more than 64 bits of bytes.  A call
    that passes the check of its sizes stops at the missing weights."""
    s = moe.Shape(4, 64, 1024, 2, 1, 64)
    lay = ctypes.byref(moe.MoeLayout(*([0x20000] * len(moe.LAYOUT_FIELDS))))
    n = moe.moe_w4_workspace_bytes(s)

    def calls(C_out, C_in):
        m = ctypes.byref(moe.MoeW4Matrix(C_out, C_in, 32, gated))
        yield lib.moe_w4_pack(OK16, OK16, m, 1024, None, None)
        if gated:
            yield lib.moe_w4_gated_gemm(OK16, lay, s.ref, m, None, None, OK16, OK16, n, None)
        else:
            yield lib.moe_w4_gemm(OK16, lay, s.ref, m, None, OK16, 0, OK16, n, None)

    m = ctypes.byref(moe.MoeW4Matrix(C_out, C_in, 32, gated))
    assert lib.moe_w4_packed_bytes(m, 1024) == 0
    assert list(calls(C_out, C_in)) == [UNSUPPORTED, UNSUPPORTED]
    assert list(calls(1 << 28, 32)) == [INVALID, INVALID]
    assert list(calls(8, 1 << 28)) == [INVALID, INVALID]
    # one expert's may be as large as a gated block's
    one = ctypes.byref(moe.MoeW4Matrix(1 << 28, 32, 32, gated))
    assert lib.moe_w4_packed_bytes(one, 1) == (1 << 28) * (1 + gated) // 32 * (32 * 64 + 32 * 2 * 4)


@pytest.mark.parametrize("C_in,group", [
    (128, 96), (128, 48), (7168, 127), (64, 128), (160, 64), (96, 128), (128, 0), (128, -64),
    (128, 16), (256, 256), (128, 64.5), (192, 128),
])
def test_groups_are_those_asked_for(lib, monkeypatch, C_in, group):
    """No other group stands in for one that the products do not have, here or in a layer."""
    monkeypatch.setattr(moe, "load", lambda: pytest.fail("reached the library"))
    with pytest.raises(ValueError, match="group: expected 32, 64 or 128"):
        moe.quantize_w4(torch.zeros(2, 8, C_in, dtype=bf), group)
    s = moe.Shape(4, C_in, 2, 1, 1, 128)
    gate, down = torch.zeros(2, 128, C_in, dtype=bf), torch.zeros(2, C_in, 128, dtype=bf)
    with pytest.raises(ValueError, match="group: expected 32, 64 or 128"):
        moe.MoELayer(s, gate, gate, down, device="cpu", w4=group)
