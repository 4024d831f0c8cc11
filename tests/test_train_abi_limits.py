"""Host-side refusals of the grouped products at the ends of their sizes: answered without a
GPU, before any launch."""
import ctypes

import pytest

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe

INVALID, UNSUPPORTED = 1, 2
OK16 = ctypes.c_void_p(0x10000)  # never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load()


def calls(lib, shape, ws=OK16, rows=OK16):
    """The three products of this shape on 64 x 64 matrices."""
    c, n = ctypes.byref(shape.c()), ctypes.c_size_t(moe.moe_workspace_bytes(shape))
    lay = ctypes.byref(moe.MoeLayout(*([0x20000] * len(moe.LAYOUT_FIELDS))))
    yield lib.moe_grouped_gemm(rows, lay, c, 64, 64, OK16, OK16, 0, ws, n, None)
    yield lib.moe_grouped_gemm_input_grad(rows, lay, c, 64, 64, OK16, OK16, 0, ws, n, None)
    yield lib.moe_grouped_gemm_weight_grad(rows, OK16, lay, c, 64, 64, OK16, 1, 0, ws, n, None)


@pytest.mark.parametrize("N,k", [(2 ** 31 - 2 ** 20, 1), (2 ** 31 - 1, 1), (2 ** 28 - 2 ** 17, 8)])
def test_more_rows_than_their_blocks_can_be_counted(lib, N, k):
    shape = moe.Shape(N, 64, 8, k, 2, 64)
    assert moe.moe_workspace_bytes(shape) > 0  # other calls take it
    # the size is refused before the missing tensor is
    assert all(status == UNSUPPORTED for status in calls(lib, shape, rows=None))
    shape = moe.Shape((2 ** 31 - 2 ** 20 - 1) // k, 64, 8, k, 2, 64)
    assert all(status == INVALID for status in calls(lib, shape, rows=None))


def test_workspace_off_its_words(lib):
    """The tile counters and the error word are 32-bit atomics."""
    shape = moe.Shape(64, 64, 8, 2, 2, 64)
    for at in (0x10001, 0x10002, 0x10003):
        assert all(status == INVALID for status in calls(lib, shape, ws=ctypes.c_void_p(at)))
