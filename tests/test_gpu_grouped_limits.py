"""Grouped products at the most rows (2^31 - 2^20 - 1) and the widest matrices (2^31 - 8) that
they take: block counts, coordinates and contractions at the end of 32 bits.  All values are
powers of two, so that every element is known: short sums are exact, and sums over 2^31 terms
are rounded to nearest in fp32 a few times (2^-24 each) and once to bf16 (2^-8).  Up to 70 GB
of device memory."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_grouped_seconds import layout_of

pytestmark = pytest.mark.gpu
MOST, WIDEST = 2 ** 31 - 2 ** 20 - 1, 2 ** 31 - 8
BF = dict(dtype=torch.bfloat16, device="cuda")


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def all_equal(t, value):
    """Without a mask of the whole tensor."""
    return t.amin().item() == value and t.amax().item() == value


def close(got, want):
    """A sum over 2^31 terms of the same sign."""
    bound = 2.0 ** -22 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0)
    assert ((got.double() - want).abs() <= bound * want).all()


@pytest.mark.parametrize("counts", [[MOST], [300, MOST - 305, 5]], ids=str)
def test_most_rows(counts):
    shape, lay, at = layout_of(counts)
    rows, out = torch.ones(MOST, 8, **BF), torch.empty(MOST, 8, **BF)
    w = torch.ones(shape.E, 8, 8, **BF) * 2.0 ** torch.arange(shape.E, device="cuda")[:, None, None]
    ws = moe.workspace(shape)
    for call in (moe.moe_grouped_gemm, moe.moe_grouped_gemm_input_grad):
        out.fill_(7.0)
        call(rows, lay, shape, w.bfloat16(), out, ws)
        assert moe.moe_get_error(ws) == 0
        for e in range(shape.E):
            assert all_equal(out[at[e]:at[e + 1]], 8.0 * 2 ** e)
    dw = torch.empty(shape.E, 8, 8, device="cuda")
    moe.moe_grouped_gemm_weight_grad(rows, rows, lay, shape, dw, ws)
    assert moe.moe_get_error(ws) == 0
    close(dw, torch.tensor(counts, dtype=torch.float64, device="cuda")[:, None, None])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("back", [False, True], ids=["forward", "rows' gradient"])
def test_longest_contraction(back, dtype):
    shape, lay, _ = layout_of([3])
    scale = 2.0 ** torch.arange(3, device="cuda")[:, None]
    a = torch.empty(3, WIDEST, **BF).copy_(scale.bfloat16().expand(3, WIDEST))
    w = torch.ones(1, *((WIDEST, 8) if back else (8, WIDEST)), **BF)
    out = torch.empty(3, 8, dtype=dtype, device="cuda")
    ws = moe.workspace(shape)
    call = moe.moe_grouped_gemm_input_grad if back else moe.moe_grouped_gemm
    call(a, lay, shape, w, out, ws)
    assert moe.moe_get_error(ws) == 0
    close(out, (scale * WIDEST).double().expand(3, 8))


@pytest.mark.parametrize("back", [False, True], ids=["forward", "rows' gradient"])
def test_widest_output(back):
    shape, lay, _ = layout_of([1])
    w = torch.ones(1, *((8, WIDEST) if back else (WIDEST, 8)), **BF)
    out = torch.empty(1, WIDEST, **BF)
    ws = moe.workspace(shape)
    call = moe.moe_grouped_gemm_input_grad if back else moe.moe_grouped_gemm
    call(torch.ones(1, 8, **BF), lay, shape, w, out, ws)
    assert moe.moe_get_error(ws) == 0
    assert all_equal(out, 8.0)


@pytest.mark.parametrize("wide_in", [False, True], ids=["C_out", "C_in"])
def test_widest_weights_gradient(wide_in):
    shape, lay, _ = layout_of([3])
    wide, narrow = torch.ones(3, WIDEST, **BF), torch.ones(3, 8, **BF)
    dw = torch.empty(1, *((8, WIDEST) if wide_in else (WIDEST, 8)), **BF)
    dout, rows = (narrow, wide) if wide_in else (wide, narrow)
    ws = moe.workspace(shape)
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    assert moe.moe_get_error(ws) == 0
    assert all_equal(dw, 3.0)
