"""Grouped products with few tiles and long contractions, which several CTA pairs share:
against a float64 product of the same bf16 values.

Tolerances.  An fp32 output's terms are added up in chains of 512 with truncation, the
chains and the pairs' sums to nearest: every addition loses at most 2^-23 of the sum of
the terms' magnitudes, so the error is below (512 + K / 512 + 4) * 2^-23 of that sum.  A
bf16 output's chains are a pair's whole share, at most K terms, and it rounds once, by at
most 2^-9 of the value (2^-8 with room for the fp32 error in it)."""
import numpy as np
import pytest
import torch

from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def problem(counts, ci, co, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    R, E = int(sum(counts)), len(counts)
    shape = moe.Shape(R, 8, E, 1, 1, 8)
    lay = moe.Layout(shape)
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    lay["expert_counts"].copy_(torch.tensor(counts, dtype=torch.int32))
    lay["expert_offsets"].copy_(torch.from_numpy(offs))

    def normal(*size, std=1.0):
        return (torch.randn(*size, generator=gen, device="cuda") * std).bfloat16()

    return (shape, lay, [slice(int(a), int(b)) for a, b in zip(offs[:-1], offs[1:])],
            normal(R, ci), normal(R, co, std=0.1), normal(E, co, ci, std=ci ** -0.5),
            moe.workspace(shape))


def check(got, a, b):
    """got against a @ b, bf16 operands as float64."""
    K = a.shape[1]
    ref, mag = a @ b, a.abs() @ b.abs()
    chain = 512 if got.dtype == torch.float32 else K
    bound = (chain + K / 512 + 4) * 2.0 ** -23 * mag
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs()
    assert torch.isfinite(got.float()).all()
    worst = ((got.double() - ref).abs() - bound).max().item() if got.numel() else -1.0
    assert worst <= 0.0, f"{worst} over the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,width", [(1024, 8), (1032, 264), (2056, 72), (4096, 520), (7000, 136)])
@pytest.mark.parametrize("counts", [[1], [3, 0, 5], [33], [130, 7], [257]], ids=str)
def test_long_contractions_of_few_rows(counts, K, width, dtype):
    shape, lay, seg, rows, _, w, ws = problem(counts, K, width)
    out = torch.full((shape.N, width), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    shape2, lay2, _, _, dout, w2, ws2 = problem(counts, width, K, seed=1)
    drows = torch.full((shape.N, width), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_input_grad(dout, lay2, shape2, w2, drows, ws2)
    assert moe.moe_get_error(ws) == 0 and moe.moe_get_error(ws2) == 0
    for e, s in enumerate(seg):
        check(out[s], rows[s].double(), w[e].double().T)
        check(drows[s], dout[s].double(), w2[e].double())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ci,co", [(8, 8), (72, 136), (264, 520)])
@pytest.mark.parametrize("counts", [[2048], [4099, 1], [0, 3000, 17], [1500, 513, 2049]], ids=str)
def test_weight_gradients_of_many_rows(counts, ci, co, dtype):
    shape, lay, seg, rows, dout, _, ws = problem(counts, ci, co)
    dw = torch.full((shape.E, co, ci), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    assert moe.moe_get_error(ws) == 0
    for e, s in enumerate(seg):
        check(dw[e], dout[s].double().T, rows[s].double())


def test_accumulate():
    shape, lay, seg, rows, dout, _, ws = problem([0, 3001, 200], 136, 264)
    fresh = torch.empty(3, 264, 136, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, fresh, ws)
    start = torch.randn(3, 264, 136, device="cuda")
    start[0, 0, 0] = -0.0
    acc = start.clone()
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, acc, ws, accumulate=True)
    assert torch.equal(acc, start + fresh)      # one fp32 addition an element
    assert torch.equal(acc[0].view(torch.int32), start[0].view(torch.int32))  # nothing added


def test_same_results_every_run_and_stream():
    shape, lay, seg, rows, dout, w, ws = problem([1, 20], 4096, 264)
    out = [torch.empty(21, 264, device="cuda") for _ in range(6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(out):
        moe.moe_grouped_gemm(rows, lay, shape, w, o, ws, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(out[0], o) for o in out[1:])


def test_rows_of_other_experts_stay_as_they_were():
    """A row block of 256 runs into the next expert's rows: neither their values get into
    this expert's sums nor its stores into them."""
    counts = [5, 9]
    shape, lay, seg, rows, dout, w, ws = problem(counts, 2048, 72)
    clean = torch.empty(14, 72, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, clean, ws)
    lay["expert_counts"][1] = 0
    rows[5:] = float("nan")
    out = torch.full((14, 72), 7.0, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    assert torch.equal(out[:5], clean[:5]) and (out[5:] == 7.0).all()


def test_more_row_blocks_than_rows_allow_are_reported():
    """Experts whose segments overlap are no layout; tiles past those that the rows allow
    for are not launched."""
    shape, lay, seg, rows, dout, w, ws = problem([2, 0, 0, 0], 2048, 72)
    lay["expert_counts"].fill_(2)
    lay["expert_offsets"].zero_()
    moe.moe_grouped_gemm(rows, lay, shape, w, torch.zeros(2, 72, device="cuda"), ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 1    # 4 blocks of 2 rows


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [8, 40, 64, 104, 128, 136, 192, 264, 320, 360, 384, 392])
def test_widths_of_the_last_column_block(width, dtype):
    """Column blocks of 256 and what is left: from 8 columns to a whole block."""
    counts = [300, 5, 270]
    shape, lay, seg, rows, dout, w, ws = problem(counts, 200, width)
    out = torch.full((shape.N, width), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    shape2, lay2, _, rows2, dout2, w2, ws2 = problem(counts, width, 200, seed=1)
    drows = torch.full((shape.N, width), float("nan"), dtype=dtype, device="cuda")
    dw = torch.full((3, 200, width), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm_input_grad(dout2, lay2, shape2, w2, drows, ws2)
    moe.moe_grouped_gemm_weight_grad(dout2, rows2, lay2, shape2, dw, ws2)
    assert moe.moe_get_error(ws) == 0 and moe.moe_get_error(ws2) == 0
    for e, s in enumerate(seg):
        check(out[s], rows[s].double(), w[e].double().T)
        check(drows[s], dout2[s].double(), w2[e].double())
        check(dw[e], dout2[s].double().T, rows2[s].double())
