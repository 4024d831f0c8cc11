"""Grouped products and their gradients against a float64 product of the same
bf16 values, at segment lengths, widths and types where the tiling can go wrong.

Tolerances.  A bf16 output rounds once: relative error 2^-9 an element, and its
fp32 accumulation stays far below that.  An fp32 output is a sum of bf16
products (exact in fp32) added up in chains of 512 terms with truncation, then
to nearest: every addition loses at most 2^-23 of a partial sum, so the error is
below (512 + K / 512) * 2^-23 of the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def make_layout(counts, k=1):
    """A layout whose expert e has counts[e] rows (the order of the tokens does
    not matter to the products)."""
    R, E = int(sum(counts)), len(counts)
    shape = moe.Shape(R, 8, E, 1, 1, 8)
    lay = moe.Layout(shape)
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    lay["expert_counts"].copy_(torch.tensor(counts, dtype=torch.int32))
    lay["expert_offsets"].copy_(torch.from_numpy(offs))
    return shape, lay, offs


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()


def check(got, ref, mag, terms):
    """got against float64 ref; mag: the sum of the terms' magnitudes."""
    assert torch.isfinite(got.float()).all()
    err = (got.double() - ref).abs()
    bound = (512 + terms / 512) * 2.0 ** -23 * mag
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * ref.abs()
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0.0, f"{worst} over the bound, at an error of {err.max().item()}"


COUNTS = [
    [1],
    [0, 0, 3, 0],
    [16, 64, 256, 512],
    [15, 17, 63, 65, 1, 0, 255, 257],
    [700, 0, 1, 1283, 90],
    [0, 0],
]
WIDTHS = [(8, 8), (64, 64), (128, 256), (264, 72), (520, 1032)]


def problem(counts, ci, co, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    shape, lay, offs = make_layout(counts)
    R, E = shape.N, shape.E
    rows, dout = normal(gen, R, ci), normal(gen, R, co, std=0.1)
    w = normal(gen, E, co, ci, std=ci ** -0.5)
    return shape, lay, offs, rows, dout, w, moe.workspace(shape)


def segments(offs):
    return [slice(int(a), int(b)) for a, b in zip(offs[:-1], offs[1:])]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ci,co", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_products_against_float64(counts, ci, co, dtype):
    shape, lay, offs, rows, dout, w, ws = problem(counts, ci, co)
    R, E = shape.N, shape.E
    out = torch.full((R, co), float("nan"), dtype=dtype, device="cuda")
    drows = torch.full((R, ci), float("nan"), dtype=dtype, device="cuda")
    dw = torch.full((E, co, ci), float("nan"), dtype=dtype, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    moe.moe_grouped_gemm_input_grad(dout, lay, shape, w, drows, ws)
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_error(ws) == 0
    r, d, m = rows.double(), dout.double(), w.double()
    for e, s in enumerate(segments(offs)):
        check(out[s], r[s] @ m[e].T, r[s].abs() @ m[e].T.abs(), ci)
        check(drows[s], d[s] @ m[e], d[s].abs() @ m[e].abs(), co)
        check(dw[e], d[s].T @ r[s], d[s].T.abs() @ r[s].abs(), int(offs[e + 1] - offs[e]))


def test_long_contractions_keep_fp32_precision():
    """8192 positive terms: additions that truncated all the way would be off by
    some 1e-4 of the sum, the bound of the chained sum is 16 times lower than
    that of a single chain."""
    K = 8192
    shape, lay, offs, _, _, _, ws = problem([K], 8, 8)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rows, dout = normal(gen, K, 128).abs(), normal(gen, K, 256).abs()
    dw = torch.empty(1, 256, 128, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    ref = dout.double().T @ rows.double()
    check(dw[0], ref, ref, K)
    # and on average far below the bound
    assert ((dw[0].double() - ref).abs() / ref).mean().item() < 4e-6


def test_accumulate_adds_in_fp32():
    counts = [70, 0, 129]
    shape, lay, offs, rows, dout, w, ws = problem(counts, 264, 136)
    fresh = torch.empty(3, 136, 264, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, fresh, ws)
    start = torch.randn(3, 136, 264, device="cuda")
    acc = start.clone()
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, acc, ws, accumulate=True)
    assert torch.equal(acc, start + fresh)      # one fp32 addition an element
    assert torch.equal(acc[1], start[1])        # no rows: nothing is added


def test_neighbours_values_do_not_leak():
    """Inf and NaN in one expert's rows stay out of every other expert's outputs,
    also where a block of the contraction runs past the segment's end."""
    counts = [37, 21, 70]
    shape, lay, offs, rows, dout, w, ws = problem(counts, 136, 72)
    clean = torch.empty(3, 72, 136, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, clean, ws)
    s = segments(offs)[1]
    rows[s], dout[s] = float("inf"), float("nan")
    w[1] = float("nan")
    dw = torch.empty_like(clean)
    out = torch.empty(shape.N, 72, device="cuda")
    drows = torch.empty(shape.N, 136, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    moe.moe_grouped_gemm_input_grad(dout, lay, shape, w, drows, ws)
    for e in (0, 2):
        assert torch.equal(dw[e], clean[e])
        assert torch.isfinite(out[segments(offs)[e]]).all()
        assert torch.isfinite(drows[segments(offs)[e]]).all()
    assert torch.isnan(dw[1]).all()


def test_same_results_every_run():
    counts = [300, 5, 0, 1000]
    shape, lay, offs, rows, dout, w, ws = problem(counts, 520, 264)
    a, b = (torch.empty(4, 264, 520, device="cuda") for _ in range(2))
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, a, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, b, ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_no_rows():
    shape, lay, offs, rows, dout, w, ws = problem([0, 0], 64, 64)
    dw = torch.full((2, 64, 64), 3.0, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws, accumulate=True)
    assert (dw == 3.0).all()
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    assert (dw == 0.0).all()


def test_segments_outside_the_rows_are_reported():
    shape, lay, offs, rows, dout, w, ws = problem([40, 24], 64, 64)
    lay["expert_counts"][1] = 25
    out = torch.zeros(64, 64, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
    assert moe.moe_get_error(ws) == 1
    assert (out[40:] == 0).all() and (out[:40] != 0).any()


def test_refusals():
    shape, lay, offs, rows, dout, w, ws = problem([40, 24], 64, 72)
    out = torch.empty(64, 72, device="cuda")
    with pytest.raises(ValueError, match="rows: expected shape"):
        moe.moe_grouped_gemm(rows[:63], lay, shape, w, out, ws)
    with pytest.raises(ValueError, match="out: expected bf16 or fp32"):
        moe.moe_grouped_gemm(rows, lay, shape, w, out.half(), ws)
    with pytest.raises(ValueError, match="rows: expected torch.bfloat16"):
        moe.moe_grouped_gemm(rows.half(), lay, shape, w, out, ws)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_grouped_gemm(dout, lay, shape, w.transpose(1, 2), out[:, :64].contiguous(), ws)
    dw = torch.empty(2, 72, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws, accumulate=True)
    assert e.value.status == 2
    odd = torch.empty(2, 60, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grouped_gemm(rows, lay, shape, odd, out.new_empty(64, 60), ws)
    assert e.value.status == 2
