"""A weights' gradient whose one long expert keeps a pair of CTAs busy for more than a second:
the waits that last as long as its contraction (the scheduler's for the next tile, the block
end's for the last rows) are no timeouts.

All values are powers of two, so that every partial sum of 512 terms is exact; the sums of
those and the last, shorter one are rounded to nearest, 2^-24 each, a handful of them."""
import pytest
import torch

from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def layout_of(counts):
    """A layout with the segments alone: the products read nothing else of it."""
    shape = moe.Shape(sum(counts), 8, len(counts), 1, 1, 8)
    lay = moe.Layout.__new__(moe.Layout)
    small = moe.Layout(moe.Shape(1, 8, len(counts), 1, 1, 8))
    lay.shape, lay.tensors, lay.c = shape, small.tensors, small.c
    at = torch.tensor([0] + counts).cumsum(0)
    lay["expert_counts"].copy_(torch.tensor(counts))
    lay["expert_offsets"].copy_(at)
    return shape, lay, at.tolist()


def test_contraction_of_seconds():
    # more experts than there are pairs: no tile is shared, and the scheduler hands some out
    counts = [3] * 40 + [(1 << 29) + 5] + [2] * 60
    shape, lay, at = layout_of(counts)
    rows = torch.ones(shape.N, 8, dtype=torch.bfloat16, device="cuda")
    dout = torch.full_like(rows, 0.5)
    dw = torch.empty(shape.E, 8, 8, device="cuda")
    ws = moe.workspace(shape)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    end.record()
    assert moe.moe_get_error(ws) == 0
    print(f"{start.elapsed_time(end):.0f} ms")
    want = torch.tensor(counts, dtype=torch.float64, device="cuda") * 0.5
    assert ((dw.double() - want[:, None, None]).abs() <= 2.0 ** -22 * want[:, None, None]).all()
