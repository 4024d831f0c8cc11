"""4-bit products at the ends of what their layouts and streams may be, with the tolerances of the
operators' other tests."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_w4 import Case

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
INVALID = 1


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,rows", [(8, 4096), (1024, 3000), (700, 16384)])
def test_segments_that_overlap_are_reported(E, rows, gated):
    """No more passes than the rows can fill are run: their number would leave 32 bits for large
    ones.  What is written is within the rows, and the next call is as it should be."""
    c = Case(rows, E, 1, 128, 40, 128, gated, seed=3)
    want = c.run()
    c.check(want)
    offsets, counts = c.lay["expert_offsets"].clone(), c.lay["expert_counts"].clone()
    c.lay["expert_offsets"].zero_()
    c.lay["expert_counts"].fill_(rows)
    pad = 4096
    flat = torch.full((want.numel() + 2 * pad,), 7.0, dtype=bf, device="cuda")
    c.run(out=flat[pad:-pad].view(want.shape))
    assert moe.moe_get_error(c.ws) == INVALID
    assert (flat[:pad] == 7.0).all() and (flat[-pad:] == 7.0).all()
    c.lay["expert_offsets"].copy_(offsets)
    c.lay["expert_counts"].copy_(counts)
    c.ws[:4] = 0
    out = c.run()
    assert torch.equal(out, want) and moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("E,rows", [(1, 129), (4, 320), (1024, 1024), (5, 17), (33, 40)])
def test_the_most_passes_that_a_layout_can_have(E, rows):
    """One row to each expert but the last: not taken for an overlap."""
    counts = [1] * (E - 1) + [0]
    counts[-1] = rows - sum(counts)
    c = Case(rows, E, 1, 256, 40, 64, False, seed=4, counts=counts)
    c.check(c.run())
