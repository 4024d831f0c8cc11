"""4-bit products in each form of the kernel: 16, 32 and 64 rows a pass by groups of 32, 64 and 128
weights, plain and gated, on segments of even and uneven lengths, with the tolerances of the
operators' other tests."""
import pytest
import torch

from test_gpu_w4 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [
    [9, 12, 5, 16], [3, 0, 33, 1],                    # 16 rows a pass
    [24, 32, 17, 31], [1, 70, 0, 20], [33, 33, 33, 33],  # 32
    [64, 40, 65, 48], [0, 200, 7, 1],                 # 64, of groups of 32 32
])
def test_rows_of_a_pass(counts, group, gated):
    c = Case(sum(counts), 4, 1, 640, 264, group, gated, seed=30, counts=counts)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run(), out)
    if not gated:
        c.check(c.run(torch.float32))
