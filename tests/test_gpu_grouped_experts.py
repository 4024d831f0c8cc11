"""Grouped products with more experts than a lane of the scheduler has lanes for, and than the
weights' gradient sorts (512), up to the 1024 that a shape may have: every output element
against float64 (tolerances of test_gpu_grouped_split), the same bits from a second call."""
import numpy as np
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_grouped_split import check, problem

pytestmark = pytest.mark.gpu


def draw(E, rows, skew, seed):
    rng = np.random.default_rng(seed)
    p = (1.0 + np.arange(E)) ** -skew
    return rng.multinomial(rows, rng.permutation(p / p.sum())).tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,skew", [(37, 0.0), (6000, 1.0), (90000, 0.5)])
@pytest.mark.parametrize("E", [257, 300, 511, 512, 513, 1000, 1024])
def test_many_experts(E, rows, skew, dtype):
    counts = draw(E, rows, skew, E + rows)
    shape, lay, seg, r, d, w, ws = problem(counts, 72, 136, seed=E)

    def run():
        out = torch.full((shape.N, 136), float("nan"), dtype=dtype, device="cuda")
        drows = torch.full((shape.N, 72), float("nan"), dtype=dtype, device="cuda")
        dw = torch.full((E, 136, 72), float("nan"), dtype=dtype, device="cuda")
        moe.moe_grouped_gemm(r, lay, shape, w, out, ws)
        moe.moe_grouped_gemm_input_grad(d, lay, shape, w, drows, ws)
        moe.moe_grouped_gemm_weight_grad(d, r, lay, shape, dw, ws)
        return out, drows, dw

    out, drows, dw = run()
    assert moe.moe_get_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip((out, drows, dw), run()))
    R, D, M = r.double(), d.double(), w.double()
    for e, s in enumerate(seg):
        if counts[e] == 0:
            assert (dw[e] == 0).all()
            continue
        check(out[s], R[s], M[e].T)
        check(drows[s], D[s], M[e])
        check(dw[e], D[s].T, R[s])
