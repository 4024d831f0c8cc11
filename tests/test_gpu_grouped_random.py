"""Grouped products and gradients on seeded random sizes: experts, segment lengths (skewed,
empty, one row), widths, contractions and types drawn together, so that combinations that no
hand-picked case names are checked too: every output element against float64 (tolerances of
test_gpu_grouped_split), no element left unwritten, the same bits from a second call."""
import numpy as np
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_grouped_split import check, problem

pytestmark = pytest.mark.gpu


def draw(i):
    rng = np.random.default_rng(4200 + i)
    E = int(rng.choice([1, 2, 5, 8, 31, 32, 33, 64, 100, 256]))
    rows = int(2 ** rng.uniform(0, 12))
    p = (1.0 + np.arange(E)) ** -float(rng.choice([0.0, 1.0, 2.0]))
    counts = rng.multinomial(rows, rng.permutation(p / p.sum())).tolist()

    def width():
        return 8 * max(1, int(2 ** rng.uniform(0, 9.3)) // 2)

    ci, co = width(), width()
    while E * ci * co > 1 << 25:
        ci, co = (ci // 16 * 8 or 8, co) if ci > co else (ci, co // 16 * 8 or 8)
    dtype = torch.float32 if rng.random() < 0.5 else torch.bfloat16
    return counts, ci, co, dtype


@pytest.mark.parametrize("i", range(48))
def test_random_sizes(i):
    counts, ci, co, dtype = draw(i)
    shape, lay, seg, rows, dout, w, ws = problem(counts, ci, co, seed=i)

    def run():
        out = torch.full((shape.N, co), float("nan"), dtype=dtype, device="cuda")
        drows = torch.full((shape.N, ci), float("nan"), dtype=dtype, device="cuda")
        dw = torch.full((shape.E, co, ci), float("nan"), dtype=dtype, device="cuda")
        moe.moe_grouped_gemm(rows, lay, shape, w, out, ws)
        moe.moe_grouped_gemm_input_grad(dout, lay, shape, w, drows, ws)
        moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
        return out, drows, dw

    out, drows, dw = run()
    assert moe.moe_get_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip((out, drows, dw), run()))
    for e, s in enumerate(seg):
        check(out[s], rows[s].double(), w[e].double().T)
        check(drows[s], dout[s].double(), w[e].double())
        check(dw[e], dout[s].double().T, rows[s].double())
