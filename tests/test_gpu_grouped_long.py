"""Grouped products over contractions of millions of terms, and the precision that the partial
sums of fp32 outputs are there for: positive terms, so that what the tensor cores' truncating
additions lose adds up.

Tolerances.  The tensor core adds 16 products at a time into its fp32 accumulator and drops
what is below the last place: at most 2^-23, on average (over a value's place between two
powers of two, and half a unit) 0.36 * 2^-23 = 4.3e-8 of the partial sum.  A chain's partial
sums are half of its whole on average.
 - bf16 outputs: chains of at most 32768 terms lose at most 2048 * 2^-23 of the sum; the
   chains' sums are added to nearest (2^-24 each, at most 2048 of them here); one rounding
   to bf16's 8 significant bits, 2^-8.  One chain over all the terms would lose 1.1e-2 over
   2^23 terms.
 - fp32 outputs: chains of 512 terms lose 32 / 2 * 4.3e-8 = 6.9e-7 on average, and the
   additions to nearest next to nothing.  One chain over 2048 terms, which is the share of
   each of four pairs of 8192, would lose 2.8e-6, and over all 8192 1.1e-5: 1.5e-6 is
   between."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_grouped import make_layout

pytestmark = pytest.mark.gpu
BF16_BOUND = 2.0 ** -8 + (2048 + 1024) * 2.0 ** -23


def positive(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).abs_()


def product(a, b, step=1 << 20):
    """a [m, K] times b [K, n] in float64, a stretch of K at a time."""
    out = 0.0
    for k in range(0, a.shape[1], step):
        out = out + a[:, k:k + step].double() @ b[k:k + step].double()
    return out


def bf16_close(got, want):
    rel = (got.double() - want).abs() / want
    assert rel.max().item() <= BF16_BOUND, rel.max().item()


@pytest.mark.parametrize("counts", [[(1 << 25) + 5],                 # pairs share the rows
                                    [7] * 60 + [(1 << 23) + 21] + [1, 0] * 20],  # one pair has them
                         ids=["one expert", "101 experts"])
def test_weights_gradient_of_many_rows_in_bf16(counts):
    shape, lay, offs = make_layout(counts)
    rows, dout = positive(shape.N, 8, seed=1), positive(shape.N, 16, seed=2)
    dw = torch.empty(shape.E, 16, 8, dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace(shape)
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    assert moe.moe_get_error(ws) == 0
    for e in {0, counts.index(max(counts)), shape.E - 1}:
        s = slice(int(offs[e]), int(offs[e + 1]))
        if counts[e]:
            bf16_close(dw[e], product(dout[s].T, rows[s]))
        else:
            assert (dw[e] == 0).all()


@pytest.mark.parametrize("rows_n", [3, 130])
@pytest.mark.parametrize("back", [False, True], ids=["forward", "rows' gradient"])
def test_long_rows_in_bf16(rows_n, back):
    """One matrix whose rows (or columns) are 2^23 long: tiles of few rows, and of 256."""
    K, n = (1 << 23) + 72, 8
    shape, lay, _ = make_layout([rows_n])
    a, w = positive(rows_n, K, seed=3), positive(1, *((K, n) if back else (n, K)), seed=4)
    out = torch.empty(rows_n, n, dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace(shape)
    if back:
        moe.moe_grouped_gemm_input_grad(a, lay, shape, w, out, ws)
    else:
        moe.moe_grouped_gemm(a, lay, shape, w, out, ws)
    assert moe.moe_get_error(ws) == 0
    bf16_close(out, product(a, w[0] if back else w[0].T))


def mean_error(got, want):
    return ((got.double() - want).abs() / want).mean().item()


@pytest.mark.parametrize("ci,co", [(128, 256), (4096, 4096)], ids=["shared", "a pair each"])
def test_partial_sums_of_fp32_weights_gradients(ci, co):
    K = 8192
    shape, lay, _ = make_layout([K])
    rows, dout = positive(K, ci, seed=5), positive(K, co, seed=6)
    dw = torch.empty(1, co, ci, device="cuda")
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, moe.workspace(shape))
    assert mean_error(dw[0], dout.double().T @ rows.double()) < 1.5e-6


@pytest.mark.parametrize("back", [False, True], ids=["forward", "rows' gradient"])
@pytest.mark.parametrize("rows_n,n", [(40, 512), (40, 16384), (700, 256), (2600, 2048)])
def test_partial_sums_of_fp32_rows(rows_n, n, back):
    """Tiles of few rows and of 256, few enough for pairs to share one and more than that."""
    K = 8192
    shape, lay, _ = make_layout([rows_n])
    a, w = positive(rows_n, K, seed=7), positive(1, *((K, n) if back else (n, K)), seed=8)
    out = torch.empty(rows_n, n, device="cuda")
    ws = moe.workspace(shape)
    if back:
        moe.moe_grouped_gemm_input_grad(a, lay, shape, w, out, ws)
    else:
        moe.moe_grouped_gemm(a, lay, shape, w, out, ws)
    assert mean_error(out, a.double() @ (w[0] if back else w[0].T).double()) < 1.5e-6
