"""Orthogonalised momentum of gradients at the end of fp32's range, with the tolerances of the
operator's other tests (a factor cancels: these matrices are like any others)."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_muon import check, normal, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [2.0 ** 62, 2.0 ** 63, 1.6e38, torch.finfo(torch.float32).max])
@pytest.mark.parametrize("M,N", [(128, 512), (72, 40)])
def test_entries_whose_squares_leave_fp32(value, M, N):
    """Entries of one size: the eight of a thread are all as large as an entry can be."""
    shape = moe.MuonShape(2, M, N)
    grad = torch.where(normal(1, 2, M, N) > 0, value, -value)
    out, _ = run(grad, None, shape)
    check(grad, None, shape, out, None)


def test_large_entries_among_small_ones():
    """The large ones' squares leave fp32, the others' do not matter beside them."""
    shape = moe.MuonShape(3, 64, 136)
    grad = normal(2, 3, 64, 136)
    grad[0, :8] *= 2.0 ** 125
    grad[1, :, :16] *= 2.0 ** 125
    grad[2] *= 2.0 ** 20
    out, _ = run(grad, None, shape)
    check(grad, None, shape, out, None)
    bf = grad.bfloat16()
    out, _ = run(bf, None, shape)
    check(bf, None, shape, out, None)


def test_momentum_near_the_end_of_the_range():
    """u = g + momentum * b' is the largest of what is added up."""
    shape = moe.MuonShape(2, 40, 264)
    sign = torch.where(normal(3, 2, 40, 264) > 0, 1.0, -1.0)
    grad, mom = sign * 1e38, sign * 5e37
    out, new = run(grad, mom, shape)
    check(grad, mom, shape, out, new)


@pytest.mark.parametrize("M,N", [(8, 24), (264, 1032), (1032, 264), (2048, 2048), (4096, 7168)])
@pytest.mark.parametrize("spread", [1.0, 1e-3])
def test_scaled_matrices_have_22_bits(M, N, spread):
    """A workspace ends with X's first halves, two copies, and its second ones times 2^11; a call of
    one step leaves those of u 2^p / (|u| + eps) there.  The second half is what the first leaves,
    2^-11 of x at most, rounded to fp16: 2^-11 of that, or 2^-25 of its unit, 2^-11.  x itself is two
    fp32 products with factors rounded to fp32: 2^-22.  spread: rows far below the others."""
    shape = moe.MuonShape(2, M, N, steps=1)
    grad = normal(4, 2, M, N)
    grad[:, 1::2] *= spread
    ws, out = moe.muon_workspace(shape), torch.empty(2, M, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_muon_update(grad, None, shape, out, ws)
    part = (2 * 2 * M * N + 255) // 256 * 256
    hi, lo = (ws[at:at + 2 * 2 * M * N].view(torch.float16).double().view(2, M, N)
              for at in (ws.numel() - 3 * part, ws.numel() - part))
    p = 0
    while 1 << 2 * p + 1 < max(M, N):
        p += 1
    g = grad.double()
    x = g * 2.0 ** p / (g.square().sum((1, 2), keepdim=True).sqrt() + shape.eps)
    off = (hi + lo * 2.0 ** -11 - x).abs()
    assert ((off - 2.0 ** -21 * x.abs() - 2.0 ** -36) <= 0).all()
