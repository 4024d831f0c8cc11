"""Every element of Muon's updates, in the kernel's forms: tiles of 256 columns by four epilogue
warps (more than four tiles a pair of SMs in each of a step's products) or by eight, and narrow
ones.

Tolerances.  As for the norm of a matrix in the operator's other tests, an update's error by the
roundings of the operands is given twice that of the same roundings in 64 bits, e.  An element's
error is at most the norm of its row of errors, and of its column: 2 min(|e_i|, |e_j|).  An element of
a product is off by fp32 sums of up to 1032 terms by at most 1032 * 2^-24 of the norms of the two
vectors that it is a product of, and no singular value is above 1.3: 1e-3 * 1.3 over all
products.  Rounding to bf16 adds 2^-8 of the number that is rounded.  Without that rounding this is
0.05 to 0.1 of the root mean square of the entries (sides of 264 to 1032): a line, a row or an
element in the wrong place, an entry of the diagonal left out or added twice is more."""
import pytest
import torch

import muon_ref as ref
from combine_warp_top_gb300 import moe
from test_gpu_muon import BETA, check, normal, run

pytestmark = pytest.mark.gpu


def check_elements(grad, mom, shape, out):
    u, _ = ref.momentum(grad, mom, BETA, shape.nesterov)
    for e in range(shape.E):
        want = ref.orthogonal(u[e], shape.steps, shape.eps)
        off = ref.orthogonal(u[e], shape.steps, shape.eps, rounded=True) - want
        bound = 2 * torch.minimum(off.norm(dim=1)[:, None], off.norm(dim=0)[None, :]) + 1.3e-3
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        over = ((out[e].double() - want).abs() - bound).max().item()
        assert over <= 0.0, (e, over)


def tiles(shape):
    """Tiles of 256 x 256 of the symmetric products and of a step's last one."""
    blocks = [-(-n // 256) for n in (min(shape.M, shape.N), shape.M, shape.N)]
    return shape.E * blocks[0] * (blocks[0] + 1) // 2, shape.E * blocks[1] * blocks[2]


@pytest.mark.parametrize("E,M,N", [
    (160, 264, 280), (160, 280, 264), (110, 328, 520), (110, 520, 328), (110, 400, 400),
    (60, 520, 776), (60, 776, 520),
])
def test_many_tiles_a_pair(E, M, N):
    """Remainders of a line, of a warp's rows and of a tile, wide and tall."""
    shape = moe.MuonShape(E, M, N)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert min(tiles(shape)) > 4 * pairs
    grad, mom = normal(1, E, M, N), normal(2, E, M, N, std=3.0)
    out, new = run(grad, mom, shape)
    check(grad, mom, shape, out, new)
    check_elements(grad, mom, shape, out)
    again, _ = run(grad, mom, shape)
    assert torch.equal(again, out)


@pytest.mark.parametrize("E,M,N", [
    (1, 8, 8), (2, 40, 264), (2, 264, 40), (1, 264, 264), (1, 392, 384), (3, 128, 1032),
    (3, 1032, 128), (1, 1000, 1032), (1, 1032, 1000), (30, 392, 520), (30, 520, 392),
    (20, 264, 1032), (20, 1032, 264), (78, 40, 264),
])
def test_elements(E, M, N):
    shape = moe.MuonShape(E, M, N)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert min(tiles(shape)) <= 4 * pairs
    grad, mom = normal(3, E, M, N), normal(4, E, M, N, std=3.0)
    out, _ = run(grad, mom, shape)
    check_elements(grad, mom, shape, out)


def test_elements_of_other_spectra():
    E, M, N = 3, 256, 320
    grad = torch.stack([
        normal(1, M, 8) @ normal(2, 8, N),
        normal(3, M, N) * torch.logspace(0, -3, M, device="cuda")[:, None],
        torch.eye(M, N, device="cuda") + 0.01 * normal(5, M, N)])
    shape = moe.MuonShape(E, M, N)
    out, _ = run(grad, None, shape)
    check_elements(grad, None, shape, out)
