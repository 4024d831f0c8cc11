"""The sigmoid router's gradient where the selected scores are small: all of them far below
what fp32 holds, or some beside larger ones, against the float64 definition.

Tolerance: expf is good to 2 units in the last place, the difference of two logits it is
taken of to half a unit of that difference (at most 16 here: 5e-7 of the exponential; 64 in
the mixed rows: 2e-6), sums over at most 32 choices and the divisions to 2 units each: 6e-6
of the magnitude of the terms, as at ordinary logits; and three steps of 2^-149 a unit of
the terms where a weight is subnormal."""
import pytest
import torch

import train_ref as ref
from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def compare(logits, ids, dw):
    N, E = logits.shape
    shape = moe.Shape(N, 8, E, ids.shape[1], 1, 8)
    out = torch.full((N, E), float("nan"), device="cuda")
    moe.moe_route_sigmoid_bias_grad(logits, ids, dw, shape, out)
    L, i, d = logits.double(), ids.long(), dw.double()
    want = ref.route_grad(L, i, d, "sigmoid_bias")
    w = ref.route_weights(L, i, "sigmoid_bias")
    scale = (w * d.abs()).sum(1, keepdim=True)
    spread = torch.zeros_like(L)
    bound = spread.scatter(1, i, (6e-6 * w + 3 * 2.0 ** -149) * (d.abs() + scale))
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= bound).all()
    return out


@pytest.mark.parametrize("N,E,k", [(5, 8, 1), (37, 24, 3), (70, 128, 8), (33, 250, 17),
                                   (9, 300, 32)])
@pytest.mark.parametrize("base", [-17.0, -60.0, -87.5, -90.0, -100.0, -104.0, -200.0, -600.0])
def test_all_scores_small(base, N, E, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    logits = base + 2.0 * torch.randn(N, E, generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices.int()
    dw = torch.randn(N, k, generator=g, device="cuda")
    got = compare(logits, ids, dw)
    if k == 1:
        assert (got == 0).all()  # one expert's weight is 1 whatever its logit
    else:
        assert (got != 0).any()


@pytest.mark.parametrize("top", [-40.0, -3.0, 0.0, 5.0, 95.0, 200.0])
def test_small_scores_beside_larger_ones(top):
    """One choice at `top`, the others down to 64 below it or below zero."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    logits = min(top, 0.0) - 64.0 * torch.rand(50, 24, generator=g, device="cuda")
    logits[:, 7] = top
    ids = torch.tensor([[7, 3, 20, 11]], device="cuda").int().repeat(50, 1)
    compare(logits, ids, torch.randn(50, 4, generator=g, device="cuda"))


def test_finite_logits_of_any_size():
    """The largest finite values: nothing overflows on the way."""
    low = torch.finfo(torch.float32).min
    logits = torch.tensor([[low, low, low, 0.0], [low, -low, 1.0, 0.0], [-low, -low, -low, 0.0],
                           [low, -200.0, low, 0.0]], device="cuda")
    ids = torch.tensor([[0, 1, 2]], device="cuda").int().repeat(4, 1)
    dw = torch.tensor([[1.0, 2.0, 4.0]], device="cuda").repeat(4, 1)
    out = torch.empty(4, 4, device="cuda")
    moe.moe_route_sigmoid_bias_grad(logits, ids, dw, moe.Shape(4, 8, 4, 3, 1, 8), out)
    third = torch.tensor([1.0, 2.0, 4.0], device="cuda") / 3 - 7.0 / 9
    assert torch.allclose(out[0, :3], third, atol=1e-6) and out[0, 3] == 0
    assert torch.isfinite(out).all()
    assert (out[2] == 0).all()       # scores of one: their derivative is 0
    assert (out[3, [0, 2, 3]] == 0).all()


def test_choices_of_probability_zero():
    """Logits of -inf among the choices and as all of them: no gradient, and no NaN."""
    inf = float("inf")
    logits = torch.tensor([[-inf, 1.0, 2.0, 0.0], [-inf, -inf, -inf, 0.0]], device="cuda")
    ids = torch.tensor([[0, 1, 2]], device="cuda").int().repeat(2, 1)
    out = torch.full((2, 4), float("nan"), device="cuda")
    moe.moe_route_sigmoid_bias_grad(logits, ids, torch.ones(2, 3, device="cuda").cumsum(1),
                                    moe.Shape(2, 8, 4, 3, 1, 8), out)
    assert torch.isfinite(out).all() and (out[0, [1, 2]] != 0).all()
    assert out[0, 0] == 0 and (out[1] == 0).all()
