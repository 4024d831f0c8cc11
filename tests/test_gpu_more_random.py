"""The gated block, Muon's update and the products with 4-bit weights on seeded random sizes:
experts, segment lengths (skewed, empty, one row), widths, groups, spectra and types drawn
together, so that combinations that no hand-picked case names are checked too.  Every output
element against float64 with the tolerances of the operators' own tests, and the same bits from a
second call."""
import numpy as np
import pytest
import torch

import test_gpu_gated as gated
import test_gpu_muon as muon
import test_gpu_w4 as w4
from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def draw(seed, most_rows):
    """The generator, tokens, experts, k, and segment lengths or None for routed ones."""
    rng = np.random.default_rng(seed)
    E = int(rng.choice([1, 2, 5, 8, 31, 33, 64, 100]))
    N = max(1, int(2 ** rng.uniform(0, np.log2(most_rows))))
    if rng.random() < 0.5:
        return rng, N, E, int(rng.integers(1, min(E, 8) + 1)), None
    p = (1.0 + np.arange(E)) ** -float(rng.choice([0.0, 1.0, 2.0]))
    return rng, N, E, 1, rng.multinomial(N, rng.permutation(p / p.sum())).tolist()


def width(rng, most):
    return 8 * max(1, int(2 ** rng.uniform(0, np.log2(most / 8))))


@pytest.mark.parametrize("i", range(20))
def test_gated_block(i):
    rng, N, E, k, counts = draw(7000 + i, 1500)
    H, I = width(rng, 900), width(rng, 700)
    c = gated.Case(N, E, k, H, I, seed=i, counts=counts)
    weights = bool(rng.random() < 0.7)
    h, gu = c.forward(weights=weights)
    c.check_forward(h, gu, weights=weights)
    assert torch.equal(c.forward(weights=weights, keep=False)[0], h)
    dgu, dw = c.grad(weights=weights)
    c.check_grad(dgu, dw, weights=weights)
    again, same = c.grad(weights=weights, in_place=True)
    assert torch.equal(again, dgu) and torch.equal(same, dw)
    assert moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("i", range(20))
def test_muon(i):
    rng = np.random.default_rng(7100 + i)
    M, N = width(rng, 1000), width(rng, 1000)
    E = int(rng.integers(1, 9))
    dtype = torch.float32 if rng.random() < 0.5 else torch.bfloat16
    shape = moe.MuonShape(E, M, N, steps=int(rng.integers(1, 7)), nesterov=bool(rng.random() < 0.5))
    grad = muon.normal(i, E, M, N, std=float(10.0 ** rng.uniform(-6, 3)), dtype=dtype)
    mom = None
    if rng.random() < 0.7:
        mom = muon.normal(100 + i, E, M, N) * grad.float().std()
    out, new = muon.run(grad, mom, shape)
    muon.check(grad, mom, shape, out, new)
    again, b = muon.run(grad, mom, shape)
    assert torch.equal(again, out) and (mom is None or torch.equal(b, new))


@pytest.mark.parametrize("i", range(32))
def test_w4(i):
    rng, N, E, k, counts = draw(7200 + i, 600)
    group = int(rng.choice([32, 64, 128]))
    c_in, c_out = group * max(1, width(rng, 2500) // group), width(rng, 700)
    c = w4.Case(N, E, k, c_in, c_out, group, bool(rng.random() < 0.5), seed=i, counts=counts)
    weighted = bool(rng.random() < 0.5)
    out = c.run(weighted=weighted)
    c.check(out, weighted=weighted)
    assert torch.equal(c.run(weighted=weighted), out)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("E", [1, 30])
def test_w4_every_weight_is_exact(group, E):
    """Rows with a single one in them: their outputs are the weights themselves, to the last bit,
    with scales from 2^-100 to 2^100."""
    c_in, c_out = 256 + group, 264
    c = w4.Case(c_in, E, 1, c_in, c_out, group, False, seed=5)
    c.scales = torch.exp2(torch.randint(-100, 101, c.scales.shape, device="cuda").float())
    c.scales = (c.scales * (1 + torch.rand(c.scales.shape, device="cuda"))).to(torch.bfloat16)
    c.w4 = moe.pack_w4(c.q, c.scales)
    c.x = torch.eye(c_in, device="cuda", dtype=torch.bfloat16)
    out = c.run(torch.float32)
    for e, (o, n) in enumerate(c.segments[:E]):
        want = w4.weights(c.q[e], c.scales[e]).T[o:o + n]
        assert torch.equal(out[o:o + n].double(), want)
    assert len(c.q.unique()) == 256
