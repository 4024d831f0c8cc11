"""Orthogonalised momentum against its definition in 64 bits.

Tolerances.  The operator rounds G, S without its diagonal and X as an operand to fp16 and nothing
else below fp32 but the output.  What those roundings do to a result depends on the matrix (small singular
values grow by 3.4445 a step, and so does what a rounding adds there), so it is computed: the
same recurrence in 64 bits with these roundings is off by e from the one without, and the
operator, whose own sums round otherwise in the last place and so round some numbers to the
other neighbour, is given 2 e.  The output's rounding to bf16 adds 2^-8 of it, fp32 sums of up
to 1032 products at most 1032 * 2^-24 = 6e-5 of the result a product, 15 products: 1e-3.
All in the Frobenius norm of a matrix.  The momentum is one fp32 multiply-add: 2^-24 of each
of its two terms, twice (the coefficient 0.95 is rounded, too)."""
import pytest
import torch

import muon_ref as ref
from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu
BETA, EPS = 0.95, 1e-7


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, *size, std=1.0, dtype=torch.float32):
    return (torch.randn(*size, generator=gen(seed), device="cuda") * std).to(dtype)


def run(grad, mom, shape, in_place=False):
    ws = moe.muon_workspace(shape)
    out = torch.full(grad.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    new = None if mom is None else mom.clone() if in_place else torch.full_like(mom, float("nan"))
    if in_place and mom is not None:
        moe.moe_muon_update(grad, new, shape, out, ws)
    else:
        moe.moe_muon_update(grad, mom, shape, out, ws, new_momentum=new)
    assert moe.moe_get_error(ws) == 0
    return out, new


def check(grad, mom, shape, out, new):
    u, b = ref.momentum(grad, mom, BETA, shape.nesterov)
    if b is not None:
        slack = 2.0 ** -23 * (BETA * mom.double().abs() + grad.double().abs())
        assert ((new.double() - b).abs() <= slack).all()
    for e in range(shape.E):
        want = ref.orthogonal(u[e], shape.steps, shape.eps)
        off = (ref.orthogonal(u[e], shape.steps, shape.eps, rounded=True) - want).norm()
        err, off, size = (out[e].double() - want).norm().item(), off.item(), want.norm().item()
        assert err <= 2 * off + (2.0 ** -8 + 1e-3) * size, (e, err, off, size)


@pytest.mark.parametrize("E,M,N", [
    (1, 8, 8), (3, 8, 24), (2, 24, 8), (2, 64, 64), (2, 40, 264), (2, 264, 40), (1, 136, 520),
    (1, 520, 136), (2, 256, 256), (1, 264, 264), (1, 392, 384), (5, 128, 1032), (3, 1032, 128),
    (1, 1000, 1032), (1, 1032, 1000), (40, 32, 72),
])
def test_sizes(E, M, N):
    shape = moe.MuonShape(E, M, N)
    grad, mom = normal(1, E, M, N), normal(2, E, M, N, std=3.0)
    out, new = run(grad, mom, shape)
    check(grad, mom, shape, out, new)


@pytest.mark.parametrize("E,M,N", [
    (80, 8, 24), (80, 24, 8), (78, 40, 264), (78, 264, 40), (40, 264, 280), (30, 392, 520),
    (30, 520, 392), (20, 264, 1032), (20, 1032, 264),
])
def test_sizes_of_many_matrices(E, M, N):
    """Too many tiles for narrow ones: 256 columns, the symmetric products by half."""
    shape = moe.MuonShape(E, M, N)
    grad, mom = normal(1, E, M, N), normal(2, E, M, N, std=3.0)
    out, new = run(grad, mom, shape)
    check(grad, mom, shape, out, new)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_momentum,nesterov", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("M,N", [(96, 200), (200, 96)])
def test_types(dtype, with_momentum, nesterov, M, N):
    shape = moe.MuonShape(2, M, N, steps=3, nesterov=nesterov)
    grad = normal(3, 2, M, N, dtype=dtype)
    mom = normal(4, 2, M, N) if with_momentum else None
    out, new = run(grad, mom, shape)
    check(grad, mom, shape, out, new)
    if with_momentum:
        again, b = run(grad, mom, shape, in_place=True)
        assert torch.equal(again, out) and torch.equal(b, new)


def test_low_rank_and_decaying_spectra():
    """Singular values far below the largest, which a rounding of X itself would bury."""
    E, M, N = 3, 256, 320
    grad = torch.stack([
        normal(1, M, 8) @ normal(2, 8, N),
        normal(3, M, 16) @ normal(4, 16, N) + 0.01 * normal(5, M, N),
        (normal(6, M, 64) * torch.logspace(0, -3, 64, device="cuda")) @ normal(7, 64, N)])
    shape = moe.MuonShape(E, M, N)
    out, _ = run(grad, None, shape)
    check(grad, None, shape, out, None)


def test_singular_values_and_scale():
    shape = moe.MuonShape(2, 128, 512)
    grad = normal(5, 2, 128, 512)
    out, _ = run(grad, None, shape)
    for e in range(2):
        s = torch.linalg.svdvals(out[e].double())
        assert 0.5 < s.min() and s.max() < 1.3
    # a factor cancels, also where the squares leave fp32: each of these is as close to the
    # definition as any other gradient
    scaled = moe.MuonShape(2, 128, 512, eps=1e-12)
    for k in (-24, 40, 100):
        a, _ = run(grad * 2.0 ** k, None, scaled)
        check(grad * 2.0 ** k, None, scaled, a, None)


@pytest.mark.parametrize("E,M,N", [(4, 2048, 1408), (2, 1536, 4096)])
def test_tiles_in_turn(E, M, N):
    """More tiles of a matrix than run at once: none may read what another has written."""
    shape = moe.MuonShape(E, M, N)
    grad = normal(11, E, M, N)
    out, _ = run(grad, None, shape)
    check(grad, None, shape, out, None)
    again, _ = run(grad, None, shape)
    assert torch.equal(out, again)


def test_zero_and_non_finite_matrices():
    """A zero matrix has a zero update; an infinity or a NaN stays in its matrix."""
    E, M, N = 4, 72, 264
    grad = normal(6, E, M, N)
    clean, _ = run(grad, None, moe.MuonShape(E, M, N))
    bad = grad.clone()
    bad[0] = 0.0
    bad[1, 3, 5] = float("inf")
    bad[2, 71, 263] = float("nan")
    out, _ = run(bad, None, moe.MuonShape(E, M, N))
    assert (out[0] == 0).all()
    assert out[1].isnan().all() and out[2].isnan().all()
    assert torch.equal(out[3], clean[3])


def test_same_bits_streams_and_graph():
    shape = moe.MuonShape(6, 520, 264)
    grad, mom = normal(7, 6, 520, 264), normal(8, 6, 520, 264)
    first, new = run(grad, mom, shape)
    ws = moe.muon_workspace(shape)
    out, buf = torch.zeros_like(first), torch.zeros_like(new)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        moe.moe_muon_update(grad, mom, shape, out, ws, new_momentum=buf)
    st.synchronize()
    assert torch.equal(out, first) and torch.equal(buf, new)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_muon_update(grad, mom, shape, out, ws, new_momentum=buf)
        moe.moe_muon_update(grad, mom, shape, out, ws, new_momentum=buf)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(buf, new)


def test_nothing_beside_the_outputs_is_written():
    shape = moe.MuonShape(2, 264, 136)
    n, pad = 2 * 264 * 136, 4096
    grad, mom = normal(9, 2, 264, 136), normal(10, 2, 264, 136)
    out = torch.full((n + 2 * pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    new = torch.full((n + 2 * pad,), 7.0, device="cuda")
    need = moe.moe_muon_workspace_bytes(shape)
    ws = torch.full((need + 2 * pad,), 171, dtype=torch.uint8, device="cuda")
    ws[pad:pad + 256] = 0
    moe.moe_muon_update(grad, mom, shape, out[pad:pad + n].view(2, 264, 136),
                        ws[pad:pad + need], new_momentum=new[pad:pad + n].view(2, 264, 136))
    want, b = run(grad, mom, shape)
    assert torch.equal(out[pad:pad + n].view_as(want), want)
    assert torch.equal(new[pad:pad + n].view_as(b), b)
    for t, v in ((out, 7.0), (new, 7.0), (ws, 171)):
        assert (t[:pad] == v).all() and (t[-pad:] == v).all()
