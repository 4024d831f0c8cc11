"""Offsets that pass 32 bits, in the gated block, Muon and the 4-bit products: what lies behind
them is compared with the same work at small offsets, the gated block's bit for bit.

Muon's norm is summed from other parts for other numbers of matrices, which moves X by 2^-24 or
so and so some of its roundings, and those of G and S, to the other neighbour.  Each of the two
results is off by no more than its output's rounding, 2^-8, and as much for the operands':
together 2 * 2 * 2^-8 of the norm; half of that is asked for."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_gated import Case as Gated
from test_gpu_w4 import Case as W4, weights

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def fill(t, seed, std):
    """Normal values, a slice at a time."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for part in t.view(-1).split(1 << 28):
        part.normal_(0.0, std, generator=g)
    return t


def test_gated_rows_past_two_and_four_gigabytes():
    """2 * I * R elements of gu pass 2^31; the last expert's rows against a call of their own."""
    N, H, I, last = 150000, 64, 8192, 700
    c = Gated(N, 2, 1, H, 8, counts=[N - last, last])
    c.shape = s = moe.Shape(N, 8, 2, 1, 1, I)
    c.ws = moe.gated_workspace(s)
    w_gu = fill(torch.empty(2, 2 * I, H, dtype=bf, device="cuda"), 1, H ** -0.5)
    w_d = fill(torch.empty(2, H, I, dtype=bf, device="cuda"), 2, H ** -0.5)
    gu, h = torch.empty(N, 2 * I, dtype=bf, device="cuda"), torch.empty(N, I, dtype=bf, device="cuda")
    moe.moe_gated_gemm(c.x, c.lay, s, w_gu, c.w, gu, h, c.ws)
    one = Gated(last, 1, 1, H, 8, counts=[last])
    one.shape = t = moe.Shape(last, 8, 1, 1, 1, I)
    one.ws = moe.gated_workspace(t)
    pairs = torch.empty(N, dtype=torch.long, device="cuda")
    pairs[c.lay["pair_row"].long()] = torch.arange(N, device="cuda")
    w = c.w.reshape(-1)[pairs[N - last:]].view(last, 1).contiguous()
    gu1, h1 = torch.empty(last, 2 * I, dtype=bf, device="cuda"), torch.empty(last, I, dtype=bf, device="cuda")
    x, d = c.x[N - last:].contiguous(), c.d[N - last:].contiguous()
    moe.moe_gated_gemm(x, one.lay, t, w_gu[1:], w, gu1, h1, one.ws)
    assert torch.equal(gu[N - last:], gu1) and torch.equal(h[N - last:], h1)
    dw, dw1 = torch.empty(N, 1, device="cuda"), torch.empty(last, 1, device="cuda")
    moe.moe_gated_gemm_grad(c.d, c.lay, s, w_d, c.w, gu, gu, dw, c.ws)  # in place
    moe.moe_gated_gemm_grad(d, one.lay, t, w_d[1:], w, gu1, gu1, dw1, one.ws)
    assert torch.equal(gu[N - last:], gu1)
    assert torch.equal(dw.reshape(-1)[pairs[N - last:]], dw1.reshape(-1))
    assert moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("M,N", [(4096, 8192), (8192, 4096)])
def test_muon_of_many_large_matrices(M, N):
    E = 70  # 2.3e9 elements
    shape = moe.MuonShape(E, M, N, steps=2)
    grad = fill(torch.empty(E, M, N, dtype=bf, device="cuda"), 3, 1e-3)
    out, ws = torch.empty_like(grad), moe.muon_workspace(shape)
    moe.moe_muon_update(grad, None, shape, out, ws)
    assert moe.moe_get_error(ws) == 0
    del ws
    one = moe.MuonShape(1, M, N, steps=2)
    alone, ws = torch.empty(1, M, N, dtype=bf, device="cuda"), moe.muon_workspace(one)
    for e in (0, 63, 69):
        moe.moe_muon_update(grad[e:e + 1], None, one, alone, ws)
        diff = (out[e].float() - alone[0].float()).norm() / alone.float().norm()
        assert diff <= 2 * 2.0 ** -8, (e, diff.item())


def test_w4_matrices_past_four_gigabytes():
    E, c_in, c_out, group = 80, 8192, 14336, 128
    c = W4(3 * E, E, 1, 128, 8, 64, False, counts=[3] * E)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    q = torch.randint(0, 256, (E, c_out, c_in // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = fill(torch.empty(E, c_out, c_in // group, dtype=bf, device="cuda"), 6, 0.01)
    w4 = moe.pack_w4(q, scales)
    assert w4.data.numel() > 1 << 32
    x = fill(torch.empty(3 * E, c_in, dtype=bf, device="cuda"), 7, 1.0)
    out = torch.empty(3 * E, c_out, device="cuda")
    moe.moe_w4_gemm(x, c.lay, c.shape, w4, out, c.ws)
    for e in (0, 72, 79):
        o, n = c.segments[e]
        w = weights(q[e], scales[e])
        want = x[o:o + n].double() @ w.T
        off = (2.0 ** -19 + c_in / 16 * 2.0 ** -24) * (x[o:o + n].double().abs() @ w.abs().T)
        assert ((out[o:o + n].double() - want).abs() <= off).all(), e
    assert moe.moe_get_error(c.ws) == 0
