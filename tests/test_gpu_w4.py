"""Products with 4-bit weights against float64 definitions.

Tolerances.  The weights' whole numbers and the rows are exact bf16 operands; a group's products
are added by the tensor core, 16 at a time with truncation (group / 16 * 2^-23 of the terms'
magnitudes at most), then scaled and added to the row's sum in fp32, rounded to nearest (2^-24
of the sum so far, twice), and joined from at most as many blocks as there are chunks.  With
S the sum of the magnitudes of a row's terms that is at most (2^-19 + 2 * C_in / 32 * 2^-24) S.
A bf16 output rounds once more, 2^-8 of it.  The gate: as in the gated block's tests."""
import pytest
import torch

import train_ref as ref
from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8
bf = torch.bfloat16


def normal(seed, *size, std=1.0, dtype=bf):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*size, generator=g, device="cuda") * std).to(dtype)


def unpack(q):
    """[..., C_in / 2] bytes to [..., C_in] whole numbers."""
    return torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1)


def weights(q, scales):
    group = q.shape[-1] * 2 // scales.shape[-1]
    return (unpack(q).double() - 8) * scales.double().repeat_interleave(group, -1)


class Case:
    def __init__(self, N, E, k, c_in, c_out, group, gated, seed=0, counts=None):
        self.shape = s = moe.Shape(N, 8, E, k, 1, 8)
        self.lay, self.ws = moe.Layout(s), moe.w4_workspace(s)
        logits = normal(seed, N, E, dtype=torch.float32)
        if counts is not None:
            assert k == 1 and sum(counts) == N
            ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to("cuda")
            logits.scatter_(1, ids[:, None], 20.0)
        ids = torch.empty(N, k, dtype=torch.int32, device="cuda")
        self.w = torch.empty(N, k, device="cuda")
        moe.moe_route(logits, s, ids, self.w)
        moe.moe_dispatch_layout(ids, None, s, self.lay, self.ws)
        self.w = normal(seed + 9, N, k, dtype=torch.float32).abs() + 0.1
        self.segments = list(zip(self.lay["expert_offsets"].tolist(),
                                 self.lay["expert_counts"].tolist()))
        self.w_row = self.w.double().reshape(-1)[ref.pairs_of_rows(self.lay["pair_row"])][:, None]
        rows = c_out * (2 if gated else 1)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        self.q = torch.randint(0, 256, (E, rows, c_in // 2), generator=g, device="cuda",
                               dtype=torch.uint8)
        self.scales = (normal(seed + 2, E, rows, c_in // group, dtype=torch.float32) * 0.2 *
                       c_in ** -0.5).to(bf)
        self.w4 = moe.pack_w4(self.q, self.scales, gated=gated)
        self.x = normal(seed + 3, s.R, c_in)
        self.c_in, self.c_out, self.gated = c_in, c_out, gated

    def run(self, out_type=bf, weighted=True, out=None):
        if out is None:
            out = torch.full((self.shape.R, self.c_out), float("nan"), dtype=out_type,
                             device="cuda")
        if self.gated:
            moe.moe_w4_gated_gemm(self.x, self.lay, self.shape, self.w4,
                                  self.w if weighted else None, out, self.ws)
        else:
            moe.moe_w4_gemm(self.x, self.lay, self.shape, self.w4, out, self.ws)
        return out

    def check(self, out, weighted=True):
        y = torch.zeros(self.shape.R, self.q.shape[1], dtype=torch.float64, device="cuda")
        off = torch.zeros_like(y)
        for e, (o, c) in enumerate(self.segments[:self.shape.E]):
            w = weights(self.q[e], self.scales[e])
            y[o:o + c] = self.x[o:o + c].double() @ w.T
            off[o:o + c] = self.x[o:o + c].double().abs() @ w.abs().T
        off *= 2.0 ** -19 + self.c_in / 16 * 2.0 ** -24
        if self.gated:
            w = self.w_row if weighted else torch.ones_like(self.w_row)
            g, u = y.chunk(2, 1)
            og, ou = off.chunk(2, 1)
            want = ref.swiglu(y, w)
            off = w * (1.1 * og * (u.abs() + ou) + (g * torch.sigmoid(g)).abs() * ou)
            off = off + 4e-6 * want.abs()
            y = want
        assert torch.isfinite(out.float()).all()
        bound = off + (BF16 * y.abs() if out.dtype == bf else 0.0) + 1e-37
        over = ((out.double() - y).abs() - bound).max().item()
        assert over <= 0.0, over
        assert moe.moe_get_error(self.ws) == 0


SIZES = [  # N, E, k, c_in, c_out
    (1, 4, 1, 128, 8), (1, 8, 8, 384, 264), (1, 4, 2, 2048, 1032), (5, 1, 1, 1152, 520),
    (16, 8, 2, 640, 72), (40, 4, 1, 256, 256), (33, 64, 6, 1408, 136), (100, 3, 2, 896, 328),
    (70, 1, 1, 3200, 104), (300, 2, 2, 128, 40), (9, 300, 4, 512, 16),
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,E,k,c_in,c_out", SIZES)
def test_products(N, E, k, c_in, c_out, group):
    c_in = c_in // 128 * 128 + (group if group < 128 else 0)  # an end inside a chunk
    c = Case(N, E, k, c_in, c_out, group, False)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run(), out)
    c.check(c.run(torch.float32))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,E,k,c_in,c_out", SIZES)
def test_gated_products(N, E, k, c_in, c_out, group):
    c_in = c_in // 128 * 128 + (group if group < 128 else 0)
    c = Case(N, E, k, c_in, c_out, group, True, seed=20)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run(), out)
    c.check(c.run(weighted=False), weighted=False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", [
    [0, 0, 5, 0], [7, 8, 9, 1], [0, 33, 0, 64], [200, 1, 1, 1], [0, 0, 0, 1], [65, 129, 0, 0],
])
def test_ragged_segments(counts, gated):
    c = Case(sum(counts), 4, 1, 704, 136, 64, gated, seed=40, counts=counts)
    c.check(c.run())


def test_quantise():
    """The nearest of 16 steps, and what packing and products make of them."""
    w = normal(50, 3, 40, 384, std=0.02)
    w[0, 0, :128] = 0.0
    w[0, 1, :64] *= 1e-30
    for group in (32, 64, 128):
        q = torch.full((3, 40, 192), 255, dtype=torch.uint8, device="cuda")
        scales = torch.full((3, 40, 384 // group), float("nan"), dtype=bf, device="cuda")
        moe.moe_w4_quantize(w, q, scales)
        v = w.float().view(3, 40, -1, group)
        s = (v.abs().amax(3) / 7.0).to(bf)
        assert torch.equal(scales, s)
        safe = torch.where(s > 0, s.float(), torch.ones_like(s.float())).unsqueeze(3)
        want = torch.where(s.unsqueeze(3) > 0, (torch.round(v / safe) + 8).clamp(0, 15),
                           torch.full_like(v, 8.0))
        assert torch.equal(unpack(q), want.view(3, 40, 384).to(torch.uint8))
        a, b = moe.pack_w4(q, scales), moe.quantize_w4(w, group)
        assert torch.equal(a.data, b.data)


def test_values_stay_in_their_rows():
    """A row's NaN or infinity reaches no other row; masked ends of a chunk hold none."""
    for counts in ([5, 2, 3], [30, 40, 21]):
        c = Case(sum(counts), 3, 1, 448, 72, 64, False, seed=60, counts=counts)
        want = c.run()
        row = counts[0]  # the first of the second expert's
        c.x[row, 0], c.x[row, 447] = float("nan"), float("inf")
        out = c.run()
        keep = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
        keep[row] = False
        assert torch.equal(out[keep], want[keep]) and out[row].isnan().all()


def test_rows_of_no_expert_are_left():
    c = Case(40, 4, 1, 256, 72, 128, False, seed=70, counts=[10, 10, 15, 5])
    want = c.run()
    c.lay["expert_counts"][3] = 2
    out = c.run()
    assert torch.equal(out[:37], want[:37]) and out[37:].isnan().all()


@pytest.mark.parametrize("N,E,k,c_in", [(3, 8, 2, 4096), (150, 4, 2, 1024)])
def test_streams_graphs_and_same_bits(N, E, k, c_in):
    a = Case(N, E, k, c_in, 520, 128, False, seed=80)
    b = Case(N, E, k, c_in, 264, 64, True, seed=81)
    b.ws = a.ws  # one workspace for calls in turn
    want = [a.run(), b.run()]
    out = [torch.zeros_like(t) for t in want]

    def both():
        a.run(out=out[0])
        b.run(out=out[1])

    def same():
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        for t in out:
            t.zero_()

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        both()
    same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
        both()
    for _ in range(3):
        g.replay()
        same()


def test_nothing_beside_the_outputs_is_written():
    c = Case(11, 5, 2, 2176, 136, 128, False, seed=90)
    want, pad = c.run(), 1024
    flat = torch.full((want.numel() + 2 * pad,), 7.0, dtype=bf, device="cuda")
    need = moe.moe_w4_workspace_bytes(c.shape)
    ws = torch.full((need + 2 * pad,), 171, dtype=torch.uint8, device="cuda")
    ws[pad:pad + need] = 0
    c.ws = ws[pad:pad + need]
    c.run(out=flat[pad:-pad].view(want.shape))
    assert torch.equal(flat[pad:-pad].view(want.shape), want)
    assert (flat[:pad] == 7.0).all() and (flat[-pad:] == 7.0).all()
    assert (ws[:pad] == 171).all() and (ws[-pad:] == 171).all()
