"""The gated block in one kernel, forward and back, against float64 definitions.

Tolerances.  A product of K terms: the tensor core adds 16 of them at a time into its fp32
accumulator and truncates, 2^-23 of the sum so far at most, so K / 16 * 2^-23 = K * 7.5e-9 of
the sum of the terms' magnitudes.  What that does to an output is its derivative by g, u or dh
times that: |SiLU'| <= 1.1.  The hardware's exponential and divide: 4e-6 of a term's magnitude
(|g| < 12 here).  A bf16 output rounds once, 2^-8.  A row's sum over I columns: 128 of them in
order and then ceil(I / 128) parts, 2^-24 of the terms' magnitudes each."""
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


def within(got, want, slack, what):
    assert torch.isfinite(got.float()).all(), what
    bound = slack + (BF16 * want.abs() if got.dtype == bf else 0.0) + 1e-37
    over = ((got.double() - want).abs() - bound).max().item()
    assert over <= 0.0, f"{what}: {over} over the bound"


class Case:
    """N tokens routed to k of E experts, or the given rows an expert."""

    def __init__(self, N, E, k, H, I, seed=0, counts=None, placement=None):
        self.shape = s = moe.Shape(N, 8, E, k, 1, I)
        self.lay, self.ws = moe.Layout(s), moe.gated_workspace(s)
        logits = normal(seed, N, E, dtype=torch.float32)
        if counts is not None:  # k = 1: the first counts[0] tokens go to expert 0, and so on
            assert k == 1 and sum(counts) == N
            ids = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to("cuda")
            logits.scatter_(1, ids[:, None], 20.0)
        self.ids = torch.empty(N, k, dtype=torch.int32, device="cuda")
        self.w = torch.empty(N, k, device="cuda")
        moe.moe_route(logits, s, self.ids, self.w)
        if counts is not None:
            self.w.copy_(normal(seed + 9, N, 1, dtype=torch.float32).abs() + 0.1)
        moe.moe_dispatch_layout(self.ids, placement, s, self.lay, self.ws)
        self.H, self.I, self.R = H, I, s.R
        self.segments = list(zip(self.lay["expert_offsets"].tolist(),
                                 self.lay["expert_counts"].tolist()))
        self.w_row = self.w.double().reshape(-1)[ref.pairs_of_rows(self.lay["pair_row"])][:, None]
        self.x, self.d = normal(seed + 1, s.R, H), normal(seed + 2, s.R, H)
        self.w_gu = normal(seed + 3, E, 2 * I, H, std=1.5 * H ** -0.5)
        self.w_d = normal(seed + 4, E, H, I, std=H ** -0.5)
        self.gu = normal(seed + 5, s.R, 2 * I, std=1.5)

    def product(self, rows, w, eq):
        out = [torch.einsum(eq, rows[o:o + c].double(), w[e].double())
               for e, (o, c) in enumerate(self.segments[:self.shape.E])]
        full = torch.zeros(self.R, out[0].shape[1], dtype=torch.float64, device="cuda")
        for (o, c), v in zip(self.segments, out):
            full[o:o + c] = v
        return full

    def forward(self, weights=True, keep=True):
        h = torch.full((self.R, self.I), float("nan"), dtype=bf, device="cuda")
        gu = torch.full((self.R, 2 * self.I), float("nan"), dtype=bf, device="cuda") if keep else None
        moe.moe_gated_gemm(self.x, self.lay, self.shape, self.w_gu, self.w if weights else None, gu,
                           h, self.ws)
        return h, gu

    def check_forward(self, h, gu, weights=True):
        G = self.product(self.x, self.w_gu, "ri,oi->ro")
        off = self.H * 7.5e-9 * self.product(self.x.abs(), self.w_gu.abs(), "ri,oi->ro")
        if gu is not None:
            within(gu, G, off, "gu")
        w = self.w_row if weights else torch.ones_like(self.w_row)
        g, u = G.chunk(2, 1)
        og, ou = off.chunk(2, 1)
        want = ref.swiglu(G, w)
        slack = w * (1.1 * og * (u.abs() + ou) + (g * torch.sigmoid(g)).abs() * ou)
        within(h, want, slack + 4e-6 * want.abs(), "h")

    def grad(self, weights=True, sums=True, in_place=False):
        gu = self.gu.clone() if in_place else self.gu
        dgu = gu if in_place else torch.full_like(gu, float("nan"))
        dw = torch.full((self.shape.N, self.shape.k), float("nan"), device="cuda") if sums else None
        moe.moe_gated_gemm_grad(self.d, self.lay, self.shape, self.w_d,
                                self.w if weights else None, gu, dgu, dw, self.ws)
        return dgu, dw

    def check_grad(self, dgu, dw, weights=True):
        D = self.product(self.d, self.w_d, "ro,oi->ri")
        off = self.H * 7.5e-9 * self.product(self.d.abs(), self.w_d.abs(), "ro,oi->ri")
        w = self.w_row if weights else torch.ones_like(self.w_row)
        G = self.gu.double()
        g, u = G.chunk(2, 1)
        want, sums = ref.swiglu_grad(D, G, w)
        per = torch.cat([1.1 * w * u.abs(), w * (g * torch.sigmoid(g)).abs()], 1)
        mag = torch.cat([w * D.abs() * (1 + g.abs()) * u.abs(), w * D.abs() * g.abs()], 1)
        within(dgu, want, per * torch.cat([off, off], 1) + 4e-6 * mag, "dgu")
        if dw is not None:
            act = (g * torch.sigmoid(g) * u).abs()
            rel = 4e-6 + (128 + (self.I + 127) // 128) * 2.0 ** -24
            slack = (off * act).sum(1) + rel * (D.abs() * act).sum(1)
            rows = self.lay["pair_row"].long()
            within(dw, sums[rows].view_as(dw), slack[rows].view_as(dw), "dtopk_w")


SIZES = [  # N, E, k, H, I
    (1, 4, 1, 8, 8), (1, 8, 8, 64, 40), (3, 8, 2, 264, 136), (16, 8, 2, 512, 264),
    (67, 8, 3, 72, 128), (64, 8, 2, 128, 256), (130, 2, 1, 520, 72), (300, 2, 2, 64, 392),
    (700, 3, 2, 200, 120), (1025, 4, 2, 1032, 520), (33, 64, 6, 136, 64), (5, 1, 1, 2056, 1032),
    (2000, 2, 1, 40, 1416),
]


@pytest.mark.parametrize("N,E,k,H,I", SIZES)
def test_forward(N, E, k, H, I):
    c = Case(N, E, k, H, I)
    h, gu = c.forward()
    c.check_forward(h, gu)
    again, _ = c.forward(keep=False)
    assert torch.equal(again, h)
    h, gu = c.forward(weights=False)
    c.check_forward(h, gu, weights=False)
    assert moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("N,E,k,H,I", SIZES)
def test_grad(N, E, k, H, I):
    c = Case(N, E, k, H, I, seed=20)
    dgu, dw = c.grad()
    c.check_grad(dgu, dw)
    again, _ = c.grad(sums=False)
    assert torch.equal(again, dgu)
    again, same = c.grad(in_place=True)
    assert torch.equal(again, dgu) and torch.equal(same, dw)
    dgu, dw = c.grad(weights=False)
    c.check_grad(dgu, dw, weights=False)
    assert moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("counts", [
    [0, 0, 5, 0], [1, 255, 256, 257], [31, 33, 0, 64], [600, 1, 1, 1], [0, 0, 0, 1], [65, 65, 0, 0],
])
def test_ragged_segments(counts):
    c = Case(sum(counts), 4, 1, 136, 200, seed=40, counts=counts)
    c.check_forward(*c.forward())
    c.check_grad(*c.grad())
    perm = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")
    c = Case(sum(counts), 4, 1, 72, 104, seed=41, counts=counts, placement=perm)
    c.check_forward(*c.forward())
    c.check_grad(*c.grad())


@pytest.mark.parametrize("N", [24, 900])
def test_values_stay_in_their_rows(N):
    """A row's NaN or infinity reaches no other row, an expert's matrix no other expert's rows."""
    c = Case(N, 3, 1, 264, 136, seed=50, counts=[N // 3 - 1, N // 3, N // 3 + 1])
    h, gu = c.forward()
    dgu, dw = c.grad()
    (o0, n0), (o1, n1) = c.segments[0], c.segments[1]
    c.x[o0, 3], c.d[o0, 5] = float("nan"), float("inf")
    c.w_gu[1, 0, 0], c.w_d[1, 0, 0] = float("inf"), float("nan")
    h2, gu2 = c.forward()
    dgu2, dw2 = c.grad()
    rows = torch.ones(c.R, dtype=torch.bool, device="cuda")
    rows[o0] = False
    rows[o1:o1 + n1] = False
    assert torch.equal(h2[rows], h[rows]) and torch.equal(gu2[rows], gu[rows])
    assert torch.equal(dgu2[rows], dgu[rows])
    clean = rows[c.lay["pair_row"].long()].view(N, 1)
    assert torch.equal(dw2[clean], dw[clean])
    assert not h2[o0].isfinite().all() and not dgu2[o0].isfinite().all()


def test_rows_of_no_expert_are_left():
    """A layout whose segments end before the rows do."""
    c = Case(700, 4, 1, 64, 136, seed=60, counts=[300, 200, 150, 50])
    h, gu = c.forward()
    dgu, dw = c.grad()
    c.lay["expert_counts"][3] = 20
    h2, gu2 = c.forward()
    dgu2, dw2 = c.grad()
    assert torch.equal(h2[:670], h[:670]) and h2[670:].isnan().all()
    assert torch.equal(gu2[:670], gu[:670]) and gu2[670:].isnan().all()
    assert torch.equal(dgu2[:670], dgu[:670]) and dgu2[670:].isnan().all()
    there = (c.lay["pair_row"] < 670).view(700, 1)
    assert torch.equal(dw2[there], dw[there]) and dw2[~there].isnan().all()


def test_gradient_against_differences():
    c = Case(9, 4, 2, 40, 24, seed=70)
    c.gu.copy_(c.forward()[1])
    dgu, dw = c.grad()
    pairs = ref.pairs_of_rows(c.lay["pair_row"])
    D = c.product(c.d, c.w_d, "ro,oi->ri")

    def loss(G, W):
        return (D * ref.swiglu(G, W.reshape(-1)[pairs].unsqueeze(1))).sum()

    e, G, W = 1e-5, c.gu.double(), c.w.double()
    for seed in range(4):
        v = normal(80 + seed, *G.shape, dtype=torch.float64)
        u = normal(90 + seed, *W.shape, dtype=torch.float64)
        step = (loss(G + e * v, W + e * u) - loss(G - e * v, W - e * u)) / (2 * e)
        told = (dgu.double() * v).sum() + (dw.double() * u).sum()
        mag = (dgu.double() * v).abs().sum() * BF16 + 1e-5 * (dw.double() * u).abs().sum()
        assert (step - told).abs() <= mag + 1e-6 * step.abs()


@pytest.mark.parametrize("N", [5, 400])
def test_streams_graphs_and_same_bits(N):
    c = Case(N, 8, 2, 136, 264, seed=100)
    h, gu = c.forward()
    dgu, dw = c.grad()
    out = [torch.zeros_like(t) for t in (h, gu, dgu, dw)]

    def both():
        moe.moe_gated_gemm(c.x, c.lay, c.shape, c.w_gu, c.w, out[1], out[0], c.ws)
        moe.moe_gated_gemm_grad(c.d, c.lay, c.shape, c.w_d, c.w, c.gu, out[2], out[3], c.ws)

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (h, gu, dgu, dw)))
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
    c = Case(300, 4, 2, 72, 136, seed=110)
    want = [*c.forward()[::-1], *c.grad()]
    pad = 2048

    def guarded(like):
        flat = torch.full((like.numel() + 2 * pad,), 7.0, dtype=like.dtype, device="cuda")
        return flat, flat[pad:-pad].view(like.shape)

    flats, outs = zip(*(guarded(t) for t in want))
    moe.moe_gated_gemm(c.x, c.lay, c.shape, c.w_gu, c.w, outs[0], outs[1], c.ws)
    moe.moe_gated_gemm_grad(c.d, c.lay, c.shape, c.w_d, c.w, c.gu, outs[2], outs[3], c.ws)
    for flat, out, t in zip(flats, outs, want):
        assert torch.equal(out, t)
        assert (flat[:pad] == 7.0).all() and (flat[-pad:] == 7.0).all()
