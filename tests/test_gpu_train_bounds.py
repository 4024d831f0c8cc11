"""Bounds of the training operators: nothing is written outside an output or to an
input, tensors that are only 16-byte aligned, offsets past 2^31 elements, other
streams and CUDA graphs."""
import pytest
import torch

import train_ref as ref
from combine_warp_top_gb300 import moe
from test_gpu_grouped import check, make_layout, segments

pytestmark = pytest.mark.gpu

GUARD = 4096 + 16  # the views start 16 bytes off a 32-byte boundary
FILL = 0xA5


class Box:
    """A tensor between two guard bands; `data` fills it, else it holds the fill byte."""
    made = []

    def __init__(self, shape, dtype, data=None):
        n = 1
        for s in shape:
            n *= s
        size = n * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((2 * GUARD + size,), FILL, dtype=torch.uint8, device="cuda")
        self.t = self.raw[GUARD:GUARD + size].view(dtype).view(shape)
        self.size = size
        if data is not None:
            self.t.copy_(data)
        self.before = self.raw.clone() if data is not None else None
        Box.made.append(self)

    def check(self):
        assert (self.raw[:GUARD] == FILL).all() and (self.raw[GUARD + self.size:] == FILL).all()
        if self.before is not None:
            assert torch.equal(self.raw, self.before), "an input has changed"


@pytest.fixture(autouse=True)
def boxes():
    Box.made = []
    yield
    torch.cuda.synchronize()
    for b in Box.made:
        b.check()


def rnd(*shape, dtype=torch.bfloat16, seed=0, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def put(*shape, dtype=torch.bfloat16, seed=0, std=1.0):
    return Box(shape, dtype, rnd(*shape, dtype=dtype, seed=seed, std=std)).t


def out(*shape, dtype=torch.bfloat16):
    return Box(shape, dtype).t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,ci,co", [([3, 0, 130, 17], 8, 24), ([40], 72, 136),
                                          ([5, 300], 264, 520)])
def test_grouped_guards(counts, ci, co, dtype):
    shape, lay, offs = make_layout(counts)
    R, E, ws = shape.N, shape.E, moe.workspace(shape)
    rows, dout = put(R, ci), put(R, co, seed=1)
    w = put(E, co, ci, seed=2)
    o, dr, dw = out(R, co, dtype=dtype), out(R, ci, dtype=dtype), out(E, co, ci, dtype=dtype)
    moe.moe_grouped_gemm(rows, lay, shape, w, o, ws)
    moe.moe_grouped_gemm_input_grad(dout, lay, shape, w, dr, ws)
    moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, dw, ws)
    r, d, m = rows.double(), dout.double(), w.double()
    for e, s in enumerate(segments(offs)):
        check(o[s], r[s] @ m[e].T, r[s].abs() @ m[e].T.abs(), ci)
        check(dr[s], d[s] @ m[e], d[s].abs() @ m[e].abs(), co)
        check(dw[e], d[s].T @ r[s], d[s].T.abs() @ r[s].abs(), counts[e])


@pytest.mark.parametrize("N,E,k,I", [(7, 4, 3, 40), (61, 8, 2, 136), (3000, 8, 2, 264)])
def test_swiglu_guards(N, E, k, I):
    shape = moe.Shape(N, 8, E, k, 1, I)
    ids, w = torch.empty(N, k, dtype=torch.int32, device="cuda"), out(N, k, dtype=torch.float32)
    moe.moe_route(rnd(N, E, dtype=torch.float32), shape, ids, w)
    lay = moe.Layout(shape)
    moe.moe_dispatch_layout(ids, None, shape, lay, moe.workspace(shape))
    gu, dh = put(shape.R, 2 * I), put(shape.R, I, seed=1)
    h, dgu, dw = out(shape.R, I), out(shape.R, 2 * I), out(N, k, dtype=torch.float32)
    moe.moe_swiglu(gu, w, lay, shape, h)
    moe.moe_swiglu_grad(dh, gu, w, lay, shape, dgu, dw)
    w_row = w.double().reshape(-1)[ref.pairs_of_rows(lay["pair_row"])].unsqueeze(1)
    want, sums = ref.swiglu_grad(dh.double(), gu.double(), w_row)
    assert (h.double() - ref.swiglu(gu.double(), w_row)).abs().max() < 0.05
    assert (dgu.double() - want).abs().max() < 0.05
    sums = sums[lay["pair_row"].long()].view(N, k)
    assert (dw.double() - sums).norm() <= 1e-5 * sums.norm()


@pytest.mark.parametrize("N,E,k", [(5, 6, 2), (33, 64, 6), (9, 1021, 3)])
def test_route_grad_guards(N, E, k):
    shape = moe.Shape(N, 8, E, k, 1, 8)
    logits = put(N, E, dtype=torch.float32)
    ids = torch.topk(logits, k, dim=1).indices.int()
    dw = put(N, k, dtype=torch.float32, seed=1)
    w = torch.softmax(logits.gather(1, ids.long()), 1)
    for router in ("softmax", "full_softmax", "sigmoid_bias"):
        d = out(N, E, dtype=torch.float32)
        if router == "softmax":
            moe.moe_route_grad(ids, w, dw, shape, d)
        else:
            getattr(moe, f"moe_route_{router}_grad")(logits, ids, dw, shape, d)
        want = ref.route_grad(logits.double(), ids.long(), dw.double(), router)
        assert (d.double() - want).abs().max() <= 1e-5 * want.abs().max()


@pytest.mark.parametrize("N,H", [(3, 8), (9, 40), (70, 200), (5, 520), (301, 1096), (4, 8264)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_norm_guards(N, H, stream):
    ns = moe.NormShape(N, H, gate="channel", stream=stream, eps=1e-5, residual_scale=0.5)
    st, f32 = ns.stream_dtype, torch.float32
    y, r = put(N, H), put(N, H, dtype=st, seed=1)
    wp, gate, wn = (put(H, dtype=f32, seed=s) for s in (2, 3, 4))
    s, x, rp, rn = out(N, H, dtype=st), out(N, H), out(N, dtype=f32), out(N, dtype=f32)
    moe.moe_block_norm(y, r, wp, gate, wn, ns, s, x, rp, rn)
    want_s, want_x = ref.block_norm(y.double(), r.double(), wp.double(), gate.double(),
                                    wn.double(), 0.5, 1e-5, True, True)
    assert (s.double() - want_s).norm() <= 4e-3 * want_s.norm()
    assert (x.double() - want_x).norm() <= 4e-3 * want_x.norm()
    ds, dx = put(N, H, dtype=st, seed=5), put(N, H, seed=6)
    dy, dr = out(N, H), out(N, H, dtype=st)
    dwp, dg, dwn = (out(H, dtype=f32) for _ in range(3))
    kept = s.clone()
    moe.moe_block_norm_grad(ds, dx, y, s, wp, gate, wn, rp, rn, ns, dy, dr, dwp, dg, dwn,
                            moe.norm_workspace(ns))
    assert torch.equal(s, kept)
    sh = s.double() * rn.double()[:, None]
    want = (dx.double() * sh).sum(0)
    assert (dwn.double() - want).norm() <= 1e-5 * want.norm()
    for t in (dy, dr, dwp, dg):
        assert torch.isfinite(t.float()).all()


def test_norm_and_swiglu_beyond_2_31_elements():
    N, H = 262208, 8192  # 2.148e9 elements
    assert N * H > 2 ** 31
    ns = moe.NormShape(N, H, eps=1e-5)
    y = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(y)
    at = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    y[at], r[at] = rnd(5, H), rnd(5, H, seed=1)
    s, x = torch.empty_like(y), torch.empty_like(y)
    rp, rn = (torch.empty(N, device="cuda") for _ in range(2))
    moe.moe_block_norm(y, r, None, None, None, ns, s, x, rp, rn)
    want_s, want_x = ref.block_norm(y[at].double(), r[at].double(), None, 1.0, None, 1.0, 1e-5,
                                    True, True)
    assert (s[at].double() - want_s).norm() <= 4e-3 * want_s.norm()
    assert (x[at].double() - want_x).norm() <= 4e-3 * want_x.norm()
    dy, dr = y.new_empty(N, H), y.new_empty(N, H)
    dw = torch.empty(H, device="cuda")
    moe.moe_block_norm_grad(r, y, y, s, None, None, None, rp, rn, ns, dy, dr, None, None, dw,
                            moe.norm_workspace(ns))
    want = (y[at].double() * s[at].double() * rn[at].double()[:, None]).sum(0)
    assert (dw.double() - want).norm() <= 1e-5 * want.norm()
    assert torch.isfinite(dy[at].float()).all() and (dr[N - 3] == 0).all()
    # the same memory as rows of [g | u]
    shape = moe.Shape(N, 8, 4, 1, 1, H // 2)
    lay = moe.Layout(shape)
    rows = torch.arange(N, dtype=torch.int32, device="cuda")
    lay["row_token"].copy_(rows)
    lay["pair_row"].copy_(rows)
    w = torch.full((N, 1), 0.5, device="cuda")
    h = x.view(-1)[:N * H // 2].view(N, H // 2)
    moe.moe_swiglu(y, w, lay, shape, h)
    want = ref.swiglu(y[at].double(), 0.5)
    assert (h[at].double() - want).norm() <= 4e-3 * want.norm()
    dgu, dtw = dr, torch.empty(N, 1, device="cuda")
    moe.moe_swiglu_grad(h, y, w, lay, shape, dgu, dtw)
    want, sums = ref.swiglu_grad(h[at].double(), y[at].double(), 0.5)
    assert (dgu[at].double() - want).norm() <= 4e-3 * want.norm()
    assert (dtw[at, 0].double() - sums).norm() <= 1e-5 * sums.norm()


def test_grouped_beyond_2_31_elements():
    counts, ci, co = [262000, 208], 64, 8200
    R = sum(counts)
    assert R * co > 2 ** 31
    shape, lay, offs = make_layout(counts)
    ws = moe.workspace(shape)
    rows, w = rnd(R, ci), rnd(2, co, ci, seed=1, std=0.125)
    o = torch.empty(R, co, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(rows, lay, shape, w, o, ws)
    at = torch.tensor([0, 261999, 262000, R - 1], device="cuda")
    for i in at.tolist():
        e = 0 if i < 262000 else 1
        want = rows[i].double() @ w[e].double().T
        check(o[i], want, rows[i].double().abs() @ w[e].double().T.abs(), ci)
    # back: the same memory as the output's gradient
    dr, dw = torch.empty(R, ci, device="cuda"), torch.empty(2, co, ci, device="cuda")
    moe.moe_grouped_gemm_input_grad(o, lay, shape, w, dr, ws)
    moe.moe_grouped_gemm_weight_grad(o, rows, lay, shape, dw, ws)
    for i in at.tolist():
        e = 0 if i < 262000 else 1
        check(dr[i], o[i].double() @ w[e].double(), o[i].double().abs() @ w[e].double().abs(), co)
    a, b = o[262000:].double(), rows[262000:].double()
    check(dw[1], a.T @ b, a.T.abs() @ b.abs(), 208)


def test_graph_and_other_stream():
    """The calls of a step captured into a CUDA graph, and on a stream of their own,
    give what they give at once."""
    counts = [70, 0, 129]
    shape, lay, offs = make_layout(counts)
    ws = moe.workspace(shape)
    R = shape.N
    rows, dout = rnd(R, 136), rnd(R, 264, seed=1)
    ns = moe.NormShape(R, 264, gate="channel", eps=1e-5)
    v = [rnd(264, dtype=torch.float32, seed=s) for s in (2, 3, 4)]
    nws = moe.norm_workspace(ns)

    def step(t, stream=None):
        moe.moe_grouped_gemm_weight_grad(dout, rows, lay, shape, t[0], ws, stream=stream)
        moe.moe_block_norm(dout, dout, v[0], v[1], v[2], ns, t[1], t[2], t[3], t[4],
                           stream=stream)
        moe.moe_block_norm_grad(dout, t[2], dout, t[1], v[0], v[1], v[2], t[3], t[4], ns, t[5],
                                t[6], t[7], t[8], t[9], nws, stream=stream)

    def fresh():
        f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        b = lambda: torch.zeros(R, 264, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        return [f(3, 264, 136), b(), b(), f(R), f(R), b(), b(), f(264), f(264), f(264)]

    want, on_stream, graphed = fresh(), fresh(), fresh()
    step(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(on_stream, side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graphed)
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, on_stream, graphed):
        assert torch.equal(a, b) and torch.equal(a, c)
