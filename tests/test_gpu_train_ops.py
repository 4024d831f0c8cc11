"""The activation, router and block-norm gradients against float64 definitions
and against differences of those definitions.

Tolerances.  A bf16 output rounds once (half a unit: 2^-9 relative, taken as
2^-8).  In fp32, the hardware exponential is good to 2 + 1.2 |x| units in the
last place (CUDA's bound; |x| < 8 here: 12 units, 1.4e-6) and divide, rsqrt and
the few products after it to some 2 units each: 4e-6 of the magnitude of the
terms.  A sum of n terms in fp32 adds at most n / 2 units of the terms'
magnitudes per level of its fixed order: 5e-6 (warp tree over at most 128 terms
a thread), 1e-5 over rows."""
import pytest
import torch

import train_ref as ref
from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, slack, what):
    """|got - want| <= slack (+ one rounding of a bf16 output), element by element."""
    assert torch.isfinite(got.float()).all(), what
    bound = slack + (BF16 * want.abs() if got.dtype == torch.bfloat16 else 0.0)
    over = ((got.double() - want).abs() - bound).max().item()
    assert over <= 0.0, f"{what}: {over} over the bound"


# ---- SwiGLU ----------------------------------------------------------------------------

def routed(N, E, k, I, dedup=False, seed=0):
    W = 2 if E % 2 == 0 else 1
    shape = moe.Shape(N, 8, E, k, W, I, dedup=dedup)
    ids = torch.empty(N, k, dtype=torch.int32, device="cuda")
    w = torch.empty(N, k, device="cuda")
    moe.moe_route(normal(gen(seed), N, E), shape, ids, w)
    lay, ws = moe.Layout(shape), moe.workspace(shape)
    moe.moe_dispatch_layout(ids, None, shape, lay, ws)
    return shape, lay, w


@pytest.mark.parametrize("N,E,k,I,dedup", [
    (1, 4, 1, 8, False), (5, 4, 3, 264, False), (67, 8, 2, 1032, True), (3, 64, 32, 4104, False),
    (2500, 8, 2, 72, False),     # enough rows for a warp each
])
def test_swiglu(N, E, k, I, dedup):
    shape, lay, w = routed(N, E, k, I, dedup)
    g = gen(1)
    gu = normal(g, shape.R, 2 * I, std=2.0, dtype=torch.bfloat16)
    dh = normal(g, shape.R, I, dtype=torch.bfloat16)
    h, dgu = torch.empty_like(dh), torch.empty_like(gu)
    dw = torch.full((N, k), float("nan"), device="cuda")
    moe.moe_swiglu(gu, w, lay, shape, h)
    moe.moe_swiglu_grad(dh, gu, w, lay, shape, dgu, dw)
    w_row = w.double().reshape(-1)[ref.pairs_of_rows(lay["pair_row"])].unsqueeze(1)
    G, D = gu.double(), dh.double()
    want = ref.swiglu(G, w_row)
    within(h, want, 4e-6 * want.abs(), "h")
    want, sums = ref.swiglu_grad(D, G, w_row)
    mag = w_row * D.abs() * (1 + G[:, :I].abs()) * G[:, I:].abs()
    mag = torch.cat([mag, w_row * D.abs() * G[:, :I].abs()], 1)
    within(dgu, want, 4e-6 * mag, "dgu")
    terms = (D * G[:, :I] * torch.sigmoid(G[:, :I]) * G[:, I:]).abs().sum(1)
    rows = lay["pair_row"].long()
    within(dw, sums[rows].view(N, k), 9e-6 * terms[rows].view(N, k), "dtopk_w")
    # without weights: ones, and no gradient wanted
    moe.moe_swiglu(gu, None, lay, shape, h)
    want = ref.swiglu(G, torch.ones_like(w_row))
    within(h, want, 4e-6 * want.abs(), "h, weights of one")
    moe.moe_swiglu_grad(dh, gu, None, lay, shape, dgu, None)
    want, _ = ref.swiglu_grad(D, G, torch.ones_like(w_row))
    within(dgu, want, 4e-6 * mag / w_row, "dgu, weights of one")


def test_swiglu_saturated_gates():
    """Gates far out: SiLU is 0 and x there, and its derivative 0 and 1."""
    shape, lay, w = routed(4, 4, 1, 64)
    gu = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda")
    gu[:, :32], gu[:, 32:64] = -1e4, 1e4
    h = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_swiglu(gu, None, lay, shape, h)
    assert (h[:, :32] == 0).all() and (h[:, 32:] == gu[:, 32:64]).all()
    dgu, dw = torch.empty_like(gu), torch.empty(4, 1, device="cuda")
    moe.moe_swiglu_grad(torch.ones_like(h), gu, None, lay, shape, dgu, dw)
    assert (dgu[:, :32] == 0).all() and (dgu[:, 32:64] == 1).all()
    assert (dgu[:, 64:96] == 0).all() and (dgu[:, 96:] == gu[:, 32:64]).all()


def test_swiglu_gradient_against_differences():
    shape, lay, w = routed(9, 4, 2, 40)
    g = gen(2)
    gu, dh = normal(g, 18, 80, dtype=torch.bfloat16), normal(g, 18, 40, dtype=torch.bfloat16)
    dgu, dw = torch.empty_like(gu), torch.empty(9, 2, device="cuda")
    moe.moe_swiglu_grad(dh, gu, w, lay, shape, dgu, dw)
    pairs = ref.pairs_of_rows(lay["pair_row"])

    def loss(G, W):
        return (dh.double() * ref.swiglu(G, W.reshape(-1)[pairs].unsqueeze(1))).sum()

    e, G, W = 1e-5, gu.double(), w.double()
    for seed in range(4):
        v, u = normal(gen(seed), 18, 80).double(), normal(gen(9 + seed), 9, 2).double()
        step = (loss(G + e * v, W + e * u) - loss(G - e * v, W - e * u)) / (2 * e)
        told = (dgu.double() * v).sum() + (dw.double() * u).sum()
        mag = (dgu.double() * v).abs().sum() * BF16 + 1e-5 * (dw.double() * u).abs().sum()
        assert (step - told).abs() <= mag + 1e-6 * step.abs()


# ---- the router's gradient ---------------------------------------------------------------

CALLS = {"full_softmax": "moe_route_full_softmax_grad", "sigmoid_bias": "moe_route_sigmoid_bias_grad"}


def run_route_grad(router, logits, ids, w, dw, shape):
    out = torch.full((shape.N, shape.E), float("nan"), device="cuda")
    if router == "softmax":
        moe.moe_route_grad(ids, w, dw, shape, out)
    else:
        getattr(moe, CALLS[router])(logits, ids, dw, shape, out)
    return out


def route(router, N, E, k, seed=0):
    shape = moe.Shape(N, 8, E, k, 1, 8)
    logits = normal(gen(seed), N, E, std=2.0)
    ids = torch.empty(N, k, dtype=torch.int32, device="cuda")
    w = torch.empty(N, k, device="cuda")
    if router == "softmax":
        moe.moe_route(logits, shape, ids, w)
    elif router == "full_softmax":
        moe.moe_route_full_softmax(logits, shape, ids, w)
    else:
        moe.moe_route_sigmoid_bias(logits, normal(gen(7), E, std=0.1), shape, ids, w)
    return shape, logits, ids, w


@pytest.mark.parametrize("router", ["softmax", "full_softmax", "sigmoid_bias"])
@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (3, 7, 7), (65, 8, 2), (130, 130, 5), (1000, 256, 8),
                                   (33, 257, 32), (20, 512, 6), (9, 1021, 4), (40, 1024, 32),
                                   (20011, 64, 6)])
def test_route_grad(router, N, E, k):
    shape, logits, ids, w = route(router, N, E, k)
    dw = normal(gen(3), N, k)
    got = run_route_grad(router, logits, ids, w, dw, shape)
    i = ids.long()
    want = ref.route_grad(logits.double(), i, dw.double(), router)
    wr = ref.route_weights(logits.double(), i, router)
    scale = (wr * dw.double().abs()).sum(1, keepdim=True)  # what the subtraction cancels against
    p = torch.softmax(logits.double(), 1) if router == "full_softmax" else \
        torch.zeros_like(want).scatter_(1, i, wr)
    d = torch.zeros_like(want).scatter_(1, i, dw.double().abs())
    within(got, want, 6e-6 * p * (d + scale), router)
    if router != "full_softmax":
        assert (got.double()[p == 0] == 0).all()


@pytest.mark.parametrize("router", ["softmax", "full_softmax", "sigmoid_bias"])
def test_route_gradient_against_differences(router):
    shape, logits, ids, w = route(router, 50, 24, 3)
    dw = normal(gen(4), 50, 3)
    got = run_route_grad(router, logits, ids, w, dw, shape).double()
    e, L, i = 1e-6, logits.double(), ids.long()
    for seed in range(4):
        v = normal(gen(seed), 50, 24).double()

        def loss(x):
            return (dw.double() * ref.route_weights(x, i, router)).sum()

        step = (loss(L + e * v) - loss(L - e * v)) / (2 * e)
        assert (step - (got * v).sum()).abs() <= 1e-5 * (got * v).abs().sum() + 1e-7


def test_route_grad_masked_experts():
    """Experts masked by -inf have probability 0 and gradient 0."""
    shape, logits, ids, w = route("full_softmax", 16, 40, 2)
    logits[:, 5:] = float("-inf")
    ids = torch.stack([torch.zeros(16), torch.ones(16)], 1).int().cuda()
    dw = normal(gen(5), 16, 2)
    got = run_route_grad("full_softmax", logits, ids, w, dw, shape)
    assert torch.isfinite(got).all() and (got[:, 5:] == 0).all() and (got[:, :5] != 0).all()


def test_route_grad_unaligned_rows():
    """fp32 tensors that start off the 16-byte grid (E odd, a view) still work."""
    shape, logits, ids, w = route("full_softmax", 31, 64, 4)
    dw = normal(gen(6), 31, 4)
    want = run_route_grad("full_softmax", logits, ids, w, dw, shape)
    flat = torch.empty(31 * 64 + 1, device="cuda")
    off = flat[1:].view(31, 64)
    off.copy_(logits)
    out = torch.empty(31 * 64 + 1, device="cuda")[1:].view(31, 64)
    moe.moe_route_full_softmax_grad(off, ids, dw, shape, out)
    assert (out - want).abs().max() <= 2e-6 * want.abs().max()


@pytest.mark.parametrize("router", ["softmax", "full_softmax", "sigmoid_bias"])
@pytest.mark.parametrize("N,E,k", [(9, 48, 1), (131, 64, 8), (77, 64, 9), (63, 100, 16),
                                   (50, 128, 17), (66, 252, 16), (35, 256, 17), (4097, 128, 6)])
def test_route_grad_of_several_tokens_a_warp(router, N, E, k):
    test_route_grad(router, N, E, k)


@pytest.mark.parametrize("router", ["softmax", "full_softmax", "sigmoid_bias"])
def test_route_grad_ids_out_of_range_take_no_part(router):
    """One choice of some tokens is no expert: the others' gradients are those of the choices
    that are left, and nothing is written outside the rows."""
    shape, logits, ids, w = route(router, 37, 24, 3)
    dw = normal(gen(8), 37, 3)
    bad = torch.zeros(37, 3, dtype=torch.bool, device="cuda")
    bad[::2, 1] = True
    broken = torch.where(bad, torch.tensor([-1, 24, 1 << 30], device="cuda").int()[None], ids)
    guard = torch.full((39, 24), 5.0, device="cuda")
    out = guard[1:38]
    if router == "softmax":
        moe.moe_route_grad(broken, w, dw, shape, out)
    else:
        getattr(moe, CALLS[router])(logits, broken, dw, shape, out)
    assert (guard[0] == 5).all() and (guard[38] == 5).all() and torch.isfinite(out).all()
    # as if that choice had no weight: zero where it was, the others among themselves
    i, keep = ids.long(), (~bad).double()
    L, d = logits.double(), dw.double() * keep
    if router == "softmax":
        wk = w.double() * keep
        g = wk * (d - (wk * d).sum(1, keepdim=True))
        want = torch.zeros_like(L).scatter_(1, i, g * keep)
    elif router == "full_softmax":
        p = torch.softmax(L, 1)
        dd = torch.zeros_like(L).scatter_(1, i, d)
        want = p * (dd - (p * dd).sum(1, keepdim=True))
    else:
        s = torch.sigmoid(L.gather(1, i)) * keep
        wk = s / s.sum(1, keepdim=True)
        g = wk * (d - (wk * d).sum(1, keepdim=True)) * (1 - torch.sigmoid(L.gather(1, i)))
        want = torch.zeros_like(L).scatter_(1, i, g * keep)
    # terms of at most |dw| and their sum, as in test_route_grad
    bound = 6e-6 * (dw.double().abs().sum(1, keepdim=True) * 2)
    assert ((out.double() - want).abs() <= bound).all()


# ---- block norms -------------------------------------------------------------------------

EPS, ALPHA = 1e-5, 0.75


def norm_case(N, H, gate, stream, post, seed=0):
    g = gen(seed)
    ns = moe.NormShape(N, H, post=post, pre=True, gate=gate, stream=stream, eps=EPS,
                       residual_scale=ALPHA)
    st = ns.stream_dtype
    t = dict(y=normal(g, N, H, std=3.0, dtype=torch.bfloat16), residual=normal(g, N, H, dtype=st),
             w_post=1 + normal(g, H, std=0.2) if post else None, w_pre=1 + normal(g, H, std=0.2),
             gate=None if gate == "none" else normal(g, *ns.gate_shape()),
             ds=normal(g, N, H, dtype=st), dx=normal(g, N, H, dtype=torch.bfloat16))
    return ns, t


def wide(t, ns):
    """The inputs in float64, the gate shaped to broadcast over the rows."""
    d = {n: None if v is None else v.double() for n, v in t.items()}
    d["g"] = 1.0 if ns.gate == "none" else d["gate"][:, None] if ns.gate == "token" else d["gate"]
    return d


NORMS = [(1, 8, "none", "bf16", True), (3, 72, "channel", "fp32", True),
         (130, 256, "token", "bf16", True), (37, 520, "channel", "bf16", False),
         (5, 264, "token", "fp32", False), (301, 1032, "channel", "bf16", True),
         (2, 7168, "token", "bf16", True), (700, 4096, "none", "fp32", True),
         (4, 8200, "channel", "bf16", True), (3, 16384, "token", "fp32", True),
         (2000, 64, "channel", "bf16", True)]


@pytest.mark.parametrize("N,H,gate,stream,post", NORMS)
def test_block_norm(N, H, gate, stream, post):
    ns, t = norm_case(N, H, gate, stream, post)
    d = wide(t, ns)
    s, x = torch.empty_like(t["residual"]), torch.empty_like(t["y"])
    rp, rn = (torch.empty(N, device="cuda") for _ in range(2))
    moe.moe_block_norm(t["y"], t["residual"], t["w_post"], t["gate"], t["w_pre"], ns, s, x,
                       rp if post else None, rn)
    want_s, want_x = ref.block_norm(d["y"], d["residual"], d["w_post"], d["g"], d["w_pre"], ALPHA,
                                    EPS, post, True)
    mag = ALPHA * d["residual"].abs() + (want_s - ALPHA * d["residual"]).abs()
    within(s, want_s, 4e-6 * mag, "s")
    r = ref.rstd(want_s, EPS)
    within(x, want_x, 8e-6 * mag * r * d["w_pre"].abs(), "x")
    assert ((rn.double() - r[:, 0]) / r[:, 0]).abs().max() <= 4e-6
    if post:
        r = ref.rstd(d["y"], EPS)[:, 0]
        assert ((rp.double() - r) / r).abs().max() <= 2e-6
    # in place on the residual stream
    again = t["residual"].clone()
    moe.moe_block_norm(t["y"], again, t["w_post"], t["gate"], t["w_pre"], ns, again, x)
    assert torch.equal(again, s)


def run_norm_grad(ns, t, s, rp, rn, accumulate=False, into=None):
    H = ns.H
    out = into or dict(
        dy=torch.empty_like(t["y"]), dr=torch.empty_like(t["residual"]),
        dw_post=torch.empty(H, device="cuda") if ns.post else None,
        dgate=None if t["gate"] is None else torch.empty_like(t["gate"]),
        dw_pre=torch.empty(H, device="cuda"))
    moe.moe_block_norm_grad(t["ds"], t["dx"], t["y"], s, t["w_post"], t["gate"], t["w_pre"], rp,
                            rn, ns, out["dy"], out["dr"], out["dw_post"], out["dgate"],
                            out["dw_pre"], moe.norm_workspace(ns), accumulate=accumulate)
    return out


@pytest.mark.parametrize("N,H,gate,stream,post", NORMS)
def test_block_norm_grad(N, H, gate, stream, post):
    ns, t = norm_case(N, H, gate, stream, post)
    s = normal(gen(5), N, H, dtype=ns.stream_dtype)  # a stored stream
    d = wide(t, ns)
    S = s.double()
    rn = ref.rstd(S, EPS).float()[:, 0]
    rp = ref.rstd(d["y"], EPS).float()[:, 0] if post else None
    got = run_norm_grad(ns, t, s, rp, rn)
    # the formula, and beside each value the magnitude of the terms it is made of
    r, one = rn.double()[:, None], torch.ones(H, dtype=torch.float64, device="cuda")
    sh, b = S * r, d["dx"] * d["w_pre"]
    g = d["ds"] + r * (b - sh * (b * sh).mean(1, keepdim=True))
    g_mag = d["ds"].abs() + r * (b.abs() + sh.abs() * (b * sh).abs().mean(1, keepdim=True))
    within(got["dr"], ALPHA * g, 8e-6 * ALPHA * g_mag, "dresidual")
    q = rp.double()[:, None] if post else 1.0
    w = d["w_post"] if post else one
    yh = d["y"] * q
    c, c_mag = d["g"] * g * w, abs(d["g"]) * g_mag * w.abs()
    dy = q * (c - (yh * (c * yh).mean(1, keepdim=True) if post else 0.0))
    dy_mag = q * (c_mag + (yh.abs() * (c_mag * yh.abs()).mean(1, keepdim=True) if post else 0.0))
    within(got["dy"], dy, 1.6e-5 * dy_mag, "dy")
    within(got["dw_pre"], (d["dx"] * sh).sum(0), 1.2e-5 * (d["dx"] * sh).abs().sum(0), "dw_pre")
    if post:
        within(got["dw_post"], (d["g"] * g * yh).sum(0),
               2.4e-5 * (abs(d["g"]) * g_mag * yh.abs()).sum(0), "dw_post")
    if gate != "none":
        dim = 0 if gate == "channel" else 1
        within(got["dgate"], (g * yh * w).sum(dim), 2.4e-5 * (g_mag * yh.abs() * w.abs()).sum(dim),
               "dgate")
    # adding to what is there: the sums over rows only
    acc = {n: None if v is None else v.clone() for n, v in got.items()}
    acc = run_norm_grad(ns, t, s, rp, rn, accumulate=True, into=acc)
    for n in ("dw_post", "dw_pre") + (("dgate",) if gate == "channel" else ()):
        if got[n] is not None:
            assert torch.equal(acc[n], got[n] + got[n]), n
    for n in ("dy", "dr") + (("dgate",) if gate == "token" else ()):
        assert torch.equal(acc[n], got[n]), n


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradient_against_differences(gate, post):
    N, H = 6, 48
    ns, t = norm_case(N, H, gate, "fp32", post, seed=3)
    s, x = torch.empty_like(t["residual"]), torch.empty_like(t["y"])
    rp, rn = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    moe.moe_block_norm(t["y"], t["residual"], t["w_post"], t["gate"], t["w_pre"], ns, s, x,
                       rp if post else None, rn)
    got = run_norm_grad(ns, t, s, rp if post else None, rn)
    d = wide(t, ns)
    names = dict(y="dy", residual="dr", w_pre="dw_pre")
    names.update(dict(w_post="dw_post") if post else {})
    names.update(dict(gate="dgate") if gate != "none" else {})

    def loss(v):
        g = 1.0 if gate == "none" else v["gate"][:, None] if gate == "token" else v["gate"]
        so, xo = ref.block_norm(v["y"], v["residual"], v["w_post"], g, v["w_pre"], ALPHA, EPS,
                                post, True)
        return (d["ds"] * so).sum() + (d["dx"] * xo).sum()

    e = 1e-6
    for name, grad in names.items():
        v = normal(gen(len(name)), *d[name].shape).double()
        up, down = dict(d, **{name: d[name] + e * v}), dict(d, **{name: d[name] - e * v})
        step = (loss(up) - loss(down)) / (2 * e)
        told = got[grad].double() * v
        rounding = BF16 if got[grad].dtype == torch.bfloat16 else 3e-5
        assert (step - told.sum()).abs() <= rounding * told.abs().sum() + 1e-6, name


def test_block_norm_parts():
    """The norm before the first block (no block output), the end of the last one
    (no norm after it), and rows of zeros."""
    N, H = 11, 136
    ns, t = norm_case(N, H, "none", "bf16", False)
    first = moe.NormShape(N, H, post=False, eps=EPS)
    x, rn = torch.empty_like(t["y"]), torch.empty(N, device="cuda")
    r = t["residual"].clone()
    r[3] = 0
    moe.moe_block_norm(None, r, None, None, None, first, None, x, None, rn)
    R = r.double()
    want = R * ref.rstd(R, EPS)
    within(x, want, 4e-6 * want.abs(), "x")
    assert (x[3] == 0).all() and rn[3].item() == pytest.approx(EPS ** -0.5, rel=1e-6)
    dr = torch.empty_like(r)
    moe.moe_block_norm_grad(None, t["dx"], None, r, None, None, None, None, rn, first, None, dr,
                            None, None, None, moe.norm_workspace(first))
    D = t["dx"].double()
    q = rn.double()[:, None]
    want = q * (D - R * q * (D * R * q).mean(1, keepdim=True))
    within(dr, want, 8e-6 * q * (D.abs() + (R * q).abs() * (D * R * q).abs().mean(1, keepdim=True)),
           "dresidual")
    last = moe.NormShape(N, H, post=True, pre=False, eps=EPS)
    s, rp = torch.empty_like(r), torch.empty(N, device="cuda")
    y = t["y"].clone()
    y[2] = 0
    moe.moe_block_norm(y, t["residual"], None, None, None, last, s, None, rp)
    Y = y.double()
    want = t["residual"].double() + Y * ref.rstd(Y, EPS)
    within(s, want, 4e-6 * (t["residual"].double().abs() + Y.abs() * ref.rstd(Y, EPS)), "s")
    assert torch.equal(s[2], t["residual"][2])
    dy, dw = torch.empty_like(y), torch.empty(H, device="cuda")
    moe.moe_block_norm_grad(t["ds"], None, y, None, None, None, None, rp, None, last, dy, dr, dw,
                            None, None, moe.norm_workspace(last))
    assert torch.equal(dr, t["ds"]) and torch.isfinite(dy.float()).all()


def test_block_norm_same_results_every_run():
    ns, t = norm_case(700, 4096, "channel", "bf16", True)
    s = normal(gen(5), 700, 4096, dtype=torch.bfloat16)
    rn = ref.rstd(s.double(), EPS).float()[:, 0]
    rp = ref.rstd(t["y"].double(), EPS).float()[:, 0]
    a, b = run_norm_grad(ns, t, s, rp, rn), run_norm_grad(ns, t, s, rp, rn)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_no_rows():
    ns = moe.NormShape(0, 64, gate="channel")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    n, v = torch.empty(0, device="cuda"), torch.ones(64, device="cuda")
    moe.moe_block_norm(e, e, v, v, v, ns, e, e, n, n)
    dw = [torch.ones(64, device="cuda") for _ in range(3)]
    moe.moe_block_norm_grad(e, e, e, e, v, v, v, n, n, ns, e, e, *dw, moe.norm_workspace(ns),
                            accumulate=True)
    assert all((w == 1).all() for w in dw)
    moe.moe_block_norm_grad(e, e, e, e, v, v, v, n, n, ns, e, e, *dw, moe.norm_workspace(ns))
    assert all((w == 0).all() for w in dw)
