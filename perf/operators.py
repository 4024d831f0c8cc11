"""The operators of an MoE block's training step, as cases that can be timed and compared.

  grouped     matrix products grouped by expert over ragged row segments: the forward product,
              the gradient of its rows and the gradient of its weights
  swiglu      the gated activation between an expert's two products, scaled by each row's routing
              weight, and its gradient (routing weights included)
  route_grad  the gradient of the router's logits from that of the routing weights
  norm        RMS norms after a block and before the next one, fused with the block's gate, the
              residual scale and the residual add, and their gradient

run() computes a case in plain 32-bit torch operations, or (own = True) by the package's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the tiny workload's gate and up projections: a smoke-sized layer, where launches count
        dict(name="grouped forward, 64 tokens", op="grouped", dir="forward", N=64, k=2, E=8,
             c_in=128, c_out=512, out="bf16", skew=0.0),
        # one decoding step of 16 sequences on the 64-expert layer: the experts' weights stream by
        dict(name="grouped forward, decode 16", op="grouped", dir="forward", N=16, k=6, E=64,
             c_in=2048, c_out=2816, out="bf16", skew=0.0),
        # the Mixtral-shaped layer's down projection, backwards to its rows
        dict(name="grouped rows' gradient, 8192", op="grouped", dir="input_grad", N=8192, k=2, E=8,
             c_in=14336, c_out=4096, out="bf16", skew=0.0),
        # one microbatch of odd length on the 64-expert layer: its fp32 weight gradient is mostly
        # written, few rows an expert
        dict(name="grouped weights' gradient, 4099", op="grouped", dir="weight_grad", N=4099, k=6,
             E=64, c_in=2048, c_out=2816, out="fp32", skew=0.0),
        # the Zipf-skewed layer's down projection at full batch: from a few rows to tens of
        # thousands an expert
        dict(name="grouped weights' gradient, 32768", op="grouped", dir="weight_grad", N=32768, k=8,
             E=128, c_in=1536, c_out=4096, out="bf16", skew=1.0),
        # the activation of the Mixtral-shaped layer on a full batch
        dict(name="swiglu forward, 8192", op="swiglu", dir="forward", N=8192, k=2, E=8, I=14336,
             skew=0.0),
        # its gradient on the Zipf-skewed layer's full batch
        dict(name="swiglu gradient, 32768", op="swiglu", dir="grad", N=32768, k=8, E=128, I=1536,
             skew=1.0),
        # the router's gradient: weights renormalised over the selected experts
        dict(name="route gradient, 4096 of 64", op="route_grad", router="softmax", N=4096, k=6,
             E=64),
        # the same from probabilities over all experts, at a large batch
        dict(name="route gradient, 32768 of 256", op="route_grad", router="full_softmax", N=32768,
             k=8, E=256),
        # the block boundary of one decoding step of 16 sequences, gated token by token
        dict(name="norm forward, 16 tokens", op="norm", dir="forward", N=16, H=7168, gate="token",
             stream="bf16", post=True),
        # the block boundary of a prefill or training batch, fp32 residual stream, learned gate
        dict(name="norm forward, 4096 tokens", op="norm", dir="forward", N=4096, H=7168,
             gate="channel", stream="fp32", post=True),
        # its gradient on the Mixtral-shaped layer's full batch
        dict(name="norm gradient, 8192 tokens", op="norm", dir="grad", N=8192, H=4096,
             gate="channel", stream="bf16", post=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(lo, min(hi, int(round(v / step)) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(("grouped", "grouped", "swiglu", "route_grad", "norm"))
    E = rng.choice((8, 16, 48, 64, 128, 256))
    k = rng.randint(1, min(8, E))
    N = _log(rng, 1, 32768)
    if op == "grouped":
        c = dict(op=op, dir=rng.choice(("forward", "input_grad", "weight_grad")), N=N, k=k, E=E,
                 c_in=_log(rng, 64, 8192, 8), c_out=_log(rng, 64, 8192, 8),
                 out=rng.choice(("bf16", "fp32")), skew=rng.choice((0.0, 0.5, 1.0)))
        while E * c["c_in"] * c["c_out"] > 8 * 14336 * 4096:
            wide = max(("c_in", "c_out"), key=c.get)
            c[wide] = max(8, c[wide] // 24 * 8)
        while c["N"] * k * c["c_in"] * c["c_out"] > 16384 * 14336 * 4096 or \
                work(c)["bytes"] > 4.5e9:
            c["N"] //= 2
        return c
    if op == "swiglu":
        I = _log(rng, 64, 14336, 8)
        while N * k * I > 16384 * 14336:
            N = max(1, N // 2)
        return dict(op=op, dir=rng.choice(("forward", "grad")), N=N, k=k, E=E, I=I,
                    skew=rng.choice((0.0, 1.0)))
    if op == "route_grad":
        return dict(op=op, router=rng.choice(("softmax", "full_softmax", "sigmoid_bias")), N=N, k=k,
                    E=E)
    return dict(op=op, dir=rng.choice(("forward", "grad")), N=min(N, 16384),
                H=_log(rng, 64, 7168, 8), gate=rng.choice(("none", "channel", "token")),
                stream=rng.choice(("bf16", "fp32")), post=rng.choice((True, True, False)))


# ---- inputs -------------------------------------------------------------------------------

def _router(case, gen):
    """Logits whose experts' popularity falls as 1/rank^skew, and the k largest of each token."""
    N, k, E = case["N"], case["k"], case["E"]
    logits = torch.randn(N, E, generator=gen, device="cuda")
    rank = torch.randperm(E, generator=gen, device="cuda")
    logits -= 2.0 * case.get("skew", 0.0) * torch.log(rank.float() + 1.0)
    top, ids = torch.topk(logits, k, dim=1)
    return logits, ids, top


def _grouping(case, ids):
    """The expert-major order of the (token, choice) pairs: rows of an expert stand together,
    in the tokens' order."""
    E, k = case["E"], case["k"]
    order = torch.argsort(ids.reshape(-1), stable=True)
    pair_row = torch.empty_like(order)
    pair_row[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    return dict(counts=counts, order=order, pair_row=pair_row, row_token=order // k)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="bf16", std=1.0):
        out = torch.empty(*shape, dtype=DT[dtype], device="cuda")
        return out.normal_(0.0, std, generator=gen)

    op, N = case["op"], case["N"]
    if op in ("grouped", "swiglu"):
        logits, ids, top = _router(case, gen)
        g = _grouping(case, ids)
        R = N * case["k"]
        if op == "swiglu":
            t = dict(gu=normal(R, 2 * case["I"], std=1.5), topk_w=torch.softmax(top, 1))
            if case["dir"] == "grad":
                t["dh"] = normal(R, case["I"], std=1e-2)
            return dict(g, **t)
        ci, co, d = case["c_in"], case["c_out"], case["dir"]
        t = {}
        if d != "input_grad":
            t["rows"] = normal(R, ci)
        if d != "forward":
            t["dout"] = normal(R, co, std=1e-2)
        if d != "weight_grad":
            t["w"] = normal(case["E"], co, ci, std=ci ** -0.5)
        return dict(g, **t)
    if op == "route_grad":
        logits, ids, top = _router(case, gen)
        t = dict(logits=logits)
        if case["router"] == "softmax":
            t["topk_w"] = torch.softmax(top, 1)
        elif case["router"] == "full_softmax":
            t["topk_w"] = torch.softmax(logits, 1).gather(1, ids)
        else:
            bias = 0.1 * torch.randn(case["E"], generator=gen, device="cuda")
            scores = torch.sigmoid(logits)
            ids = torch.topk(scores + bias, case["k"], dim=1).indices
            top = scores.gather(1, ids)
            t["topk_w"] = top / top.sum(1, keepdim=True)
        return dict(t, ids=ids.int(), dtopk_w=normal(N, case["k"], dtype="fp32", std=1e-2))
    H, st = case["H"], case["stream"]
    w = lambda: 1.0 + normal(H, dtype="fp32", std=0.1)  # noqa: E731
    t = dict(y=normal(N, H, std=3.0), w_pre=w(), w_post=w() if case["post"] else None, gate=None)
    if case["gate"] == "channel":
        t["gate"] = 0.5 + normal(H, dtype="fp32", std=0.1)
    elif case["gate"] == "token":
        t["gate"] = torch.sigmoid(normal(N, dtype="fp32"))
    if case["dir"] == "forward":
        return dict(t, residual=normal(N, H, dtype=st, std=2.0))
    s = normal(N, H, dtype=st, std=2.0)
    return dict(t, s=s, ds=normal(N, H, dtype=st, std=1e-2), dx=normal(N, H, std=1e-2),
                rstd_pre=_rstd(s.float()), rstd_post=_rstd(t["y"].float()) if case["post"] else None)


EPS, RESIDUAL_SCALE = 1e-6, 0.75


def _rstd(v):
    return torch.rsqrt((v * v).mean(1) + EPS)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] == "grouped":
        # the segments' lengths, which a program without grouped products needs on the host
        state["sizes"] = state["counts"].tolist()
    if not own:
        return state
    # the package's handles and buffers: the dispatch layout that the forward pass has made, a
    # workspace, the outputs
    from combine_warp_top_gb300 import moe
    op, N = case["op"], case["N"]
    bf = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda *shape: torch.empty(*shape, dtype=torch.float32, device="cuda")  # noqa: E731
    if op == "norm":
        H = case["H"]
        state["shape"] = moe.NormShape(N, H, post=case["post"], pre=True, gate=case["gate"],
                                       stream=case["stream"], eps=EPS,
                                       residual_scale=RESIDUAL_SCALE)
        like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        if case["dir"] == "forward":
            state.update(s=torch.empty_like(state["residual"]), x=bf(N, H), rstd_pre=f32(N),
                         rstd_post=f32(N) if case["post"] else None)
        else:
            state.update(dy=bf(N, H), dresidual=torch.empty_like(state["s"]),
                         dw_post=like(state["w_post"]), dgate=like(state["gate"]),
                         dw_pre=like(state["w_pre"]), ws=moe.norm_workspace(state["shape"]))
        return state
    if op == "route_grad":
        state["shape"] = moe.Shape(N, 8, case["E"], case["k"], 1, 8)
        state["dlogits"] = f32(N, case["E"])
        return state
    I = case["I"] if op == "swiglu" else case["c_out"]
    shape = moe.Shape(N, case.get("c_in", 8), case["E"], case["k"], 1, I)
    layout = moe.Layout(shape)
    counts = state["counts"]
    for name, value in (("expert_counts", counts), ("row_token", state["row_token"]),
                        ("expert_offsets", torch.cat([counts.new_zeros(1), counts.cumsum(0)])),
                        ("rank_offsets", counts.new_tensor([0, shape.R])),
                        ("pair_row", state["pair_row"])):
        layout[name].copy_(value)
    state.update(shape=shape, layout=layout, ws=moe.workspace(shape))
    d, R = case["dir"], shape.R
    if op == "swiglu":
        state.update(dict(h=bf(R, I)) if d == "forward" else
                     dict(dgu=bf(R, 2 * I), dtopk_w=f32(N, case["k"])))
    else:
        size = dict(forward=(R, case["c_out"]), input_grad=(R, case["c_in"]),
                    weight_grad=(case["E"], case["c_out"], case["c_in"]))[d]
        state["out"] = torch.empty(*size, dtype=DT[case["out"]], device="cuda")
    return state


# ---- one pass -----------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return dict(grouped=_grouped, swiglu=_swiglu, route_grad=_route_grad,
                norm=_norm)[case["op"]](case, state)


def _own(case, t):
    from combine_warp_top_gb300 import moe
    op, d = case["op"], case.get("dir")
    if op == "grouped":
        if d == "forward":
            moe.moe_grouped_gemm(t["rows"], t["layout"], t["shape"], t["w"], t["out"], t["ws"])
        elif d == "input_grad":
            moe.moe_grouped_gemm_input_grad(t["dout"], t["layout"], t["shape"], t["w"], t["out"],
                                            t["ws"])
        else:
            moe.moe_grouped_gemm_weight_grad(t["dout"], t["rows"], t["layout"], t["shape"],
                                             t["out"], t["ws"])
        return t["out"]
    if op == "swiglu":
        if d == "forward":
            moe.moe_swiglu(t["gu"], t["topk_w"], t["layout"], t["shape"], t["h"])
            return t["h"]
        moe.moe_swiglu_grad(t["dh"], t["gu"], t["topk_w"], t["layout"], t["shape"], t["dgu"],
                            t["dtopk_w"])
        return t["dgu"], t["dtopk_w"]
    if op == "route_grad":
        if case["router"] == "softmax":
            moe.moe_route_grad(t["ids"], t["topk_w"], t["dtopk_w"], t["shape"], t["dlogits"])
        elif case["router"] == "full_softmax":
            moe.moe_route_full_softmax_grad(t["logits"], t["ids"], t["dtopk_w"], t["shape"],
                                            t["dlogits"])
        else:
            moe.moe_route_sigmoid_bias_grad(t["logits"], t["ids"], t["dtopk_w"], t["shape"],
                                            t["dlogits"])
        return t["dlogits"]
    if d == "forward":
        moe.moe_block_norm(t["y"], t["residual"], t["w_post"], t["gate"], t["w_pre"], t["shape"],
                           t["s"], t["x"], t["rstd_post"], t["rstd_pre"])
        return t["s"], t["x"], t["rstd_post"], t["rstd_pre"]
    moe.moe_block_norm_grad(t["ds"], t["dx"], t["y"], t["s"], t["w_post"], t["gate"], t["w_pre"],
                            t["rstd_post"], t["rstd_pre"], t["shape"], t["dy"], t["dresidual"],
                            t["dw_post"], t["dgate"], t["dw_pre"], t["ws"])
    return t["dy"], t["dresidual"], t["dw_post"], t["dgate"], t["dw_pre"]


def _grouped(case, t):
    out = DT[case["out"]]
    sizes = t["sizes"]
    if case["dir"] == "forward":
        segments = zip(t["rows"].float().split(sizes), t["w"].float())
        return torch.cat([rows @ w.T for rows, w in segments]).to(out)
    if case["dir"] == "input_grad":
        segments = zip(t["dout"].float().split(sizes), t["w"].float())
        return torch.cat([dout @ w for dout, w in segments]).to(out)
    segments = zip(t["dout"].float().split(sizes), t["rows"].float().split(sizes))
    return torch.stack([dout.T @ rows for dout, rows in segments]).to(out)


def _swiglu(case, t):
    gate, up = t["gu"].float().chunk(2, dim=1)
    weight = t["topk_w"].reshape(-1)[t["order"]].unsqueeze(1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if case["dir"] == "forward":
        return (weight * (gate * sig) * up).bfloat16()
    dh = t["dh"].float()
    silu = gate * sig
    dw = (dh * silu * up).sum(1)[t["pair_row"]].reshape(t["topk_w"].shape)
    scaled = weight * dh
    dgate = scaled * up * (sig * (1.0 + gate * (1.0 - sig)))
    return torch.cat([dgate, scaled * silu], dim=1).bfloat16(), dw


def _route_grad(case, t):
    ids, dw = t["ids"].long(), t["dtopk_w"]
    if case["router"] == "full_softmax":
        e = torch.exp(t["logits"] - t["logits"].amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        dp = torch.zeros_like(p).scatter_(1, ids, dw)
        return p * (dp - (p.gather(1, ids) * dw).sum(1, keepdim=True))
    if case["router"] == "softmax":
        w = t["topk_w"]
        d = w * (dw - (w * dw).sum(1, keepdim=True))
    else:
        s = 1.0 / (1.0 + torch.exp(-t["logits"].gather(1, ids)))
        total = s.sum(1, keepdim=True)
        d = (dw - (s / total * dw).sum(1, keepdim=True)) / total * s * (1.0 - s)
    return torch.zeros_like(t["logits"]).scatter_(1, ids, d)


def _gate(case, t):
    if t["gate"] is None:
        return 1.0
    return t["gate"] if case["gate"] == "channel" else t["gate"].unsqueeze(1)


def _norm(case, t):
    y = t["y"].float()
    gate = _gate(case, t)
    if case["dir"] == "forward":
        rstd_post = _rstd(y) if case["post"] else None
        z = y * rstd_post.unsqueeze(1) * t["w_post"] if case["post"] else y
        s = RESIDUAL_SCALE * t["residual"].float() + gate * z
        rstd_pre = _rstd(s)
        x = s * rstd_pre.unsqueeze(1) * t["w_pre"]
        return s.to(DT[case["stream"]]), x.bfloat16(), rstd_post, rstd_pre
    s, dx = t["s"].float(), t["dx"].float()
    r_pre = t["rstd_pre"].unsqueeze(1)
    s_hat = s * r_pre
    dw_pre = (dx * s_hat).sum(0)
    dx = dx * t["w_pre"]
    grad = t["ds"].float() + r_pre * (dx - s_hat * (dx * s_hat).mean(1, keepdim=True))
    dresidual = (RESIDUAL_SCALE * grad).to(DT[case["stream"]])
    y_hat = y * t["rstd_post"].unsqueeze(1) if case["post"] else y
    z = y_hat * t["w_post"] if case["post"] else y_hat
    dgate = None
    if t["gate"] is not None:
        dgate = (grad * z).sum(0 if case["gate"] == "channel" else 1)
    dz = gate * grad
    if not case["post"]:
        return dz.bfloat16(), dresidual, None, dgate, dw_pre
    dw_post = (dz * y_hat).sum(0)
    dz = dz * t["w_post"]
    dy = t["rstd_post"].unsqueeze(1) * (dz - y_hat * (dz * y_hat).mean(1, keepdim=True))
    return dy.bfloat16(), dresidual, dw_post, dgate, dw_pre


# ---- the same from the definitions, in 64 bits --------------------------------------------

def exact(case, seed):
    t = _inputs(case, seed)
    t = {n: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for n, v in t.items()}
    op, d, N = case["op"], case.get("dir"), case["N"]
    if op == "grouped":
        if 2.0 * N * case["k"] * case["c_in"] * case["c_out"] > 8e12:
            return None
        end = t["counts"].cumsum(0).tolist()
        seg = [slice(e - c, e) for e, c in zip(end, t["counts"].tolist())]
        if d == "forward":
            return torch.cat([torch.einsum("ri,oi->ro", t["rows"][s], t["w"][e])
                              for e, s in enumerate(seg)])
        if d == "input_grad":
            return torch.cat([torch.einsum("ro,oi->ri", t["dout"][s], t["w"][e])
                              for e, s in enumerate(seg)])
        return torch.stack([torch.einsum("ro,ri->oi", t["dout"][s], t["rows"][s]) for s in seg])
    if op == "swiglu":
        I, k = case["I"], case["k"]
        rows, slots = t["row_token"], t["order"] % k
        w = t["topk_w"][rows, slots][:, None]
        g, u = t["gu"][:, :I], t["gu"][:, I:]
        sig = torch.sigmoid(g)
        if d == "forward":
            return w * g * sig * u
        dw = torch.zeros_like(t["topk_w"])
        dw[rows, slots] = torch.einsum("ri,ri->r", t["dh"], g * sig * u)
        dg = w * t["dh"] * u * (sig + g * sig * (1 - sig))
        return torch.cat([dg, w * t["dh"] * g * sig], 1), dw
    if op == "route_grad":
        ids, dw = t["ids"].long(), t["dtopk_w"]
        take = torch.zeros(N, case["k"], case["E"], dtype=torch.float64, device="cuda")
        take.scatter_(2, ids[:, :, None], 1.0)
        if case["router"] == "full_softmax":
            p = torch.softmax(t["logits"], 1)
            dp = torch.einsum("nk,nke->ne", dw, take)
            return p * dp - p * (p * dp).sum(1, keepdim=True)
        if case["router"] == "softmax":
            w = t["topk_w"]  # an input, as the forward pass has left it
            return torch.einsum("nk,nke->ne", w * dw - w * (w * dw).sum(1, keepdim=True), take)
        s = torch.sigmoid(t["logits"].gather(1, ids))
        S = s.sum(1, keepdim=True)
        ds = dw / S - (s * dw).sum(1, keepdim=True) / S ** 2
        return torch.einsum("nk,nke->ne", ds * s * (1 - s), take)
    y, H = t["y"], case["H"]
    gate = torch.ones((), dtype=torch.float64, device="cuda") if t["gate"] is None else t["gate"]
    gate = gate[:, None] if case["gate"] == "token" else gate
    if d == "forward":
        r_post = (y.square().sum(1) / H + EPS) ** -0.5 if case["post"] else None
        z = t["w_post"] * y * r_post[:, None] if case["post"] else y
        s = RESIDUAL_SCALE * t["residual"] + gate * z
        r_pre = (s.square().sum(1) / H + EPS) ** -0.5
        return s, t["w_pre"] * s * r_pre[:, None], r_post, r_pre
    a, r = t["dx"] * t["w_pre"], t["rstd_pre"][:, None]
    grad = t["ds"] + r * a - r ** 3 * t["s"] * (a * t["s"]).sum(1, keepdim=True) / H
    dw_pre = torch.einsum("nh,nh,nl->h", t["dx"], t["s"], r)
    q = t["rstd_post"][:, None] if case["post"] else torch.ones(N, 1, dtype=a.dtype, device="cuda")
    w = t["w_post"] if case["post"] else torch.ones(H, dtype=a.dtype, device="cuda")
    share = grad * y * q
    dgate = None
    if case["gate"] != "none":
        dgate = (share * w).sum(0 if case["gate"] == "channel" else 1)
    b = gate * grad * w
    dy = q * b - q ** 3 * y * (b * y).sum(1, keepdim=True) / H if case["post"] else b
    dw_post = (gate * share).sum(0) if case["post"] else None
    return dy, RESIDUAL_SCALE * grad, dw_post, dgate, dw_pre


# ---- what a pass cannot do without --------------------------------------------------------

def work(case):
    op, d, N = case["op"], case.get("dir"), case["N"]
    size = {"bf16": 2, "fp32": 4}
    if op == "grouped":
        R, ci, co, E = N * case["k"], case["c_in"], case["c_out"], case["E"]
        used = E * (1.0 - (1.0 - case["k"] / E) ** N)  # experts with rows, for even routing
        out = size[case["out"]]
        if d == "forward":
            moved = 2 * R * ci + 2 * used * ci * co + out * R * co
        elif d == "input_grad":
            moved = 2 * R * co + 2 * used * ci * co + out * R * ci
        else:
            moved = 2 * R * (ci + co) + out * E * ci * co
        return {"bytes": moved, "flops": 2.0 * R * ci * co}
    if op == "swiglu":
        R, I = N * case["k"], case["I"]
        moved = R * I * 2 * (3 if d == "forward" else 5) + R * (4 + 8)
        return {"bytes": moved + (R * 4 if d == "grad" else 0),
                "flops": R * I * (6.0 if d == "forward" else 14.0)}
    if op == "route_grad":
        E, k = case["E"], case["k"]
        reads = E * 4 if case["router"] == "full_softmax" else k * 4
        return {"bytes": N * (E * 4 + reads + k * 8), "flops": N * (6.0 * E + 4.0 * k)}
    H, st = case["H"], size[case["stream"]]
    if d == "forward":
        return {"bytes": N * H * (2 + 2 * st + 2) + 8 * N, "flops": 9.0 * N * H}
    return {"bytes": N * H * (2 + 2 + 2 * st + 2 + st) + 8 * N + 20 * H, "flops": 24.0 * N * H}
