"""Operators of an MoE layer's expert matrices, as cases that can be timed and compared.

  gated  an expert's gated feed-forward block up to its down product: both projections, the
         activation and the product with the routing weight in one kernel, and the gradient of the
         same from the rows behind the down product
  muon   the update of per-expert matrices by an orthogonalised momentum: the momentum itself and
         Newton-Schulz products
  w4     products of few rows with matrices of 4-bit weights that share a scale by groups, plain
         and gated: the experts of a decoding step

run() computes a case in plain 32-bit torch operations, or (own = True) by the package's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decoding step of 16 sequences on the 64-expert layer: the matrices stream by
        dict(name="gated forward, decode 16", op="gated", dir="forward", N=16, k=6, E=64, H=2048,
             I=1408, keep=False, skew=0.0),
        # a microbatch of odd length of the same layer in training: gate and up columns are kept
        dict(name="gated forward, 4099 tokens", op="gated", dir="forward", N=4099, k=6, E=64,
             H=2048, I=1408, keep=True, skew=0.0),
        # the Mixtral-shaped layer's full batch
        dict(name="gated forward, 8192 tokens", op="gated", dir="forward", N=8192, k=2, E=8,
             H=4096, I=14336, keep=True, skew=0.0),
        # that microbatch of the 64-expert layer, backwards
        dict(name="gated gradient, 4099 tokens", op="gated", dir="grad", N=4099, k=6, E=64, H=2048,
             I=1408, skew=0.0),
        # the Zipf-skewed layer's full batch, backwards: from a few rows to tens of thousands an
        # expert
        dict(name="gated gradient, 32768 tokens", op="gated", dir="grad", N=32768, k=8, E=128,
             H=4096, I=1536, skew=1.0),
        # the tiny layer's stacked gate and up matrices: launches count
        dict(name="muon, 8 of 512 x 128", op="muon", E=8, M=512, N=128, grad="fp32",
             momentum=True),
        # the 64-expert layer's down matrices
        dict(name="muon, 64 of 2048 x 1408", op="muon", E=64, M=2048, N=1408, grad="fp32",
             momentum=True),
        # 16 experts of the DeepSeek-V3-shaped layer: one matrix each
        dict(name="muon, 16 of 2048 x 7168", op="muon", E=16, M=2048, N=7168, grad="bf16",
             momentum=True),
        # one token of the DeepSeek-V3-shaped layer: 8 experts' down matrices
        dict(name="w4 down, 1 token", op="w4", gated=False, N=1, k=8, E=256, c_in=2048, c_out=7168,
             group=128, out="bf16", skew=0.0),
        # a decoding step of 16 sequences there: gate and up
        dict(name="w4 gated, 16 tokens", op="w4", gated=True, N=16, k=8, E=256, c_in=7168,
             c_out=2048, group=128, out="bf16", skew=0.0),
        # 64 sequences on the 64-expert layer, finer groups
        dict(name="w4 gated, 64 tokens", op="w4", gated=True, N=64, k=6, E=64, c_in=2048,
             c_out=1408, group=64, out="bf16", skew=0.0),
        # an odd, larger batch on the Mixtral-shaped layer: some 32 rows an expert
        dict(name="w4 down, 129 tokens", op="w4", gated=False, N=129, k=2, E=8, c_in=14336,
             c_out=4096, group=128, out="fp32", skew=0.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("gated", "gated", "muon", "w4", "w4"))
    E = rng.choice((8, 16, 48, 64, 128, 256))
    k = rng.randint(1, min(8, E))
    if op == "gated":
        c = dict(op=op, dir=rng.choice(("forward", "grad")), N=_log(rng, 1, 32768), k=k, E=E,
                 H=_log(rng, 64, 8192, 8), I=_log(rng, 64, 14336, 8),
                 skew=rng.choice((0.0, 0.5, 1.0)))
        if c["dir"] == "forward":
            c["keep"] = rng.random() < 0.6
        while E * c["H"] * c["I"] > 8 * 4096 * 14336:
            wide = max(("H", "I"), key=c.get)
            c[wide] = max(8, c[wide] // 24 * 8)
        while work(c)["flops"] > 3.8e12 or work(c)["bytes"] > 4e9:
            c["N"] //= 2
        return c
    if op == "muon":
        c = dict(op=op, E=_log(rng, 1, 64), M=_log(rng, 64, 8192, 8), N=_log(rng, 64, 8192, 8),
                 grad=rng.choice(("bf16", "fp32")), momentum=rng.random() < 0.7)
        while c["E"] > 1 and (work(c)["flops"] > 7.8e12 or c["E"] * c["M"] * c["N"] > 2.3e8):
            c["E"] //= 2
        while work(c)["flops"] > 7.8e12:
            wide = max(("M", "N"), key=c.get)
            c[wide] = c[wide] // 16 * 8
        return c
    group = rng.choice((32, 64, 128))
    c = dict(op=op, gated=rng.random() < 0.5, N=_log(rng, 1, 160), k=k, E=E,
             c_in=_log(rng, 128, 14336, group), c_out=_log(rng, 64, 14336, 8), group=group,
             out="bf16", skew=rng.choice((0.0, 1.0)))
    if not c["gated"]:
        c["out"] = rng.choice(("bf16", "fp32"))
    while c["E"] * c["c_in"] * c["c_out"] > 256 * 2048 * 7168:
        wide = max(("c_in", "c_out"), key=c.get)
        c[wide] = max(group, c[wide] // (2 * group) * group)
    while work(c)["flops"] > 3e11:
        c["N"] //= 2
    return c


# ---- inputs -------------------------------------------------------------------------------

def _routing(case, gen):
    """The selected experts of each token and their routing weights, popularity of the experts
    falling as 1/rank^skew, and the expert-major order of the (token, choice) pairs."""
    N, k, E = case["N"], case["k"], case["E"]
    logits = torch.randn(N, E, generator=gen, device="cuda")
    rank = torch.randperm(E, generator=gen, device="cuda")
    logits -= 2.0 * case["skew"] * torch.log(rank.float() + 1.0)
    top, ids = torch.topk(logits, k, dim=1)
    order = torch.argsort(ids.reshape(-1), stable=True)
    pair_row = torch.empty_like(order)
    pair_row[order] = torch.arange(order.numel(), device=order.device)
    return dict(counts=torch.bincount(ids.reshape(-1), minlength=E), order=order,
                pair_row=pair_row, row_token=order // k, topk_w=torch.softmax(top, 1))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="bf16", std=1.0):
        out = torch.empty(*shape, dtype=DT[dtype], device="cuda")
        return out.normal_(0.0, std, generator=gen)

    op = case["op"]
    if op == "muon":
        E, M, N = case["E"], case["M"], case["N"]
        # gradients of a trained matrix: a few strong directions over a noise of many
        rank = max(1, min(M, N) // 16)
        t = dict(grad=normal(E, M, N, dtype=case["grad"], std=1e-3))
        left, right = normal(E, M, rank, std=1e-1), normal(E, rank, N, std=2e-2)
        for e in range(E):
            t["grad"][e] += (left[e].float() @ right[e].float() * rank ** -0.5).to(t["grad"].dtype)
        if case["momentum"]:
            t["momentum"] = normal(E, M, N, dtype="fp32", std=3e-3)
        return t
    g = _routing(case, gen)
    R, E, k = case["N"] * case["k"], case["E"], case["k"]
    if op == "gated":
        H, I = case["H"], case["I"]
        if case["dir"] == "forward":
            return dict(g, rows=normal(R, H), w=normal(E, 2 * I, H, std=H ** -0.5))
        return dict(g, dout=normal(R, H, std=1e-2), w=normal(E, H, I, std=I ** -0.5),
                    gu=normal(R, 2 * I))
    ci, rows = case["c_in"], case["c_out"] * (2 if case["gated"] else 1)
    groups = ci // case["group"]
    q = torch.empty(E, rows, ci // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rows, groups, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        # normal weights by their groups' largest, in steps of a seventh of it
        w = normal(rows, groups, case["group"], dtype="fp32", std=ci ** -0.5)
        scales[e] = (w.abs().amax(2) / 7.0).bfloat16()
        v = (torch.round(w / scales[e].float().unsqueeze(2)) + 8.0).clamp(0.0, 15.0)
        v = v.to(torch.uint8).view(rows, ci // 2, 2)
        q[e] = v[:, :, 0] | (v[:, :, 1] << 4)
    return dict(g, rows=normal(R, ci), q=q, scales=scales)


STEPS, BETA, EPS = 5, 0.95, 1e-7
A, B, C = 3.4445, -4.7750, 2.0315  # the quintic of a Newton-Schulz step


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] != "muon":
        # the segments' lengths, which a program without grouped products needs on the host
        state["sizes"] = state["counts"].tolist()
    elif not own:
        state["new_momentum"] = torch.empty_like(state["momentum"]) if case["momentum"] else None
    if not own:
        return state
    # the package's handles and buffers: the dispatch layout that the forward pass has made,
    # workspaces, packed weights, the outputs
    from combine_warp_top_gb300 import moe
    op, N = case["op"], case["N"]
    bf = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if op == "muon":
        state["shape"] = moe.MuonShape(case["E"], case["M"], N, steps=STEPS, momentum=BETA,
                                       nesterov=True, eps=EPS)
        state["out"] = bf(case["E"], case["M"], N)
        state["ws"] = moe.muon_workspace(state["shape"])
        if case["momentum"]:
            state["new_momentum"] = torch.empty_like(state["momentum"])
        return state
    width = case["I"] if op == "gated" else case["c_out"]
    shape = moe.Shape(N, case["H"] if op == "gated" else 8, case["E"], case["k"], 1, width)
    layout = moe.Layout(shape)
    counts, R = state["counts"], shape.R
    for name, value in (("expert_counts", counts), ("row_token", state["row_token"]),
                        ("expert_offsets", torch.cat([counts.new_zeros(1), counts.cumsum(0)])),
                        ("rank_offsets", counts.new_tensor([0, R])),
                        ("pair_row", state["pair_row"])):
        layout[name].copy_(value)
    state.update(shape=shape, layout=layout)
    if op == "w4":
        state["w4"] = moe.pack_w4(state["q"], state["scales"], gated=case["gated"])
        state["ws"] = moe.w4_workspace(shape)
        state["out"] = torch.empty(R, case["c_out"], dtype=DT[case["out"]], device="cuda")
        del state["q"], state["scales"]
        return state
    state["ws"] = moe.gated_workspace(shape)
    if case["dir"] == "forward":
        state.update(h=bf(R, width), gu=bf(R, 2 * width) if case["keep"] else None)
    else:
        state.update(dgu=bf(R, 2 * width), dtopk_w=torch.empty_like(state["topk_w"]))
    return state


# ---- one pass -----------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return dict(gated=_gated, muon=_muon, w4=_w4)[case["op"]](case, state)


def _own(case, t):
    from combine_warp_top_gb300 import moe
    op = case["op"]
    if op == "muon":
        moe.moe_muon_update(t["grad"], t.get("momentum"), t["shape"], t["out"], t["ws"],
                            new_momentum=t.get("new_momentum"))
        return t["out"], t.get("new_momentum")
    if op == "w4":
        if case["gated"]:
            moe.moe_w4_gated_gemm(t["rows"], t["layout"], t["shape"], t["w4"], t["topk_w"],
                                  t["out"], t["ws"])
        else:
            moe.moe_w4_gemm(t["rows"], t["layout"], t["shape"], t["w4"], t["out"], t["ws"])
        return t["out"]
    if case["dir"] == "forward":
        moe.moe_gated_gemm(t["rows"], t["layout"], t["shape"], t["w"], t["topk_w"], t["gu"],
                           t["h"], t["ws"])
        return (t["h"], t["gu"]) if case["keep"] else t["h"]
    moe.moe_gated_gemm_grad(t["dout"], t["layout"], t["shape"], t["w"], t["topk_w"], t["gu"],
                            t["dgu"], t["dtopk_w"], t["ws"])
    return t["dgu"], t["dtopk_w"]


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _gated(case, t):
    weight = t["topk_w"].reshape(-1)[t["order"]].unsqueeze(1)
    if case["dir"] == "forward":
        gu = torch.cat([rows.float() @ w.float().T
                        for rows, w in zip(t["rows"].split(t["sizes"]), t["w"])])
        gate, up = gu.chunk(2, dim=1)
        h = (weight * _silu(gate) * up).bfloat16()
        return (h, gu.bfloat16()) if case["keep"] else h
    dh = torch.cat([dout.float() @ w.float()
                    for dout, w in zip(t["dout"].split(t["sizes"]), t["w"])])
    gate, up = t["gu"].float().chunk(2, dim=1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    dw = (dh * silu * up).sum(1)[t["pair_row"]].reshape(t["topk_w"].shape)
    scaled = weight * dh
    dgate = scaled * up * (sig * (1.0 + gate * (1.0 - sig)))
    return torch.cat([dgate, scaled * silu], dim=1).bfloat16(), dw


def _muon(case, t):
    update = t["grad"].float()
    if case["momentum"]:
        torch.add(t["grad"], t["momentum"], alpha=BETA, out=t["new_momentum"])
        update = update + BETA * t["new_momentum"]
    tall = case["M"] > case["N"]
    x = update.transpose(1, 2) if tall else update
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = A * x + (B * gram + C * (gram @ gram)) @ x
    out = (x.transpose(1, 2) if tall else x).bfloat16().contiguous()
    return out, t["new_momentum"]


def _w4(case, t):
    segments = []
    for e, rows in enumerate(t["rows"].split(t["sizes"])):
        if rows.shape[0] == 0:
            continue
        q = t["q"][e]
        v = torch.stack([q & 15, q >> 4], dim=2).float() - 8.0
        w = v.view(q.shape[0], -1, case["group"]) * t["scales"][e].float().unsqueeze(2)
        segments.append(rows.float() @ w.view(q.shape[0], -1).T)
    y = torch.cat(segments)
    if case["gated"]:
        gate, up = y.chunk(2, dim=1)
        y = t["topk_w"].reshape(-1)[t["order"]].unsqueeze(1) * _silu(gate) * up
    return y.to(DT[case["out"]])


# ---- the same from the definitions, in 64 bits --------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 9e12:
        return None
    t = _inputs(case, seed)
    if case["op"] == "muon":
        g = t["grad"].double()
        buf = None
        if case["momentum"]:
            buf = BETA * t["momentum"].double() + g
            g = g + BETA * buf
        out = torch.empty_like(g)
        for e in range(case["E"]):
            x = g[e] if case["M"] <= case["N"] else g[e].T
            x = x / (torch.linalg.vector_norm(x) + EPS)
            eye = torch.eye(x.shape[0], dtype=x.dtype, device="cuda")
            for _ in range(STEPS):
                p = x @ x.T
                x = (A * eye + p @ (B * eye + C * p)) @ x
            out[e] = x if case["M"] <= case["N"] else x.T
        return out, buf
    end = t["counts"].cumsum(0).tolist()
    seg = [slice(e - c, e) for e, c in zip(end, t["counts"].tolist())]
    w_row = t["topk_w"].double()[t["row_token"], t["order"] % case["k"]][:, None]
    if case["op"] == "w4":
        rows, cols = case["c_out"] * (2 if case["gated"] else 1), case["c_in"]
        y = torch.zeros(case["N"] * case["k"], rows, dtype=torch.float64, device="cuda")
        for e, s in enumerate(seg):
            if s.start == s.stop:
                continue
            w = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
            w[:, 0::2] = (t["q"][e] % 16).double() - 8
            w[:, 1::2] = (t["q"][e] // 16).double() - 8
            w *= t["scales"][e].double().repeat_interleave(case["group"], dim=1)
            y[s] = torch.einsum("ri,oi->ro", t["rows"][s].double(), w)
        if not case["gated"]:
            return y
        g, u = y[:, :case["c_out"]], y[:, case["c_out"]:]
        return w_row * g * torch.sigmoid(g) * u
    I = case["I"]
    if case["dir"] == "forward":
        gu = torch.cat([torch.einsum("ri,oi->ro", t["rows"][s].double(), t["w"][e].double())
                        for e, s in enumerate(seg)])
        h = w_row * gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        return (h, gu) if case["keep"] else h
    dh = torch.cat([torch.einsum("ro,oi->ri", t["dout"][s].double(), t["w"][e].double())
                    for e, s in enumerate(seg)])
    g, u = t["gu"][:, :I].double(), t["gu"][:, I:].double()
    sig = torch.sigmoid(g)
    dw = torch.zeros(case["N"], case["k"], dtype=torch.float64, device="cuda")
    dw[t["row_token"], t["order"] % case["k"]] = torch.einsum("ri,ri->r", dh, g * sig * u)
    return torch.cat([w_row * dh * u * (sig + g * sig * (1 - sig)), w_row * dh * g * sig], 1), dw


# ---- what a pass cannot do without --------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp32": 4}
    E = case["E"]
    if case["op"] == "muon":
        n = E * case["M"] * case["N"]
        m, l = sorted((case["M"], case["N"]))
        # products of symmetric matrices by half: the Gram matrix, its square, and their sum
        # times the whole matrix
        flops = STEPS * E * (3.0 * m * m * l + 1.0 * m * m * m)
        return {"bytes": n * (size[case["grad"]] + (8 if case["momentum"] else 0) + 2),
                "flops": flops}
    R, k = case["N"] * case["k"], case["k"]
    used = E * (1.0 - (1.0 - k / E) ** case["N"])  # experts with rows, for even routing
    if case["op"] == "gated":
        H, I = case["H"], case["I"]
        if case["dir"] == "forward":
            return {"bytes": 2 * R * H + 2 * used * 2 * I * H + R * I * (6 if case["keep"] else 2),
                    "flops": 4.0 * R * H * I}
        return {"bytes": 2 * R * H + 2 * used * H * I + R * I * 8 + R * 4,
                "flops": 2.0 * R * H * I}
    ci, rows = case["c_in"], case["c_out"] * (2 if case["gated"] else 1)
    return {"bytes": used * rows * (ci / 2 + 2 * ci / case["group"]) + 2 * R * ci
            + size[case["out"]] * R * case["c_out"], "flops": 2.0 * R * ci * rows}
