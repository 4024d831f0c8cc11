"""A training step of one MoE block on the library's kernels.

    residual stream r
      x   = norm(r) w_pre                      moe_block_norm
      y   = MoE(x)                             router, dispatch, experts, combine
      out = alpha r + gate * norm(y) w_post    moe_block_norm

MoETrainBlock keeps the fp32 parameters, the activations that the backward pass
needs and the gradients; forward() and backward() run every product, activation,
norm and routing step as calls of the C ABI (moe.py).  The routing weights scale
h between an expert's two products (moe_swiglu), so the combine is a plain sum of a
token's k rows and each row's gradient is its token's: the dispatch and the combine
of the forward pass serve the backward pass with their roles exchanged.

    python -m combine_warp_top_gb300.train          # a few steps on a toy regression
    python -m combine_warp_top_gb300.train --muon   # with the fused gate and Muon
"""
from __future__ import annotations

import sys

import torch

from . import moe


class MoETrainBlock:
    """N tokens of width H, E experts, top-k softmax routing (renormalised over the
    selected experts), SwiGLU width I.

    params: fp32 tensors by name -- w_router [E, H], w_gate_up [E, 2*I, H] (gate rows
    first), w_down [E, H, I], w_pre, w_post, gate [H]; grads: the same, filled by
    backward() (added to when accumulate=True).  The expert and router products run
    on bf16 copies made by refresh(), which a step calls after it has changed params.

    What is rounded to bf16 on the way: every operand of a product, the router's
    matrix and its logits' gradient among them, for the tensor cores take no more (the
    logits themselves, the routing weights, all parameters' gradients and the residual
    stream with its gradient stay fp32); and the two parts of dx and their sum, the
    experts' and the router's, because the norm before the block takes its dx in bf16, as
    it gives x.  Each is 2^-8 at most, as at the block's other activations.
    """

    def __init__(self, N, H, E, k, I, residual_scale=1.0, eps=1e-6, seed=0, device="cuda",
                 fuse_gate=False):
        """fuse_gate: the gate and its gradient inside the products before and behind them
        (moe_gated_gemm, moe_gated_gemm_grad): less memory traffic, and g, u and dh are not
        rounded to bf16 on their way.  It pays on full batches: 8192 tokens of 2 of 8 experts,
        4096 -> 2 x 14336, 2062 and 1232 us forward and back where the calls apart take 2215 and
        1345; 4099 tokens of 6 of 64, 2048 -> 2 x 1408, 231 and 170, 258 and 178.  Its gradient has
        tiles of 256 rows only: with less than some 250 rows an expert it is slower than
        the calls apart (512 tokens of the latter 107 and 94 us, 16 tokens 90 and 66)."""
        self.fuse_gate = bool(fuse_gate)
        self.shape = s = moe.Shape(N, H, E, k, 1, I)
        # the router is a product of one group: all N rows, one matrix
        self.dense = moe.Shape(N, H, 1, 1, 1, I)
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        f32 = dict(dtype=torch.float32, device=device)
        bf = dict(dtype=torch.bfloat16, device=device)

        def normal(*size, std):
            return torch.randn(*size, generator=gen, **f32) * std

        self.params = dict(
            w_router=normal(E, H, std=H ** -0.5), w_gate_up=normal(E, 2 * I, H, std=H ** -0.5),
            w_down=normal(E, H, I, std=I ** -0.5), w_pre=torch.ones(H, **f32),
            w_post=torch.ones(H, **f32), gate=torch.ones(H, **f32))
        self.grads = {n: torch.zeros_like(p) for n, p in self.params.items()}
        self.w = {n: torch.empty_like(self.params[n], dtype=torch.bfloat16)
                  for n in ("w_router", "w_gate_up", "w_down")}
        # the router's product has a multiple of 8 columns: the rest are zeros
        E8 = (E + 7) // 8 * 8
        self.w["w_router"] = torch.zeros(E8, H, **bf)
        self.d_router = torch.zeros(1, E8, H, **f32)
        self.logits_all = torch.empty(N, E8, **f32)
        self.dlogits_bf = torch.zeros(N, E8, **bf)
        self.pre = moe.NormShape(N, H, post=False, pre=True, stream="fp32", eps=eps)
        self.post = moe.NormShape(N, H, post=True, pre=False, gate="channel", stream="fp32",
                                  eps=eps, residual_scale=residual_scale)
        self.layout = moe.Layout(s, device)
        self.dense_layout = moe.Layout(self.dense, device)
        self.dense_layout["expert_counts"].fill_(N)
        self.dense_layout["expert_offsets"].copy_(torch.tensor([0, N], dtype=torch.int32))
        self.ws = (moe.gated_workspace if fuse_gate else moe.workspace)(s, device)
        self.dense_ws = moe.workspace(self.dense, device)
        self.ws_pre, self.ws_post = (moe.norm_workspace(n, device) for n in (self.pre, self.post))
        R = s.R
        self.x, self.y, self.dy, self.dx = (torch.empty(N, H, **bf) for _ in range(4))
        self.rows, self.y_rows, self.d_rows = (torch.empty(R, H, **bf) for _ in range(3))
        self.gu, self.dgu = (torch.empty(R, 2 * I, **bf) for _ in range(2))
        self.h = torch.empty(R, I, **bf)
        self.dh = None if fuse_gate else torch.empty(R, I, **bf)
        self.logits, self.dlogits = (torch.empty(N, E, **f32) for _ in range(2))
        self.dx_router, self.dx_experts = (torch.empty(N, H, **bf) for _ in range(2))
        self.ids = torch.empty(N, k, dtype=torch.int32, device=device)
        self.topk_w, self.dtopk_w = (torch.empty(N, k, **f32) for _ in range(2))
        self.ones = torch.ones(N, k, **f32)
        self.rstd_pre, self.rstd_post = (torch.empty(N, **f32) for _ in range(2))
        # the residual stream as the block has taken it in, as it has left it, its gradient
        self.stream, self.out, self.d_stream = (torch.empty(N, H, **f32) for _ in range(3))
        self.momenta = None  # of muon()
        self.refresh()

    def refresh(self):
        """The bf16 copies of the matrices, from the fp32 parameters."""
        for n, t in self.w.items():
            t[:self.shape.E].copy_(self.params[n])

    def forward(self, residual):
        """residual fp32 [N, H]; returns the next residual stream, fp32 [N, H] (a buffer
        of the block, overwritten by the next call).  Keeps what backward() needs of this
        call, a copy of the residual among it, which the norm that reads it writes on its
        way: the tensor given may be the block's own output, and may change afterwards."""
        s, p, lay, ws = self.shape, self.params, self.layout, self.ws
        moe.moe_block_norm(None, residual, None, None, p["w_pre"], self.pre, self.stream, self.x,
                           None, self.rstd_pre)
        moe.moe_grouped_gemm(self.x, self.dense_layout, self.dense, self.w["w_router"].unsqueeze(0),
                             self.logits_all, self.dense_ws)
        self.logits.copy_(self.logits_all[:, :s.E])
        moe.moe_route(self.logits, s, self.ids, self.topk_w)
        moe.moe_dispatch_layout(self.ids, None, s, lay, ws)
        moe.moe_dispatch(self.x, lay, s, self.rows)
        if self.fuse_gate:
            moe.moe_gated_gemm(self.rows, lay, s, self.w["w_gate_up"], self.topk_w, self.gu, self.h,
                               ws)
        else:
            moe.moe_grouped_gemm(self.rows, lay, s, self.w["w_gate_up"], self.gu, ws)
            moe.moe_swiglu(self.gu, self.topk_w, lay, s, self.h)
        moe.moe_grouped_gemm(self.h, lay, s, self.w["w_down"], self.y_rows, ws)
        moe.moe_combine(self.y_rows, self.ones, lay, s, None, None, self.y)
        moe.moe_block_norm(self.y, self.stream, p["w_post"], p["gate"], None, self.post, self.out,
                           None, self.rstd_post)
        return self.out

    def backward(self, d_out, accumulate=False):
        """d_out fp32 [N, H], the gradient of forward()'s result; fills grads and returns
        the gradient of the residual stream, fp32 [N, H] (a buffer of the block)."""
        s, p, g, lay, ws = self.shape, self.params, self.grads, self.layout, self.ws
        acc = dict(accumulate=accumulate)
        moe.moe_block_norm_grad(d_out, None, self.y, None, p["w_post"], p["gate"], None,
                                self.rstd_post, None, self.post, self.dy, self.d_stream,
                                g["w_post"], g["gate"], None, self.ws_post, **acc)
        # the combine's gradient: each row of an expert gets its token's
        moe.moe_dispatch(self.dy, lay, s, self.d_rows)
        moe.moe_grouped_gemm_weight_grad(self.d_rows, self.h, lay, s, g["w_down"], ws, **acc)
        if self.fuse_gate:
            moe.moe_gated_gemm_grad(self.d_rows, lay, s, self.w["w_down"], self.topk_w, self.gu,
                                    self.dgu, self.dtopk_w, ws)
        else:
            moe.moe_grouped_gemm_input_grad(self.d_rows, lay, s, self.w["w_down"], self.dh, ws)
            moe.moe_swiglu_grad(self.dh, self.gu, self.topk_w, lay, s, self.dgu, self.dtopk_w)
        moe.moe_grouped_gemm_weight_grad(self.dgu, self.rows, lay, s, g["w_gate_up"], ws, **acc)
        moe.moe_grouped_gemm_input_grad(self.dgu, lay, s, self.w["w_gate_up"], self.d_rows, ws)
        # the dispatch's gradient: a token gets the sum of its rows'
        moe.moe_combine(self.d_rows, self.ones, lay, s, None, None, self.dx_experts)
        moe.moe_route_grad(self.ids, self.topk_w, self.dtopk_w, s, self.dlogits)
        self.dlogits_bf[:, :s.E].copy_(self.dlogits)
        if accumulate:
            self.d_router[0, :s.E].copy_(g["w_router"])
        moe.moe_grouped_gemm_weight_grad(self.dlogits_bf, self.x, self.dense_layout, self.dense,
                                         self.d_router, self.dense_ws, **acc)
        g["w_router"].copy_(self.d_router[0, :s.E])
        moe.moe_grouped_gemm_input_grad(self.dlogits_bf, self.dense_layout, self.dense,
                                        self.w["w_router"].unsqueeze(0), self.dx_router,
                                        self.dense_ws)
        torch.add(self.dx_experts, self.dx_router, out=self.dx)
        # s of this norm is the residual itself, so its gradient adds to the stream's
        moe.moe_block_norm_grad(self.d_stream, self.dx, None, self.stream, None, None,
                                p["w_pre"], None, self.rstd_pre, self.pre, None, self.d_stream,
                                None, None, g["w_pre"], self.ws_pre, **acc)
        return self.d_stream

    def sgd(self, lr):
        """A plain gradient step on the fp32 parameters."""
        for n, p in self.params.items():
            p.sub_(self.grads[n], alpha=lr)
        self.refresh()


    def muon(self, lr, momentum=0.95, nesterov=True, weight_decay=0.0, sgd_lr=None):
        """A step of the Muon optimiser on the experts' matrices (gate and up ones apart), a
        plain gradient step of sgd_lr (None: lr) on the router and the norms.  An
        orthogonalised [M, N] matrix has entries of about max(M, N) ** -0.5; times 0.2 of the
        root they are the size of an Adam step, so that lr and weight_decay mean the same."""
        s, p, g = self.shape, self.params, self.grads
        matrices = dict(w_gate_up=(2 * s.E, s.I, s.H), w_down=(s.E, s.H, s.I))
        if self.momenta is None:
            self.momenta = {n: torch.zeros_like(p[n]) for n in matrices}
            self.updates = {n: torch.empty_like(self.w[n]) for n in matrices}
            need = max(moe.moe_muon_workspace_bytes(moe.MuonShape(min(E, 1024), M, N))
                       for E, M, N in matrices.values())
            self.muon_ws = torch.empty(need, dtype=torch.uint8, device=p["w_down"].device)
            self.muon_ws[:256].zero_()
        for n, (E, M, N) in matrices.items():
            grads, momenta, updates = (t.view(E, M, N) for t in (g[n], self.momenta[n],
                                                                 self.updates[n]))
            for e in range(0, E, 1024):  # as many as a call takes
                part = slice(e, min(E, e + 1024))
                shape = moe.MuonShape(part.stop - e, M, N, momentum=momentum, nesterov=nesterov)
                moe.moe_muon_update(grads[part], momenta[part], shape, updates[part], self.muon_ws)
            p[n].mul_(1.0 - lr * weight_decay).add_(self.updates[n],
                                                    alpha=-lr * 0.2 * max(M, N) ** 0.5)
        for n in p:
            if n not in matrices:
                p[n].sub_(g[n], alpha=lr if sgd_lr is None else sgd_lr)
        self.refresh()


def main(steps=60, N=512, H=256, E=8, k=2, I=512, optimizer="sgd"):
    """Fits the block to a fixed random target and prints the loss.  optimizer "muon": with
    the fused gate and the experts' matrices by Muon."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(N, H, generator=gen, device="cuda")
    target = torch.randn(N, H, generator=gen, device="cuda")
    block = MoETrainBlock(N, H, E, k, I, fuse_gate=optimizer == "muon")
    losses = []
    for step in range(steps):
        err = block.forward(x) - target
        losses.append(err.square().mean().item())
        block.backward(err * (2.0 / N))
        if optimizer == "muon":
            block.muon(0.02, sgd_lr=0.05)
        else:
            block.sgd(0.05)
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    used = [block.ws, block.dense_ws] + ([block.muon_ws] if block.momenta is not None else [])
    assert all(moe.moe_get_error(ws) == 0 for ws in used)
    return losses


if __name__ == "__main__":
    main(optimizer="muon" if "--muon" in sys.argv[1:] else "sgd")
