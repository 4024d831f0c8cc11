"""The training step of a whole MoE block (train.MoETrainBlock) against autograd of
its float64 definition on the same bf16 weights and the same routing choice."""
import pytest
import torch

from combine_warp_top_gb300 import moe, train

pytestmark = pytest.mark.gpu


def reference(block, x, ids, d_out):
    """Loss gradients by autograd in float64; the routing ids are those the kernels chose."""
    s = block.shape
    p = {n: t.double() for n, t in block.params.items()}
    p.update({n: t[:s.E].double() for n, t in block.w.items()})
    p = {n: t.requires_grad_() for n, t in p.items()}
    r = x.double().requires_grad_()
    eps = block.pre.eps

    def norm(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)

    n = norm(r) * p["w_pre"]
    logits = n @ p["w_router"].T
    i = ids.long()
    w = torch.softmax(logits.gather(1, i), 1)
    y = torch.zeros_like(r)
    for e in range(s.E):
        t, j = (i == e).nonzero(as_tuple=True)
        if t.numel():
            a = n[t] @ p["w_gate_up"][e].T
            g, u = a.chunk(2, 1)
            y = y.index_add(0, t, (w[t, j, None] * g * torch.sigmoid(g) * u) @ p["w_down"][e].T)
    out = block.post.residual_scale * r + p["gate"] * norm(y) * p["w_post"]
    (out * d_out.double()).sum().backward()
    return out.detach(), r.grad, {n: t.grad for n, t in p.items()}


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("N,H,E,k,I,alpha", [(1, 64, 4, 1, 64, 1.0), (37, 136, 8, 3, 72, 0.5),
                                             (600, 256, 16, 4, 264, 1.0)])
def test_block_step_against_autograd(N, H, E, k, I, alpha):
    block = train.MoETrainBlock(N, H, E, k, I, residual_scale=alpha, seed=N)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(N, H, generator=g, device="cuda")
    d_out = torch.randn(N, H, generator=g, device="cuda")
    out = block.forward(x).clone()
    dx = block.backward(d_out).clone()
    assert moe.moe_get_error(block.ws) == 0 and moe.moe_get_error(block.dense_ws) == 0
    want, d_want, grads = reference(block, x, block.ids, d_out)
    # activations and their gradients are rounded to bf16 some six times on the way
    # (2^-9 each, independent): 5e-3 or so of each tensor's norm, 3e-2 is well clear
    assert rel(out, want) < 3e-2
    assert rel(dx, d_want) < 3e-2
    for n, p in block.grads.items():
        if n == "w_router" and k == 1:
            assert p.abs().max() < 1e-6  # one expert's weight is 1 whatever its logit
            continue
        assert rel(p, grads[n]) < 3e-2, n
    # a second backward pass that accumulates doubles the parameters' gradients
    first = {n: p.clone() for n, p in block.grads.items()}
    block.forward(x)
    block.backward(d_out, accumulate=True)
    for n, p in block.grads.items():
        assert torch.equal(p, first[n] + first[n]), n


def test_training_reduces_the_loss():
    losses = train.main(steps=40, N=256, H=128, E=4, k=2, I=128)
    assert losses[-1] < 0.5 * losses[0]
