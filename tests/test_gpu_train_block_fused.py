"""A training step with the fused gate, and Muon on its gradients."""
import pytest
import torch

import muon_ref
from combine_warp_top_gb300 import moe, train
from test_gpu_train_block import reference, rel

pytestmark = pytest.mark.gpu


def inputs(N, H, seed=5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(N, H, generator=g, device="cuda") for _ in range(2))


@pytest.mark.parametrize("N,H,E,k,I,alpha", [(1, 64, 4, 1, 64, 1.0), (37, 136, 8, 3, 72, 0.5),
                                             (600, 256, 16, 4, 264, 1.0)])
def test_block_step_against_autograd(N, H, E, k, I, alpha):
    block = train.MoETrainBlock(N, H, E, k, I, residual_scale=alpha, seed=N, fuse_gate=True)
    x, d_out = inputs(N, H)
    out = block.forward(x).clone()
    dx = block.backward(d_out).clone()
    assert moe.moe_get_error(block.ws) == 0
    want, d_want, grads = reference(block, x, block.ids, d_out)
    # the bound of the step without the fused gate, which rounds three tensors more
    assert rel(out, want) < 3e-2 and rel(dx, d_want) < 3e-2
    for n, p in block.grads.items():
        if n == "w_router" and k == 1:
            assert p.abs().max() < 1e-6
            continue
        assert rel(p, grads[n]) < 3e-2, n


def test_muon_step():
    """The update of every expert's gate, up and down matrix, the momentum, and the rest by a
    plain gradient step."""
    N, H, E, k, I = 300, 136, 4, 2, 72
    block = train.MoETrainBlock(N, H, E, k, I, seed=3, fuse_gate=True)
    x, d_out = inputs(N, H)
    lr, sgd_lr, decay = 0.03, 0.01, 0.1
    momenta = {}
    for step in range(2):
        block.forward(x)
        block.backward(d_out)
        before = {n: p.clone() for n, p in block.params.items()}
        block.muon(lr, weight_decay=decay, sgd_lr=sgd_lr)
        for n, p in block.params.items():
            g = block.grads[n]
            if n not in ("w_gate_up", "w_down"):
                assert torch.allclose(p, before[n] - sgd_lr * g, rtol=0, atol=2.0 ** -23 * 4), n
                continue
            M, K = (I, H) if n == "w_gate_up" else (H, I)
            u, momenta[n] = muon_ref.momentum(g, momenta.get(n, torch.zeros_like(g)), 0.95, True)
            u = u.view(-1, M, K)
            moved = (before[n].double() * (1 - lr * decay) - p.double()).view(-1, M, K)
            for e in range(u.shape[0]):
                want = muon_ref.orthogonal(u[e], 5, 1e-7)
                off = (muon_ref.orthogonal(u[e], 5, 1e-7, rounded=True) - want).norm()
                got = moved[e] / (lr * 0.2 * max(M, K) ** 0.5)
                # as for the operator alone; the fp32 step adds 2^-23 of the parameter
                slack = 2.0 ** -23 * before[n].norm() / (lr * 0.2 * max(M, K) ** 0.5)
                assert (got - want).norm() <= 2 * off + (2.0 ** -8 + 1e-3) * want.norm() + slack
        assert moe.moe_get_error(block.muon_ws) == 0
    assert torch.equal(block.w["w_down"], block.params["w_down"].bfloat16())


def test_training_runs():
    losses = train.main(steps=6, N=64, H=64, E=4, k=2, I=64, optimizer="muon")
    assert len(losses) == 6 and all(v == v for v in losses)


def test_muon_of_more_matrices_than_a_call_takes():
    block = train.MoETrainBlock(4, 8, 640, 1, 8, fuse_gate=True)
    for n, g in block.grads.items():
        g.copy_(torch.randn(g.shape, device="cuda"))
    before = block.params["w_gate_up"].clone()
    block.muon(1.0)
    moved = (before - block.params["w_gate_up"]).view(-1, 8, 8) / (0.2 * 8 ** 0.5)
    for e in (0, 1023, 1024, 1279):
        u, _ = muon_ref.momentum(block.grads["w_gate_up"].view(-1, 8, 8)[e], torch.zeros(
            8, 8, device="cuda"), 0.95, True)
        want = muon_ref.orthogonal(u, 5, 1e-7)
        off = (muon_ref.orthogonal(u, 5, 1e-7, rounded=True) - want).norm()
        # as for the operator alone; 2^-22 for the step's two fp32 roundings and the way back
        assert (moved[e] - want).norm() <= 2 * off + (2.0 ** -8 + 1e-3) * want.norm() + \
            2.0 ** -22 * before.abs().max() * 8 / (0.2 * 8 ** 0.5)
