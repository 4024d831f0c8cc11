"""MoELayer with 4-bit experts: the stages run together, against the definition in 64 bits on
the values that the weights stand for.

Tolerance.  The layer rounds h, each expert's rows and the output to bf16, 2^-8 each, and
the sums of the combine are fp32: 4 * 2^-8 of the largest output, 1.6e-2."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_w4 import normal, weights

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def quantised(w, group):
    q = torch.empty(*w.shape[:-1], w.shape[-1] // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(*w.shape[:-1], w.shape[-1] // group, dtype=bf, device="cuda")
    moe.moe_w4_quantize(w, q, scales)
    return q, scales


@pytest.mark.parametrize("N,H,E,k,W,I,dedup,group", [
    (1, 256, 8, 2, 1, 384, False, 128), (16, 512, 64, 6, 1, 192, False, 64),
    (33, 256, 16, 4, 4, 128, True, 32), (150, 384, 4, 2, 1, 256, False, 128),
])
def test_layer(N, H, E, k, W, I, dedup, group):
    shape = moe.Shape(N, H, E, k, W, I, dedup=dedup)
    wg, wu = normal(1, E, I, H, std=H ** -0.5), normal(2, E, I, H, std=H ** -0.5)
    wd = normal(3, E, H, I, std=I ** -0.5)
    layer = moe.MoELayer(shape, wg, wu, wd, w4=group)
    logits, x, res = normal(4, N, E, dtype=torch.float32), normal(5, N, H), normal(6, N, H)
    out = layer.forward(logits, x, res).clone()
    layer.check_device_errors()
    g, u, d = (weights(*quantised(w, group)) for w in (wg, wu, wd))
    ids = layer.topk_ids.view(N, k).long()
    w = torch.softmax(logits.double().gather(1, ids), 1)
    want = res.double()
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            a = x[t].double()
            p, q = a @ g[e].T, a @ u[e].T
            want = want.index_add(0, t, w[t, j, None] * ((p * torch.sigmoid(p) * q) @ d[e].T))
    assert (out.double() - want).abs().max() <= 4 * 2.0 ** -8 * want.abs().max()
    # the same from packed matrices, and replayed from a graph
    pair = (moe.quantize_w4(torch.cat([wg, wu], 1), group, gated=True), moe.quantize_w4(wd, group))
    again = moe.MoELayer(shape, None, None, None, w4=pair)
    graph = again.capture(logits, x, res)
    again.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again.out[:N], out[:N])


def test_layer_with_a_shared_expert():
    shape = moe.Shape(9, 256, 8, 2, 1, 128)
    ws = (normal(1, 8, 128, 256, std=0.06), normal(2, 8, 128, 256, std=0.06),
          normal(3, 8, 256, 128, std=0.09))
    shared = (normal(4, 64, 256, std=0.06), normal(5, 64, 256, std=0.06),
              normal(6, 256, 64, std=0.12))
    logits, x = normal(7, 9, 8, dtype=torch.float32), normal(8, 9, 256)
    routed = moe.MoELayer(shape, *ws, w4=64).forward(logits, x).clone()
    both = moe.MoELayer(shape, *ws, w4=64, shared=shared).forward(logits, x).clone()
    a = x.double()
    g, u, d = (w.double() for w in shared)
    want = routed.double() + ((a @ g.T) * torch.sigmoid(a @ g.T) * (a @ u.T)) @ d.T
    assert (both.double() - want).abs().max() <= 4 * 2.0 ** -8 * want.abs().max()
