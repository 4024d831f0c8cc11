"""Calls one after the other on a stream, each reading what the one before has just written:
a kernel's blocks may start before the writes of the kernel before it have landed, so the
results have to be, bit for bit, those of calls that are waited for one by one."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from combine_warp_top_gb300.train import MoETrainBlock

pytestmark = pytest.mark.gpu


@pytest.fixture
def waits(monkeypatch):
    """Makes every call of the binding wait for the GPU."""
    def start():
        for name in [n for n in dir(moe) if n.startswith("moe_")]:
            call = getattr(moe, name)
            if not callable(call) or "bytes" in name or "error" in name:
                continue

            def waiting(*a, _call=call, **kw):
                out = _call(*a, **kw)
                torch.cuda.synchronize()
                return out

            monkeypatch.setattr(moe, name, waiting)
    return start


def steps(N, H, E, k, I, n=4):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    block = MoETrainBlock(N, H, E, k, I, residual_scale=0.5)
    got = []
    for _ in range(n):
        x = torch.randn(N, H, generator=gen, device="cuda")
        d = torch.randn(N, H, generator=gen, device="cuda")
        got.append(block.forward(x).clone())
        got.append(block.backward(d).clone())
        got += [g.clone() for g in block.grads.values()]
        block.sgd(1e-3)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("size", [(1, 64, 4, 2, 64), (70, 256, 8, 2, 136), (600, 1024, 16, 4, 512)],
                         ids=str)
def test_training_steps(size, waits):
    chained = steps(*size)
    waits()
    one_by_one = steps(*size)
    assert len(chained) == len(one_by_one)
    assert all(torch.equal(a, b) for a, b in zip(chained, one_by_one))


@pytest.mark.parametrize("stream", ["bf16", "fp32"])
@pytest.mark.parametrize("N,H", [(3, 64), (300, 1000), (2000, 4096)])
def test_norms_in_place_over_and_over(N, H, stream, waits):
    """40 boundaries in a row on one residual buffer, each block's output being the norm
    before it."""
    ns = moe.NormShape(N, H, gate="channel", stream=stream, residual_scale=0.9)

    def run():
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        r = torch.randn(N, H, generator=gen, device="cuda").to(ns.stream_dtype)
        y = torch.randn(N, H, generator=gen, device="cuda").bfloat16()
        w, gate = torch.rand(H, generator=gen, device="cuda"), torch.rand(H, generator=gen,
                                                                          device="cuda")
        x = torch.empty_like(y)
        rp, rq = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        dy, dr = torch.empty_like(y), torch.empty_like(r)
        dw, dg, dv = (torch.zeros(H, device="cuda") for _ in range(3))
        ws = moe.norm_workspace(ns)
        for _ in range(40):
            moe.moe_block_norm(y, r, w, gate, w, ns, r, x, rp, rq)
            moe.moe_block_norm_grad(dr.zero_(), x, y, r, w, gate, w, rp, rq, ns, dy, dr, dw, dg,
                                    dv, ws, accumulate=True)
            x, y = y, x
        torch.cuda.synchronize()
        return r, x, y, dy, dr, dw, dg, dv, rp, rq

    chained = run()
    waits()
    assert all(torch.equal(a, b) for a, b in zip(chained, run()))


def test_products_that_feed_each_other(waits):
    """out of one product is the rows of the next, on workspaces that are shared."""
    E, N, C = 8, 96, 256
    shape = moe.Shape(N, 8, E, 1, 1, 8)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    counts = torch.tensor([12, 0, 30, 1, 7, 40, 6, 0], dtype=torch.int32)
    lay = moe.Layout(shape)
    lay["expert_counts"].copy_(counts)
    lay["expert_offsets"][1:].copy_(counts.cumsum(0).int())
    ws = moe.workspace(shape)
    w = (torch.randn(E, C, C, generator=gen, device="cuda") * C ** -0.5).bfloat16()
    rows = torch.randn(N, C, generator=gen, device="cuda").bfloat16()

    def run():
        a, b = rows.clone(), torch.empty_like(rows)
        dw = torch.zeros(E, C, C, device="cuda")
        for _ in range(30):
            moe.moe_grouped_gemm(a, lay, shape, w, b, ws)
            moe.moe_grouped_gemm_input_grad(b, lay, shape, w, a, ws)
            moe.moe_grouped_gemm_weight_grad(a, b, lay, shape, dw, ws, accumulate=True)
        torch.cuda.synchronize()
        return a, b, dw

    chained = run()
    waits()
    assert all(torch.equal(x, y) for x, y in zip(chained, run()))
