"""Weights packed on another stream than the current one: nothing that the current stream still
does to what was in their memory before reaches them."""
import pytest
import torch

from combine_warp_top_gb300 import moe

pytestmark = pytest.mark.gpu


def test_weights_packed_on_another_stream():
    shape = moe.Shape(4, 256, 8, 2, 1, 384)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = [torch.randn(8, a, b, generator=g, device="cuda").bfloat16()
         for a, b in ((384, 256), (384, 256), (256, 384))]
    want = [t.clone() for t in moe.pack_weights(shape, *w)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory that is free and not yet written by the current stream
    junk = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(40_000_000)  # 20 ms
    for t in junk:
        t.fill_(7.0)
    del junk, t
    got = moe.pack_weights(shape, *w, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the other stream is late, and its results are dropped: their memory stays theirs
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    moe.pack_weights(shape, *w, stream=side)
    junk = [torch.full_like(t, 7.0) for t in want]
    torch.cuda.synchronize()
    assert all((t == 7.0).all() for t in junk)


def test_host_step_on_another_stream():
    """The inputs' device copies are the other stream's, too."""
    N, H, E = 512, 256, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    w = [torch.randn(E, a, b, generator=g, device="cuda").mul_(0.05).bfloat16()
         for a, b in ((384, H), (384, H), (H, 384))]
    layer = moe.MoELayer(moe.Shape(N, H, E, 2, 1, 384), *w)
    logits, x, res = (torch.randn(N, n, generator=g, device="cuda") for n in (E, H, H))
    x, res = x.bfloat16(), res.bfloat16()
    want = layer.forward(logits, x, res).cpu()
    host = [t.cpu().pin_memory() for t in (logits, x, res)]
    out = torch.empty(N, H, dtype=torch.bfloat16).pin_memory()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = [torch.empty_like(t, device="cuda") for t in host]
    torch.cuda._sleep(40_000_000)
    for t in junk:
        t.zero_()
    del junk, t
    layer.forward_host(*host, out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    layer.forward_host(*host, out.zero_(), stream=side)
    junk = [torch.zeros_like(t, device="cuda") for t in host]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all((t == 0).all() for t in junk)
