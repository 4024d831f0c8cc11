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
