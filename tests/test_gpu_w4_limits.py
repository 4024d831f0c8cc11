"""4-bit products at the ends of what their layouts and streams may be, with the tolerances of the
operators' other tests."""
import pytest
import torch

from combine_warp_top_gb300 import moe
from test_gpu_w4 import Case

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
INVALID = 1


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,rows", [(8, 4096), (1024, 3000), (700, 16384)])
def test_segments_that_overlap_are_reported(E, rows, gated):
    """No more passes than the rows can fill are run: their number would leave 32 bits for large
    ones.  What is written is within the rows, and the next call is as it should be."""
    c = Case(rows, E, 1, 128, 40, 128, gated, seed=3)
    want = c.run()
    c.check(want)
    offsets, counts = c.lay["expert_offsets"].clone(), c.lay["expert_counts"].clone()
    c.lay["expert_offsets"].zero_()
    c.lay["expert_counts"].fill_(rows)
    pad = 4096
    flat = torch.full((want.numel() + 2 * pad,), 7.0, dtype=bf, device="cuda")
    c.run(out=flat[pad:-pad].view(want.shape))
    assert moe.moe_get_error(c.ws) == INVALID
    assert (flat[:pad] == 7.0).all() and (flat[-pad:] == 7.0).all()
    c.lay["expert_offsets"].copy_(offsets)
    c.lay["expert_counts"].copy_(counts)
    c.ws[:4] = 0
    out = c.run()
    assert torch.equal(out, want) and moe.moe_get_error(c.ws) == 0


@pytest.mark.parametrize("E,rows", [(1, 129), (4, 320), (1024, 1024), (5, 17), (33, 40)])
def test_the_most_passes_that_a_layout_can_have(E, rows):
    """One row to each expert but the last: not taken for an overlap."""
    counts = [1] * (E - 1) + [0]
    counts[-1] = rows - sum(counts)
    c = Case(rows, E, 1, 256, 40, 64, False, seed=4, counts=counts)
    c.check(c.run())


def test_weights_made_on_another_stream():
    """The helpers' own memory: nothing that the current stream still does to what was there
    before reaches them, and nothing gets it before the other stream is through."""
    E, rows, c_in, group = 4, 520, 1024, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    w = torch.randn(E, rows, c_in, generator=g, device="cuda").to(bf)
    want = moe.quantize_w4(w, group).data.clone()
    q = torch.empty(E, rows, c_in // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rows, c_in // group, dtype=bf, device="cuda")
    moe.moe_w4_quantize(w, q, scales)
    side = torch.cuda.Stream()
    sizes = [q.nbytes, scales.nbytes, want.nbytes]
    wait = 40_000_000  # cycles, 20 ms

    def make(packing):
        return (moe.pack_w4(q, scales, stream=side) if packing
                else moe.quantize_w4(w, group, stream=side))

    for packing in (False, True):
        torch.cuda.synchronize()
        # the memory is free and not yet written by the current stream
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(wait)
        for t in junk:
            t.fill_(170)
        del junk, t
        w4 = make(packing)
        torch.cuda.synchronize()
        assert torch.equal(w4.data, want)
        # the other stream is late
        with torch.cuda.stream(side):
            torch.cuda._sleep(wait)
        w4 = make(packing)
        junk = [torch.full((n,), 170, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert torch.equal(w4.data, want)
        del junk


@pytest.mark.parametrize("W,dedup,with_shared", [(1, False, False), (4, True, False), (1, False, True)])
def test_layer_of_an_empty_batch_is_a_noop(W, dedup, with_shared):
    E, H, I = 8, 128, 64
    shape = moe.Shape(0, H, E, 2, W, I, dedup=dedup)
    w = [torch.zeros(E, a, b, dtype=bf, device="cuda") for a, b in ((I, H), (I, H), (H, I))]
    shared = [t[0].contiguous() for t in w] if with_shared else None
    layer = moe.MoELayer(shape, *w, w4=64, shared=shared)
    x = torch.empty(0, H, dtype=bf, device="cuda")
    layer.out.fill_(7.0)
    for res in (None, x):
        out = layer.forward(torch.empty(0, E, device="cuda"), x, res)
        torch.cuda.synchronize()
        assert (out == 7.0).all()
    layer.check_device_errors()
    assert layer.kernel_launches_per_step() == 0
    assert (layer.layout["expert_counts"] == 0).all()
