"""MoETrainBlock's backward pass does not depend on what has become of the tensor that
forward() was given: the block's own output, or a tensor that has changed since."""
import pytest
import torch

from combine_warp_top_gb300 import train
from test_gpu_train_block import reference, rel

pytestmark = pytest.mark.gpu
SIZE = dict(N=70, H=136, E=8, k=2, I=72, residual_scale=0.5)


def noise(seed, N=70, H=136):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(N, H, generator=g, device="cuda")


def gradients(block, d_out):
    dx = block.backward(d_out).clone()
    return dict({n: g.clone() for n, g in block.grads.items()}, residual=dx)


def same(a, b):
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_own_output():
    """r = block.forward(r), twice: the second call reads the buffer that it writes."""
    d = noise(1)
    block = train.MoETrainBlock(**SIZE)
    x = block.forward(block.forward(noise(0))).clone()
    got = gradients(block, d)
    other = train.MoETrainBlock(**SIZE)
    middle = other.forward(noise(0)).clone()
    assert torch.equal(other.forward(middle), x)
    same(got, gradients(other, d))
    want, d_want, grads = reference(other, middle, other.ids, d)
    assert rel(x, want) < 3e-2 and rel(got["residual"], d_want) < 3e-2
    for n, g in grads.items():
        assert rel(got[n], g) < 3e-2, n


def test_input_changes_before_the_backward_pass():
    d = noise(1)
    block, x = train.MoETrainBlock(**SIZE), noise(0)
    block.forward(x)
    want = gradients(block, d)
    block.forward(x)
    x.fill_(float("nan"))
    same(gradients(block, d), want)


def test_two_blocks_and_another_batch():
    """The first block takes another batch before the second one's backward pass."""
    d = noise(1)
    first, second = train.MoETrainBlock(**SIZE), train.MoETrainBlock(seed=1, **SIZE)
    second.forward(first.forward(noise(0)).clone())
    want = gradients(second, d)
    second.forward(first.forward(noise(0)))
    first.forward(noise(2))
    same(gradients(second, d), want)


def test_gradient_of_the_stream_as_input():
    """The buffers that backward() returns are as good an input as any."""
    block = train.MoETrainBlock(**SIZE)
    block.forward(noise(0))
    dx = block.backward(noise(1))
    kept = dx.clone()
    block.forward(dx)
    got = gradients(block, dx)
    block.forward(kept)
    same(gradients(block, kept), got)
