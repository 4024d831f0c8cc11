"""MoETrainBlock's buffers, without a GPU."""
import pytest
import torch

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe, train


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load()


def tensors(value, name):
    if isinstance(value, torch.Tensor):
        yield name, value
    elif isinstance(value, dict):
        for n, v in value.items():
            yield from tensors(v, f"{name}.{n}")
    elif isinstance(value, moe.Layout):
        yield from tensors(value.tensors, name)


def test_every_buffer_is_on_the_blocks_device(lib):
    block = train.MoETrainBlock(6, 16, 4, 2, 8, device="cpu")
    found = [t for n, v in vars(block).items() for t in tensors(v, n)]
    assert {"ws", "ws_pre", "ws_post", "dense_ws", "out"} <= {n for n, _ in found}
    for name, t in found:
        assert t.device.type == "cpu", name
