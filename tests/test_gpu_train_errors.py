"""A training run ends with an error where one of its calls has reported one on the device."""
import pytest
import torch

from combine_warp_top_gb300 import moe, train

pytestmark = pytest.mark.gpu
TIMEOUT = 5


@pytest.mark.parametrize("optimizer,call", [
    ("sgd", "moe_grouped_gemm"), ("muon", "moe_gated_gemm"), ("muon", "moe_muon_update"),
])
def test_an_error_word_ends_the_run(monkeypatch, optimizer, call):
    """The call's workspace, its last argument, is given the word that a wait which ran out
    leaves there."""
    launch = getattr(moe, call)

    def reporting(*args, **kw):
        launch(*args, **kw)
        args[-1].view(torch.int32)[0] = TIMEOUT

    train.main(steps=2, N=64, H=64, E=4, k=2, I=64, optimizer=optimizer)
    monkeypatch.setattr(moe, call, reporting)
    with pytest.raises(AssertionError):
        train.main(steps=2, N=64, H=64, E=4, k=2, I=64, optimizer=optimizer)


def test_a_run_of_no_steps():
    assert train.main(steps=0, N=64, H=64, E=4, k=2, I=64, optimizer="muon") == []
