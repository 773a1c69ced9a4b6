"""The training example learns: a policy that samples, scores, takes the losses' gradients and updates its head
with the library's calls alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_policy_update_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    from examples import policy_update

    first, last, margin = policy_update.train(steps=40, vocab=1024, rows=1024)
    # one token in eight is rewarded by chance
    assert first < 0.2 and last > 0.9
    assert margin > 0.1
    import top_sampling_apply_gb300 as tsa

    assert tsa.device_status() == 0
