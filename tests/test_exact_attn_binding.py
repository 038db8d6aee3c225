"""The binding of the exact-attention operators where it needs no GPU."""
import pytest


@pytest.fixture(scope="module")
def kvm():
    from compressed_kv_state_gb300 import build
    build.build()
    from compressed_kv_state_gb300 import kvm as mod
    return mod


@pytest.mark.parametrize("which", range(3))
def test_tensors_that_require_gradients_are_refused(kvm, which):
    """autograd does not record the forward: gradients would end there without a word."""
    import torch
    x = [torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16) for _ in range(3)]
    x[which].requires_grad_()
    w = kvm.WindowAttention(window=4)
    with pytest.raises(ValueError, match="requires gradients"):
        w.forward(*x)
    with torch.no_grad(), pytest.raises(ValueError, match="current CUDA device"):  # (the next refusal: a host tensor)
        w.forward(*x)


def test_sync_without_a_status_word_is_refused(kvm):
    """It has nothing to report from, and would pass as if nothing had gone wrong."""
    with pytest.raises(ValueError, match="status"):
        kvm.WindowAttention(window=4).sync()
