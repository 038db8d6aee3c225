"""Calls of the exact-attention operators that are allowed and rare: results of a stream of
their own, values that are not finite among a row's keys."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rope_table_on_another_stream():
    """The table's memory is the given stream's: work that is still queued on the current stream
    over a block it has freed does not reach it."""
    from compressed_kv_state_gb300 import kvm
    n, s = 30000, torch.cuda.Stream()
    want = kvm.kvm_rope_table(32, 10000.0, n)
    torch.empty_like(want).fill_(7.0)  # (the kernel is loaded)
    torch.cuda.synchronize()
    x = torch.empty_like(want)
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    x.fill_(7.0)
    del x
    tables = [kvm.kvm_rope_table(32, 10000.0, n, stream=t) for t in (s, s.cuda_stream)]
    torch.cuda.synchronize()
    tables.append(kvm.kvm_rope_table(32, 10000.0, n, stream=0))
    torch.cuda.synchronize()
    for t in tables:
        assert torch.equal(t, want)
