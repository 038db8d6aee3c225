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


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_in_a_function_of_autograd(dt):
    """forward and backward as a torch.autograd.Function calls them: the gradients that reach the
    leaves are backward()'s; without the Function the call is refused."""
    from test_gpu_window import make, op
    case = (dt, 2, 4, 2, 130, 40, 3, 32, "tokens")
    q, k, v, dout, rope = make(case, 61)
    w = op(case, rope)

    class Attend(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            out, lse = w.forward(q, k, v, need_lse=True)
            ctx.save_for_backward(q, k, v, out, lse)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, out, lse = ctx.saved_tensors
            return w.backward(q, k, v, out, dout, lse)

    out, lse = w.forward(q, k, v, need_lse=True)
    want = w.backward(q, k, v, out, dout, lse)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    with pytest.raises(ValueError, match="requires gradients"):
        w.forward(*leaves)
    got = Attend.apply(*leaves)
    got.backward(dout)
    assert torch.equal(got, out)
    for leaf, x in zip(leaves, want):
        assert torch.equal(leaf.grad, x)


def test_sync_of_a_cache_without_a_status_word_is_refused():
    from compressed_kv_state_gb300 import kvm
    own = kvm.PagedCache.empty(2, 1, 8, dtype=torch.bfloat16)
    own.sync()
    with pytest.raises(ValueError, match="status"):
        kvm.PagedCache(own.k, own.v).sync()
