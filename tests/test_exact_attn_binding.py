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


def run(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)


def test_the_plain_names_need_no_torch(kvm):
    """The ctypes names (the layer's, and the structs and functions of these operators) import
    without torch; the classes over them say what they miss."""
    r = run("import sys; sys.modules['torch'] = None\n"
            "from compressed_kv_state_gb300 import kvm\n"
            "assert kvm.lib.kvm_paged_append and kvm.kvm_rows and 'PagedCache' in dir(kvm)\n"
            "cfg = kvm.kvm_window_config(1, 2, 2, 64, 4, 0, 0, kvm.KVM_BF16)\n"
            "import ctypes; assert kvm.lib.kvm_window_scratch_bytes(ctypes.byref(cfg), 8, 0) > 0\n"
            "try: kvm.WindowAttention\n"
            "except ImportError: pass\n"
            "else: raise SystemExit('no ImportError')\n"
            "try: kvm.no_such_name\n"
            "except AttributeError: pass\n"
            "else: raise SystemExit('no AttributeError')\n")
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_torch_without_the_short_cuda_names(kvm):
    r = run("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from compressed_kv_state_gb300 import kvm\n"
            "kvm.WindowAttention(window=4), kvm.PagedCache, kvm.kvm_rope_table\n")
    assert r.returncode == 0, r.stdout + r.stderr
