"""Exact attention beside the KVM layer (include/kvm.h): a sliding window with sink tokens, and
a paged key / value cache.  Reached as kvm.WindowAttention, kvm.PagedCache and
kvm.kvm_rope_table.  The calls can be as short as a kernel launch: what each of them does on
the host is kept to a few microseconds.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .kvm import (KVM_BF16, KVM_CACHE_INT4, KVM_CACHE_PLAIN, KVM_DEV_TIMEOUT, KVM_ERR_DEVICE, KVM_ERR_INVALID_ARG,
                  KVM_ERR_TIMEOUT, KVM_FP32, KVM_POINTERS_CHECKED, KvmError, _check, kvm_last_error, kvm_paged_cache,
                  kvm_window_config, lib)

# the current device and a device's current stream: by torch's short forms where it has them
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)

_ROWS = {n: ctypes.c_int64 * (4 * n) for n in (2, 4, 8)}


def _rows(*tensors):
    """(memory, address) of the kvm_rows, one behind another, of [B, H, N, 64] tensors whose
    rows are contiguous (any other strides the library accepts: include/kvm.h)."""
    r = []
    for t in tensors:
        sb, sh, sn, one = t.stride()
        if one != 1:
            raise ValueError(f"expected tensors [batch, heads, tokens, 64] with contiguous rows, got strides {t.stride()}")
        r += (t.data_ptr(), sb, sh, sn)
    mem = _ROWS[len(tensors)](*r)
    return mem, ctypes.addressof(mem)


def _same(name: str, t, shape, dtype, device):
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")


def _vec(t, name: str, shape, dtype, device):
    """Pointer of a contiguous tensor of the given shape and dtype (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _io_code(dtype) -> int:
    if dtype is torch.bfloat16:
        return KVM_BF16
    if dtype is torch.float32:
        return KVM_FP32
    raise ValueError(f"expected bfloat16 or float32, got {dtype}")


def _on_device(device, stream):
    """The caller's current device must be the tensors' (the library runs on it); the stream
    handle of `stream` or of the current stream."""
    if device.type != "cuda" or device.index != _device_now():
        raise ValueError(f"tensors must be on the current CUDA device, got {device}")
    return _raw_stream(device.index) if stream is None else getattr(stream, "cuda_stream", stream)


def _held(x) -> int:
    """x within 32 bits (ctypes would drop the bits above them)."""
    return max(-1, min(int(x), 2**31 - 1))


def _addr(t):
    return None if t is None else t.data_ptr()


def _word(status, device):
    """Pointer of an optional status word."""
    return None if status is None else _vec(status, "status", (1,), torch.int32, device)


def _make(stream, shape, dtype, device, like=None):
    """An uninitialised tensor (strided like `like` if given) from the memory of the stream the
    call runs on: memory of another stream's could still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device) if like is None else torch.empty_like(like)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return _make(None, shape, dtype, device, like)


def _report(status):
    """Wait for the device, then report (and clear) a status word as kvm_layer_sync does."""
    if status is None:
        raise ValueError("no status word to report from: pass status=torch.zeros(1, dtype=torch.int32, device='cuda')")
    torch.cuda.synchronize(status.device)
    bits = int(status.item())
    if bits:
        status.zero_()
        if bits & KVM_DEV_TIMEOUT:
            raise KvmError(KVM_ERR_TIMEOUT, "a bounded device-side wait expired")
        raise KvmError(KVM_ERR_DEVICE, "a length, position or page index was out of range")


def kvm_rope_table(rope_dims: int, rope_theta: float, n_pos: int, device="cuda", stream=None):
    """(cos, sin) table fp32 [n_pos, rope_dims / 2, 2], built on the device."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", _device_now())
    handle = _on_device(device, stream)
    out = _make(stream, (int(n_pos), int(rope_dims) // 2, 2), torch.float32, device)
    st = lib.kvm_rope_table(int(rope_dims), float(rope_theta), int(n_pos),
                            out.data_ptr() if out.numel() else None, handle)
    _check(st, None)
    return out


def _rope_args(rope, n_pos: int, device):
    """(rope_dims, pointer) of a rope table, or (0, None)."""
    if rope is None:
        return 0, None
    if rope.dim() != 3 or rope.shape[2] != 2 or rope.shape[0] < n_pos or rope.dtype != torch.float32 \
            or not rope.is_contiguous() or rope.device != device:
        raise ValueError(f"rope: expected a contiguous float32 table [>= {n_pos}, rope_dims / 2, 2] on {device}, got "
                         f"{rope.dtype} {tuple(rope.shape)} on {rope.device}")
    return 2 * rope.shape[1], rope.data_ptr()


@functools.lru_cache(maxsize=256)
def _window_plan(batch, heads, kv_heads, head_dim, n, window, n_sinks, rope_dims, dtype):
    """(config, its address, scratch bytes of the forward and the backward) of these sizes."""
    cfg = kvm_window_config(batch, heads, kv_heads, head_dim, window, n_sinks, rope_dims,
                            _io_code(dtype) | KVM_POINTERS_CHECKED)  # (every tensor's device is looked at below)
    at = ctypes.addressof(cfg)
    nbytes = [lib.kvm_window_scratch_bytes(at, n, back) for back in (0, 1)]
    if 0 in nbytes:
        raise KvmError(KVM_ERR_INVALID_ARG, kvm_last_error(None))
    return cfg, at, nbytes[0], nbytes[1]


class WindowAttention:
    """Sliding-window attention with sink tokens (kvm_window_forward / kvm_window_backward).

    window: keys a query sees, itself included; n_sinks: first tokens that stay visible;
    rope: a kvm_rope_table (None: q and k are not rotated); status: an int32 CUDA word that
    the kernels report to, for sync() (None: nothing is reported)."""

    def __init__(self, *, window: int, n_sinks: int = 0, rope=None, status=None):
        self.window, self.n_sinks, self.rope, self.status = _held(window), _held(n_sinks), rope, status

    def _plan(self, q, k):
        if q.dim() != 4 or k.dim() != 4 or q.shape[3] != 64:
            raise ValueError(f"q and k are [batch, heads, tokens, 64], got {tuple(q.shape)} and {tuple(k.shape)}")
        b, h, n, d = q.shape
        r, ptr = _rope_args(self.rope, n, q.device)
        kv = k.shape[1]
        return ptr, (b, kv, n, 64), _window_plan(b, h, kv, d, n, self.window, self.n_sinks, r, q.dtype)

    def forward(self, q, k, v, out=None, need_lse: bool = False, stream=None):
        """out [B, H, N, 64] (strided like q when not given) of q [B, H, N, 64] and k, v
        [B, Hkv, N, 64]; with need_lse (out, lse), lse fp32 [B, H, N] for backward().
        autograd does not record the call: tensors that require gradients are refused unless
        gradients are off (torch.no_grad(), or the forward of a torch.autograd.Function whose
        backward calls backward())."""
        if (q.requires_grad or k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            raise ValueError("q, k or v requires gradients, and autograd does not record this call: make it under "
                             "torch.no_grad() (or in a torch.autograd.Function) and take the gradients from backward()")
        dev, dt = q.device, q.dtype
        handle = _on_device(dev, stream)
        rope, kvs, (cfg, at, nbytes, _) = self._plan(q, k)
        _same("k", k, kvs, dt, dev)
        _same("v", v, kvs, dt, dev)
        if out is None:
            out = _make(stream, None, None, None, q)
        else:
            _same("out", out, q.shape, dt, dev)
        rows, r = _rows(q, k, v, out)
        lse = _make(stream, q.shape[:3], torch.float32, dev) if need_lse else None
        scratch = _make(stream, nbytes, torch.uint8, dev)
        st = lib.kvm_window_forward(at, r, r + 32, r + 64, q.shape[2], rope, r + 96, _addr(lse), scratch.data_ptr(),
                                    nbytes, _word(self.status, dev), handle)
        if st:
            _check(st, None)
        return (out, lse) if need_lse else out

    def backward(self, q, k, v, out, dout, lse, dq=None, dk=None, dv=None, stream=None):
        """(dq, dk, dv) of the forward that gave out and lse; strided like q, k, v when not given."""
        dev, dt = q.device, q.dtype
        handle = _on_device(dev, stream)
        rope, kvs, (cfg, at, _, nbytes) = self._plan(q, k)
        dq = _make(stream, None, None, None, q) if dq is None else dq
        dk = _make(stream, None, None, None, k) if dk is None else dk
        dv = _make(stream, None, None, None, v) if dv is None else dv
        for name, t, s in (("k", k, kvs), ("v", v, kvs), ("out", out, q.shape), ("dout", dout, q.shape),
                           ("dq", dq, q.shape), ("dk", dk, kvs), ("dv", dv, kvs)):
            _same(name, t, s, dt, dev)
        rows, r = _rows(q, k, v, out, dout, dq, dk, dv)
        scratch = _make(stream, nbytes, torch.uint8, dev)
        st = lib.kvm_window_backward(at, r, r + 32, r + 64, r + 96, r + 128, q.shape[2], rope,
                                     _vec(lse, "lse", q.shape[:3], torch.float32, dev), r + 160, r + 192, r + 224,
                                     scratch.data_ptr(), nbytes, _word(self.status, dev), handle)
        if st:
            _check(st, None)
        return dq, dk, dv

    def sync(self):
        """Wait for the device and raise if a kernel reported through the status word (which must
        have been given: without one the kernels' reports are lost)."""
        _report(self.status)


class PagedCache:
    """A paged key / value cache over caller-owned page tensors (kvm_paged_cache).

    k, v: [n_pages, kv_heads, page_size, 64] bf16 or fp32, or uint8 [.., 32] with k_sm, v_sm
    bf16 [n_pages, kv_heads, page_size, 2] (the 4-bit format; dtype is then that of q, k, v
    and out); rope: a kvm_rope_table, or None; status: an int32 CUDA word that the kernels
    report to, for sync() (None: nothing is reported)."""

    def __init__(self, k, v, k_sm=None, v_sm=None, *, dtype=None, rope=None, status=None):
        dev = k.device
        if k.dim() != 4 or dev.type != "cuda":
            raise ValueError("pages are CUDA tensors [n_pages, kv_heads, page_size, 64] (32 bytes a row in 4 bits)")
        int4 = k.dtype is torch.uint8
        dtype = dtype or (torch.bfloat16 if int4 else k.dtype)
        n_pages, heads, page = k.shape[:3]
        shape, want = (n_pages, heads, page, 32 if int4 else 64), torch.uint8 if int4 else dtype
        pk, pv, psk, psv = _vec(k, "k", shape, want, dev), _vec(v, "v", shape, want, dev), None, None
        if int4:
            if k_sm is None or v_sm is None:
                raise ValueError("a 4-bit cache needs k_sm and v_sm")
            shape = (n_pages, heads, page, 2)
            psk, psv = _vec(k_sm, "k_sm", shape, torch.bfloat16, dev), _vec(v_sm, "v_sm", shape, torch.bfloat16, dev)
        r, rp = _rope_args(rope, 1, dev)
        self.device, self.dtype, self.kv_heads, self.page_size = dev, dtype, heads, page
        self.k, self.v, self.k_sm, self.v_sm, self.rope, self.status = k, v, k_sm, v_sm, rope, status
        self.c = kvm_paged_cache(n_pages, page, heads, 64, KVM_CACHE_INT4 if int4 else KVM_CACHE_PLAIN,
                                 _io_code(dtype) | KVM_POINTERS_CHECKED, r,
                                 _held(rope.shape[0]) if r else 0, pk, pv, psk, psv, rp)
        self.at = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, page_size: int, *, dtype, int4: bool = False, rope=None, device="cuda"):
        """A cache of its own pages (zeroed) and status word."""
        shape = (n_pages, kv_heads, page_size)
        if int4:
            pages = [torch.zeros(*shape, 32, dtype=torch.uint8, device=device) for _ in range(2)]
            sm = [torch.zeros(*shape, 2, dtype=torch.bfloat16, device=device) for _ in range(2)]
        else:
            pages, sm = [torch.zeros(*shape, 64, dtype=dtype, device=device) for _ in range(2)], (None, None)
        return cls(*pages, *sm, dtype=dtype, rope=rope, status=torch.zeros(1, dtype=torch.int32, device=device))

    def _table(self, page_table, batch: int):
        if page_table.dim() != 2:
            raise ValueError("page_table is int32 [batch, max_pages]")
        per = page_table.shape[1]
        return _vec(page_table, "page_table", (batch, per), torch.int32, self.device), per

    def append(self, k, v, start, page_table, new_lens=None, stream=None):
        """Tokens i < new_lens[b] (all when None) of k, v [batch, kv_heads, n, 64] to positions
        start[b] + i (int32 [batch]) through page_table (int32 [batch, max_pages])."""
        dev = self.device
        handle = _on_device(dev, stream)
        if k.dim() != 4:
            raise ValueError("k and v are [batch, kv_heads, tokens, 64]")
        b, _, n, _ = k.shape
        shape, one = (b, self.kv_heads, n, 64), (b,)
        _same("k", k, shape, self.dtype, dev)
        _same("v", v, shape, self.dtype, dev)
        rows, r = _rows(k, v)
        tab, per = self._table(page_table, b)
        st = lib.kvm_paged_append(self.at, r, r + 32, b, n, _vec(new_lens, "new_lens", one, torch.int32, dev),
                                  _vec(start, "start", one, torch.int32, dev), tab, per, _word(self.status, dev), handle)
        if st:
            _check(st, None)

    def read(self, start, n: int, page_table, lens=None, k=None, v=None, stream=None):
        """(k, v) [batch, kv_heads, n, 64]: the cached rows of positions start[b] + i, zeros at
        and after lens[b]."""
        dev = self.device
        handle = _on_device(dev, stream)
        b = start.shape[0]
        shape, one = (b, self.kv_heads, int(n), 64), (b,)
        k = _make(stream, shape, self.dtype, dev) if k is None else k
        v = _make(stream, shape, self.dtype, dev) if v is None else v
        _same("k", k, shape, self.dtype, dev)
        _same("v", v, shape, self.dtype, dev)
        rows, r = _rows(k, v)
        tab, per = self._table(page_table, b)
        st = lib.kvm_paged_read(self.at, r, r + 32, b, int(n), _vec(lens, "lens", one, torch.int32, dev),
                                _vec(start, "start", one, torch.int32, dev), tab, per, _word(self.status, dev), handle)
        if st:
            _check(st, None)
        return k, v

    def attend(self, q, lens, page_table, *, window: int = 0, n_sinks: int = 0, out=None, stream=None):
        """Attention of q [batch, heads, n_q, 64], the last n_q of each sequence's lens[b] cached
        tokens, over the cache (all of it, or a window and the first n_sinks tokens)."""
        dev = self.device
        handle = _on_device(dev, stream)
        if q.dim() != 4:
            raise ValueError("q is [batch, heads, tokens, 64]")
        b, h, t, _ = q.shape
        shape = (b, h, t, 64)
        _same("q", q, shape, self.dtype, dev)
        if out is None:
            out = _make(stream, None, None, None, q)
        else:
            _same("out", out, shape, self.dtype, dev)
        rows, r = _rows(q, out)
        tab, per = self._table(page_table, b)
        nbytes = lib.kvm_paged_attention_scratch_bytes(self.at, b, h, t, per)
        if nbytes == 0:
            raise KvmError(KVM_ERR_INVALID_ARG, kvm_last_error(None))
        scratch = _make(stream, nbytes, torch.uint8, dev)
        st = lib.kvm_paged_attention(self.at, r, r + 32, b, h, t, _vec(lens, "lens", (b,), torch.int32, dev), tab, per,
                                     _held(window), _held(n_sinks), scratch.data_ptr(), nbytes, _word(self.status, dev), handle)
        if st:
            _check(st, None)
        return out

    def sync(self):
        """Wait for the device and raise if a kernel reported through the status word (which must
        have been given: without one the kernels' reports are lost)."""
        _report(self.status)
