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


def fastest(f):
    """The least of three calls' times on the device, in milliseconds (after one not counted)."""
    ms = []
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        ms.append(a.elapsed_time(b))
    return min(ms[1:])


@pytest.mark.parametrize("dt,int4", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True)])
def test_a_value_that_every_query_sees_costs_the_paged_attention_nothing(dt, int4):
    """A first value that is not finite makes every result so; the call takes its usual time (rows
    computed again key by key took 500 times that; 10 leaves room for the clock)."""
    from test_gpu_paged import filled
    cache, _, q, lens, table, _ = filled((dt, int4, 1, 2, 1, 2, 40000, 16, 0, 0, 32), 3)
    clean = fastest(lambda: cache.attend(q, lens, table))
    one = torch.ones(1, 1, 1, 64, dtype=q.dtype, device="cuda")
    cache.append(one, one * float("nan"), lens * 0, table)
    assert torch.isnan(cache.attend(q, lens, table)).all()
    assert fastest(lambda: cache.attend(q, lens, table)) <= 10 * clean


@pytest.mark.parametrize("case", [
    ("bf16", False, 3, 4, 4, 5, 700, 16, 0, 0, 32), ("bf16", False, 2, 8, 2, 7, 333, 8, 0, 0, 16),
    ("bf16", False, 2, 24, 1, 3, 900, 64, 100, 16, 0), ("bf16", False, 3, 4, 2, 16, 400, 32, 40, 3, 32),
    ("bf16", False, 2, 2, 2, 4, 20, 8, 2, 0, 0), ("fp32", False, 3, 4, 4, 5, 700, 16, 0, 0, 32),
    ("fp32", False, 2, 24, 1, 3, 900, 64, 100, 16, 0), ("fp32", False, 2, 2, 2, 4, 20, 8, 2, 0, 0)],
    ids=lambda c: "-".join(map(str, c)))
def test_dims_of_keys_that_some_queries_see(case):
    """Values of the newest tokens, and with a window of the first that any query sees, are not
    finite in some dims: those dims of the queries that see them are not either, every other
    result is as near its definition as without them."""
    from exact_attn_testlib import visible, within
    from test_gpu_paged import filled, reference
    dtype, int4, B, H, Hkv, T, max_len, page, W, S, r = case
    cache, held, q, lens, table, rope = filled(case, 71)
    ref, bound = reference(case, held, q, lens, rope)
    hit = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for b in range(B):
        n = int(lens[b])
        i = n - T + torch.arange(T, device="cuda")
        first = max(0, n - T - W + 1) if W else 0
        marks = [(n - 1, 5, float("inf")), (n - 2, 17, float("nan")), (n - 2, 40, -float("inf")), (n - T + 1, 63, float("nan")),
                 (first, 0, float("inf")), (first + 1, 33, float("nan"))]
        for j, d, x in marks:
            if not max(0, n - T - W + 1 if W else n - T + 1) <= j < n:
                continue
            cache.v[int(table[b, j // page]), :, j % page, d] = x
            hit[b, :, visible(i, torch.tensor([j], device="cuda"), W, S)[:, 0], d] = True
    out = cache.attend(q, lens, table, window=W, n_sinks=S)
    cache.sync()
    assert hit.any() and not torch.isfinite(out[hit]).any()
    zero = torch.zeros((), device="cuda")
    within(torch.where(hit, zero.to(out.dtype), out), torch.where(hit, zero.double(), ref), bound, "the others")


@pytest.mark.parametrize("dt,int4", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True)])
def test_queries_before_the_first_token_beside_values_that_are_not_finite(dt, int4):
    """A sequence shorter than its queries, all of its values NaN: the queries that see nothing
    get zeros, the others NaN."""
    from test_gpu_paged import filled
    for H in (2, 6, 10):  # rows of a key head: 8, 24, 40
        case = (dt, int4, 1, H, 1, 4, 2, 8, 0, 0, 32)
        cache, _, q, lens, table, _ = filled(case, 72)
        one = torch.ones(1, 1, 2, 64, dtype=q.dtype, device="cuda")
        cache.append(one, one * float("nan"), lens * 0, table)
        out = cache.attend(q, lens, table)
        cache.sync()
        assert torch.equal(out[:, :, :2], torch.zeros_like(out[:, :, :2])) and torch.isnan(out[:, :, 2:]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("where", [0, 130, 5000])
def test_a_value_that_later_queries_see_costs_the_window_nothing(dt, where):
    """Under the causal mask a value that is not finite makes every later result so; they are not
    computed again key by key (which took 300 times the usual time).  At 5000 the eight rows of the
    tile before it are, as they do not see it: 6 times; 20 leaves room for the clock."""
    from compressed_kv_state_gb300 import kvm
    g = torch.Generator().manual_seed(81)
    n = 16384 if dt == "bf16" else 6000
    q, k, v = (torch.randn(1, 2, n, 64, generator=g).to(torch.bfloat16 if dt == "bf16" else torch.float32).cuda() for _ in range(3))
    w = kvm.WindowAttention(window=n)
    clean = w.forward(q, k, v)
    usual = fastest(lambda: w.forward(q, k, v))
    for x in (float("nan"), float("inf")):
        v[:, :, where] = x
        out = w.forward(q, k, v)
        assert not torch.isfinite(out[:, :, where:]).any()
        assert torch.equal(out[:, :, :where // 128 * 128 - 128], clean[:, :, :where // 128 * 128 - 128]) or where < 256
        assert fastest(lambda: w.forward(q, k, v)) <= 20 * usual


# dtype, B, H, Hkv, N, W, S, r, layout
DIMS = [
    ("bf16", 1, 4, 2, 700, 100, 4, 32, "heads"), ("bf16", 2, 2, 2, 1000, 130, 20, 0, "tokens"),
    ("bf16", 1, 2, 1, 640, 640, 0, 64, "heads"), ("bf16", 1, 2, 1, 300, 7, 128, 16, "heads"),
    ("bf16", 1, 24, 8, 2000, 256, 3, 32, "tokens"), ("fp32", 1, 4, 2, 700, 100, 4, 32, "heads"),
    ("fp32", 1, 2, 1, 300, 7, 128, 16, "heads"),
]


@pytest.mark.parametrize("case", DIMS, ids=["-".join(map(str, c)) for c in DIMS])
def test_dims_of_values_that_some_queries_see(case):
    """Values that are not finite in some dims, a key of the sinks and the keys next to them among
    them: those dims of the queries that see them are not finite either, every other result is as
    near its definition as without them."""
    from exact_attn_testlib import visible, window64, within
    from test_gpu_window import make, op
    dt, B, H, Hkv, N, W, S, r, layout = case
    q, k, v, _, rope = make(case, 82)
    ref, bound = window64(q, k, v, W, S, rope, q.dtype)
    hit = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    i = torch.arange(N, device="cuda")
    inf, nan = float("inf"), float("nan")
    marks = [(S, 1, nan), (S + 1, 2, inf), (N // 3, 5, inf), (N // 3 + 1, 5, -inf), (N // 2, 17, nan), (N // 2 + 40, 63, -inf), (N - 1, 9, nan)]
    if S:
        marks.append((S - 1, 0, inf))
    for j, d, x in marks:
        v[:, :, j, d] = x
        hit[:, :, visible(i, torch.tensor([j], device="cuda"), W, S)[:, 0], d] = True
    w = op(case, rope, torch.zeros(1, dtype=torch.int32, device="cuda"))
    out = w.forward(q, k, v)
    w.sync()
    assert not torch.isfinite(out[hit]).any()
    zero = torch.zeros((), device="cuda")
    within(torch.where(hit, zero.to(out.dtype), out), torch.where(hit, zero.double(), ref), bound, "the others")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_scores_of_minus_infinity(dt):
    """Keys that are -infinity under queries of ones: a query that sees one key more than those is the
    mean of the rest, one that sees only those has no softmax (NaN by the definition)."""
    from compressed_kv_state_gb300 import kvm
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator().manual_seed(83)
    q = torch.ones(1, 1, 300, 64, dtype=dtype, device="cuda")
    k, v = q.clone(), torch.randn(1, 1, 300, 64, generator=g).to(dtype).cuda()
    k[:, :, :140] = -float("inf")
    out, lse = kvm.WindowAttention(window=300).forward(q, k, v, need_lse=True)
    assert torch.isnan(out[:, :, :140]).all()
    rest = v[0, 0, 140:].double()
    n = torch.arange(1, 161, device="cuda")[:, None]
    ref = rest.cumsum(0) / n
    # equal weights of 1: the sum's and the result's rounding
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    assert ((out[0, 0, 140:].double() - ref).abs() <= u * ref.abs() + 240 * 2.0 ** -23 * rest.abs().cumsum(0) / n).all()
    score = 8.0 * 1.4426950408889634  # 64 / 8 in log2 units
    assert ((lse[0, 0, 140:].double() - (score + n[:, 0].double().log2())).abs() <= 1e-4).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_a_value_under_a_weight_that_underflows(dt):
    """A score 2,500 below the others: the key's weight is not zero by the definition, so a value
    there that is not finite reaches every query that sees it, also in a tile with masked keys."""
    from compressed_kv_state_gb300 import kvm
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    q = torch.zeros(1, 1, 200, 64, dtype=dtype, device="cuda")
    k, v = torch.zeros_like(q), torch.ones_like(q)
    q[..., 0] = 100.0
    k[:, :, 0, 0], v[:, :, 0, 3] = -200.0, float("nan")
    for w in (kvm.WindowAttention(window=200), kvm.WindowAttention(window=50, n_sinks=1), kvm.WindowAttention(window=7)):
        out = w.forward(q, k, v)
        seen = min(200, w.window) if not w.n_sinks else 200
        assert torch.isnan(out[:, :, :seen, 3]).all()
        rest = torch.cat([out[:, :, :seen, :3].flatten(), out[:, :, seen:].flatten()])
        # weights of exactly 1, so the sums are whole numbers n; 1 / n is off by 2^-24 of itself at most,
        # n times that is rounded once more: 2^-24 + 2^-24, and their product 2^-48, off 1 (bf16: to 1)
        assert ((rest.double() - 1.0).abs() <= 2.0 ** -23 + 2.0 ** -48).all()
