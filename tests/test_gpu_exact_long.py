"""The exact-attention operators at sizes where a CTA takes several tiles, a warp several
rounds of its ring and the sinks' parts reach their limit, against the 64-bit definition
within the bounds of exact_attn_testlib.  Long sequences are compared by blocks of queries
with the keys that a block can see, grouped heads by whole groups."""
import pytest
import torch

from exact_attn_testlib import attend64, rope_table, turn, turn_bound, units, visible, within
from test_gpu_paged import filled, reference
from test_gpu_window import make, op

pytestmark = pytest.mark.gpu


def group64(q, k, v, dout, held, w, s, rope, dtype, step=512):
    """One key head's group: q, dout, held [G, N, 64], k, v [N, 64]; out, grads and their bounds."""
    G, N, _ = q.shape
    pos = torch.arange(N, device=q.device)
    u = units(dtype, rope is not None, N)
    z = lambda *n: torch.zeros(*n, 64, dtype=torch.float64, device=q.device)
    out, b_out, dq, b_dq = (z(G, N) for _ in range(4))
    dk, dv, b_dk, b_dv = (z(N) for _ in range(4))
    kk = turn(k.double(), rope, pos)
    for g in range(G):
        qq = turn(q[g].double(), rope, pos)
        for at in range(0, N, step):
            i = pos[at:at + step]
            lo = max(0, at - w + 1)
            j = torch.cat([pos[:min(s, lo)], pos[lo:at + step]])
            out[g, i], b_out[g, i], gr, bd = attend64(qq[i], kk[j], v[j].double(), visible(i, j, w, s), u, dout[g, i].double(),
                                                      held[g, i].double())
            dq[g, i], b_dq[g, i] = turn(gr[0], rope, i, -1.0), turn_bound(bd[0], rope, i)
            dk[j] += gr[1]
            dv[j] += gr[2]
            b_dk[j] += bd[1]
            b_dv[j] += bd[2]
    grads = [dq, turn(dk, rope, pos, -1.0), dv]
    bounds = [b_dq, turn_bound(b_dk, rope, pos), b_dv]
    for x, y in zip(grads, bounds):
        y += (u["u_out"] + u["u_acc"]) * x.abs() + 1e-30
    return out, b_out, grads, bounds


# dtype, B, H, Hkv, N, W, S, r, layout; (b, key head) pairs compared
WINDOW = [
    # 640, 960 and 768 tiles of 128 queries: several for both of a CTA's slots
    ("bf16", 2, 16, 8, 2500, 300, 16, 32, "tokens", [(0, 0), (0, 5), (1, 7)]),
    ("bf16", 4, 40, 8, 700, 64, 0, 64, "heads", [(0, 0), (3, 7), (2, 3)]),
    ("bf16", 2, 12, 12, 4000, 129, 128, 0, "heads", [(0, 0), (1, 11), (0, 6)]),
    # eight heads a thread of the rotation pass, the third eight of both kinds
    ("bf16", 20, 20, 5, 2600, 200, 4, 32, "heads", [(0, 0), (7, 4), (19, 2)]),
    ("bf16", 20, 20, 5, 2600, 70, 0, 64, "tokens", [(0, 1), (19, 4)]),
    # the causal mask
    ("bf16", 1, 24, 24, 5000, 5000, 0, 32, "tokens", [(0, 0), (0, 23)]),
    # parts of the sinks at their limit of 256
    ("bf16", 1, 2, 1, 50100, 1, 3, 32, "heads", [(0, 0)]),
    ("fp32", 1, 2, 1, 50100, 1, 70, 16, "heads", [(0, 0)]),
    ("fp32", 1, 8, 4, 3000, 400, 5, 32, "tokens", [(0, 0), (0, 3)]),
]


@pytest.mark.parametrize("case", WINDOW, ids=["-".join(map(str, c[:9])) for c in WINDOW])
def test_window_of_many_tiles(case):
    case, pairs = case[:9], case[9]
    q, k, v, dout, rope = make(case, 51)
    w = op(case, rope, torch.zeros(1, dtype=torch.int32, device="cuda"))
    out, lse = w.forward(q, k, v, need_lse=True)
    grads = w.backward(q, k, v, out, dout, lse)
    w.sync()
    assert all(torch.isfinite(x).all() for x in (out, *grads))
    G = case[2] // case[3]
    for b, g in pairs:
        hs = slice(g * G, (g + 1) * G)
        ref, bound, rg, bg = group64(q[b, hs], k[b, g], v[b, g], dout[b, hs], out[b, hs], case[5], case[6], rope, q.dtype)
        within(out[b, hs], ref, bound, f"out {b} {g}")
        for name, x, y, z in zip(("dq", "dk", "dv"), (grads[0][b, hs], grads[1][b, g], grads[2][b, g]), rg, bg):
            within(x, y, z, f"{name} {b} {g}")
    # the same bits again, forward and backward
    o2, l2 = w.forward(q, k, v, need_lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert all(torch.equal(x, y) for x, y in zip(grads, w.backward(q, k, v, out, dout, lse)))


# dtype, int4, B, H, Hkv, T, max_len, page, W, S, r: more than seven steps a computing warp (1,216 to
# 2,432 of them), so that every ring is filled and used again
ATTEND = [
    ("bf16", False, 6, 8, 8, 1, 20000, 32, 0, 0, 32),
    ("bf16", False, 6, 32, 8, 5, 20000, 64, 0, 0, 64),
    ("bf16", True, 8, 16, 8, 1, 40000, 64, 0, 0, 32),
    ("bf16", True, 8, 16, 8, 2, 40000, 8, 0, 0, 0),
    ("bf16", True, 8, 32, 8, 4, 30000, 16, 0, 0, 32),
    ("bf16", True, 6, 40, 8, 4, 24000, 32, 0, 0, 16),
    ("fp32", False, 6, 16, 8, 1, 20000, 16, 0, 0, 32),
    ("fp32", True, 6, 16, 8, 3, 20000, 32, 0, 0, 32),
    ("bf16", False, 40, 16, 16, 3, 3000, 16, 600, 20, 32),
    # 640 items and more: a warp a row in the join
    ("bf16", True, 80, 16, 8, 2, 2500, 16, 0, 0, 32),
    ("bf16", False, 40, 16, 16, 1, 2500, 32, 0, 0, 32),
    ("fp32", False, 40, 8, 8, 2, 1500, 16, 0, 0, 16),
]


@pytest.mark.parametrize("case", ATTEND, ids=["-".join(map(str, c)) for c in ATTEND])
def test_attention_of_long_caches(case):
    cache, held, q, lens, table, rope = filled(case, 52)
    out = cache.attend(q, lens, table, window=case[8], n_sinks=case[9])
    cache.sync()
    ref, bound = reference(case, held, q, lens, rope)
    rms = within(out, ref, bound, "out")
    if case[0] == "bf16":
        assert rms <= 2.0 ** -7
    assert torch.equal(cache.attend(q, lens, table, window=case[8], n_sinks=case[9]), out)
