"""An infinity that a query sees: its column is that infinity, every other column keeps its bits.

A softmax weight is positive, so sum_j w_j v_j with one infinite v_j is that infinity; it is NaN only
where infinities of both signs meet or the weight underflows fp32.
"""
import pytest
import torch

from _attn import cu, heads, paged
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def _decode(c, q, n, max_len=None):
    dev = {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in c.items()}
    return ssm.attn_decode_step(q.to(DEV), dev["k_cache"], dev["v_cache"], dev["table"],
                                torch.tensor([n], dtype=torch.int32, device=DEV), max_len or n, dev["k_scale"],
                                dev["v_scale"], out_dtype=torch.float32, lse=True)


# one key; a warp's units; the pieces joined in a cluster; joined by the second kernel
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n,D,H", [(1, 128, 4), (40, 64, 1), (700, 128, 8), (9001, 64, 12), (9001, 128, 3)])
def test_decode_bf16_seen_infinity(n, D, H, sign):
    g = torch.Generator().manual_seed(n + D)
    k, v = torch.randn(n, 1, D, generator=g), torch.randn(n, 1, D, generator=g)
    q = heads(g, 1, H, D)
    clean, cl = _decode(paged(k, v, [n], 16, False), q, n)
    for at in sorted({0, n // 2, n - 1}):
        v2 = v.clone()
        v2[at, 0, 5] = sign * INF
        out, lse = _decode(paged(k, v2, [n], 16, False), q, n)
        assert bool((out[:, :, 5] == sign * INF).all()), (at, out[0, :, 5])
        out[:, :, 5] = clean[:, :, 5]
        assert torch.equal(out, clean) and torch.equal(lse, cl)


def test_decode_bf16_infinity_under_a_tiny_weight_and_of_both_signs():
    """A weight of 2^-115 of the largest is still positive; +inf and -inf together are NaN."""
    n, D = 20, 64
    k, v = torch.zeros(n, 1, D), torch.ones(n, 1, D)
    k[7, 0, 0] = 80.0                                   # score 80 against 0: weights e^-80
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16)
    q[:, :, 0] = 8.0
    v[3, 0, 1], v[4, 0, 2] = INF, -INF
    v[5, 0, 9], v[6, 0, 9] = INF, -INF
    out, _ = _decode(paged(k, v, [n], 16, False), q, n)
    assert bool((out[:, :, 1] == INF).all()) and bool((out[:, :, 2] == -INF).all()) and bool(out[:, :, 9].isnan().all())
    rest = [d for d in range(D) if d not in (1, 2, 9)]
    assert bool((out[:, :, rest] == 1.0).all())


def test_decode_int8_row_with_an_infinity_reads_as_nan():
    """An int8 row that held an infinity has scale +inf and reads back as NaN: so does what sees it."""
    n, D = 40, 64
    g = torch.Generator().manual_seed(2)
    k, v = torch.randn(n, 1, D, generator=g), torch.randn(n, 1, D, generator=g)
    v[11, 0, 5] = INF
    c = paged(k, v, [n], 16, True)
    q = heads(g, 1, 2, D)
    seen, _ = _decode(c, q, n)
    assert bool(seen.isnan().all())
    before, _ = _decode(c, q, 11, max_len=n)
    assert bool(before.isfinite().all())


# 256 rows x heads or fewer (weights as bf16 pairs), whole and with the keys split; more of them
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("rows,keys,H,D", [
    (1, 1, 2, 64), (60, 700, 4, 128), (9, 5000, 8, 64), (3, 4400, 2, 80), (300, 900, 2, 128), (300, 5000, 3, 64),
])
def test_prefill_seen_infinity(rows, keys, H, D, sign):
    """The infinite value in a block that every row sees, in one that some rows see, and at the last key."""
    g = torch.Generator().manual_seed(rows + keys)
    q, k, v = heads(g, rows, H, D).to(DEV), heads(g, keys, 1, D).to(DEV), heads(g, keys, 1, D).to(DEV)
    cq, ck = cu([rows]).to(DEV), cu([keys]).to(DEV)
    clean, cl = ssm.attn_prefill(q, k, v, cq, ck, rows, lse=True, out_dtype=torch.float32)
    for at in sorted({0, keys // 2, keys - rows // 2 - 1, keys - 1}):
        v2 = v.clone()
        v2[at, 0, 5] = sign * INF
        out, lse = ssm.attn_prefill(q, k, v2, cq, ck, rows, lse=True, out_dtype=torch.float32)
        first = max(0, at - (keys - rows))                  # the first row that sees it
        assert bool((out[first:, :, 5] == sign * INF).all()), at
        out[first:, :, 5] = clean[first:, :, 5]
        assert torch.equal(out, clean) and torch.equal(lse, cl)
