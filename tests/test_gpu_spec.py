"""spec_probs against the softmax in 64 bits, spec_verify against the definition in exact fractions."""
import numpy as np
import pytest
import torch

from _steps import check_probs, probs64, verify_exact
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF, NAN = float("inf"), float("nan")


# ------------------------------------------------------------------ probabilities
@pytest.mark.parametrize("r,v", [(1, 1), (3, 2), (2, 7), (5, 31), (4, 33), (3, 1000), (2, 1001), (7, 4096), (2, 32003), (1, 50280), (3, 65537),
                                 (2, 131072), (1, 262145), (40, 515), (300, 130), (1, 600001)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_sizes(r, v, dtype):
    g = torch.Generator().manual_seed(r + v)
    x = (3 * torch.randn(r, v, generator=g)).to(dtype).to(DEV)
    t = (0.2 + 2 * torch.rand(r, generator=g)).to(DEV)
    t[0] = 0.0
    for temp in (None, t):
        check_probs(ssm.spec_probs(x, temp), x, temp)


@pytest.mark.parametrize("pad_in,pad_out,off", [(3, 0, 1), (0, 5, 0), (1, 2, 3), (8, 8, 0), (4, 4, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_strides_and_neighbours(pad_in, pad_out, off, dtype):
    g = torch.Generator().manual_seed(5)
    for v in (200, 4099, 20000):
        wide = torch.full((5, v + pad_in + off), 50.0, dtype=dtype)
        wide[:, off:off + v] = (2 * torch.randn(5, v, generator=g)).to(dtype)
        x = wide.to(DEV)[:, off:off + v]
        big = torch.full((5, v + pad_out + off), 9.0, device=DEV)
        o = ssm.spec_probs(x, out=big[:, off:off + v])
        check_probs(o, x, None)
        assert (big[:, :off] == 9).all() and (big[:, off + v:] == 9).all()


@pytest.mark.parametrize("v", [5, 300, 50021])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_masked_infinite_and_nan(v, dtype):
    g = torch.Generator().manual_seed(6)
    low = torch.finfo(dtype).min
    x = torch.randn(12, v, generator=g).to(dtype)
    x[0] = -INF                                   # nothing left
    x[1, 1:] = -INF                               # one left
    x[2] = low                                    # all at the type's lowest
    x[3, ::2] = low
    x[4, 2] = INF
    x[5, 3] = NAN
    x[6, :] = -INF
    x[6, v - 1] = low
    x[8] = torch.finfo(dtype).max
    x[9, 0] = torch.finfo(dtype).max
    t = torch.tensor([1, 0.5, 2, 0.7, 1, 1, 0.3, NAN, 1, 1, INF, -1.0])
    x, t = x.to(DEV), t.to(DEV)
    o = ssm.spec_probs(x, t)
    check_probs(o, x, t)
    assert (o[0] == 0).all() and o[1, 0] == 1 and torch.isnan(o[4]).all() and torch.isnan(o[7]).all()
    check_probs(ssm.spec_probs(x), x, None)


@pytest.mark.parametrize("v", [2, 33, 1000, 50021, 131072])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_greedy_takes_the_first_largest(v, dtype):
    g = torch.Generator().manual_seed(v)
    x = torch.randint(0, 3, (9, v), generator=g).to(dtype)          # ties everywhere
    x[0] = 0.0
    x[1, v - 1] = 5
    x[2, v // 2] = 5
    x[3] = -INF
    x = x.to(DEV)
    for t in (0.0, 2.0 ** -100, -3.0):
        o = ssm.spec_probs(x, torch.full((9,), t, device=DEV))
        assert np.array_equal(o.cpu().numpy(), probs64(x, np.full(9, t)))


def test_probs_no_rows():
    assert ssm.spec_probs(torch.empty(0, 9, device=DEV)).shape == (0, 9)


# ------------------------------------------------------------------ verification
def verify(draft, p, u, q=None, n=None, **kw):
    f = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    tokens, kept = ssm.spec_verify(f(draft), f(p), f(u), f(q), f(n), **kw)
    return tokens.cpu().numpy(), kept.cpu().numpy()


def same(draft, p, u, q=None, n=None):
    got, want = verify(draft, p, u, q, n), verify_exact(draft, p, u, q, n)
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0]), (got[0], want[0])


def case(batch, n, vocab, seed, near=0.5, q=True, ragged=False):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(batch, n + 1, vocab, generator=g, dtype=torch.float64)
    p = torch.softmax(x, -1).float()
    qs = torch.softmax(x[:, :n] + near * torch.randn(batch, n, vocab, generator=g, dtype=torch.float64), -1).float() if n else \
        torch.zeros(batch, 0, vocab)
    draft = torch.multinomial(qs.reshape(-1, vocab), 1, generator=g).view(batch, n).to(I32) if n else torch.zeros(batch, 0, dtype=I32)
    u = torch.rand(batch, n + 1, generator=g)
    count = torch.randint(0, n + 1, (batch,), generator=g, dtype=I32) if ragged else None
    return draft, p, u, (qs if q else None), count


@pytest.mark.parametrize("batch,n,vocab", [(1, 0, 1), (1, 1, 1), (2, 1, 2), (9, 3, 5), (33, 4, 31), (16, 7, 257), (5, 2, 1000), (3, 33, 100),
                                           (2, 70, 40), (1, 4, 5003), (40, 0, 300), (4, 3, 9001)])
@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("ragged", [False, True])
def test_verify_is_its_definition(batch, n, vocab, q, ragged):
    same(*case(batch, n, vocab, batch * 100 + n + vocab, q=q, ragged=ragged))


@pytest.mark.parametrize("vocab", [50021, 131072, 151937, 400003])
def test_verify_large_vocabularies(vocab):
    draft, p, u, q, n = case(2, 2, vocab, vocab, near=1.0)
    same(draft, p, u, q, n)


def test_borders_that_are_met_exactly():
    """u p equal to u q is refused; a running sum equal to the border is passed."""
    p = torch.tensor([[[0.25, 0.25, 0.5], [0.125, 0.5, 0.375]]])
    q = torch.tensor([[[0.5, 0.25, 0.25]]])
    draft = torch.tensor([[0]], dtype=I32)
    for u0 in (0.0, 0.25, 0.5, 0.5 - 2.0 ** -25, 0.75):
        for u1 in (0.0, 0.125, 0.125 + 2.0 ** -24, 0.625, 0.625 - 2.0 ** -24, 1 - 2.0 ** -24, 0.25, 0.5):
            same(draft, p, torch.tensor([[u0, u1]]), q)
            same(draft, p, torch.tensor([[u0, u1]]))


def test_equal_distributions_keep_everything_and_empty_residuals_fall_back():
    draft, p, u, _, _ = case(6, 3, 50, 1)
    same(draft, p, u, p[:, :3].contiguous())
    assert (verify(draft, p, u, p[:, :3].contiguous())[1] == 3).all()
    # refused with nothing left of p - q (q above p everywhere): drawn from p
    q = torch.clamp(p[:, :3] * 1.5 + 1e-3, max=1.0)
    u[:, :3] = 0.99
    same(draft, p, u, q)


def test_rows_without_mass_and_values_that_are_none():
    draft, p, u, q, _ = case(8, 2, 40, 2)
    p[0] = 0.0
    p[1, :, 3] = NAN
    p[2, :, 5] = -1.0
    p[3] = p[3] * 8                                  # no distribution: sums up to 8
    q[4, :, 7] = NAN
    q[5] = 0.0
    p[6] = 2.0 ** -140
    p[7, :, 0] = INF
    same(draft, p, u, q)
    tokens, kept = verify(draft, p, u, q)
    assert tokens[0, 0] == -1 and kept[0] == 0


def test_draft_probabilities_above_one_leave_nothing_there():
    draft, p, u, q, _ = case(6, 2, 300, 5, near=1.0)
    u[:, 0] = 0.97
    for b, v in enumerate((1.5, 2.0, 3.99, 4.0, 7.0, INF)):
        q[b, :, 1::2] = v
    same(draft, p, u, q)


def test_masses_of_every_size():
    """Probabilities from 1 down to below 2^-62, and residuals that are the last bits of what they come from."""
    g = torch.Generator().manual_seed(6)
    p = (2.0 ** -torch.randint(0, 80, (40, 2, 700), generator=g).double() * (1 + torch.rand(40, 2, 700, generator=g, dtype=torch.float64)))
    p = (p / p.sum(-1, keepdim=True) * (0.5 + torch.rand(40, 2, 1, generator=g, dtype=torch.float64))).float()
    up, down = torch.nextafter(p[:, :1], torch.tensor(INF)), torch.nextafter(p[:, :1], torch.tensor(0.0))
    q = torch.where(torch.rand(40, 1, 700, generator=g) < 0.5, up, down)
    draft = torch.randint(0, 700, (40, 1), generator=g).to(I32)
    q[torch.arange(40), 0, draft[:, 0].long()] *= 2                  # refused for u from a half on
    u = 0.6 + 0.4 * torch.rand(40, 2, generator=g)
    same(draft, p, u, q)
    same(draft, p, u)


@pytest.mark.parametrize("q", [True, False])
def test_uniform_numbers_out_of_range(q):
    draft, p, u, qs, _ = case(6, 2, 64, 3, q=q)
    u[0], u[1], u[2], u[3] = 0.0, 1.0, -2.0, NAN
    u[4] = INF
    u[5] = 2.0 ** -60
    same(draft, p, u, qs)


@pytest.mark.parametrize("q", [True, False])
def test_bad_tokens_and_counts_are_reported(q):
    draft, p, u, qs, _ = case(7, 3, 30, 4, q=q)
    n = torch.tensor([3, 3, 3, 9, -2, 3, 0], dtype=I32)
    draft[1, 0], draft[2, 1] = 30, -1
    assert ssm.device_status() == 0
    same(draft, p, u, qs, n)
    assert ssm.device_status() == ssm.DEV_BAD_INDEX and ssm.device_status() == 0
    # a bad token that is not looked at says nothing
    n[:] = 0
    draft[:] = 1 << 30
    same(draft, p, u, qs, n)
    assert ssm.device_status() == 0


def test_strided_probabilities():
    draft, p, u, q, _ = case(5, 3, 200, 5)
    wide = torch.full((5, 6, 211), 9.0)
    wide[:, 1:5, 3:203] = p
    qw = torch.full((3, 5, 203), 9.0)                # [place, batch, vocab]
    qw[:, :, 1:201] = q.transpose(0, 1)
    want = verify_exact(draft, p, u, q)
    tokens, kept = ssm.spec_verify(draft.to(DEV), wide.to(DEV)[:, 1:5, 3:203], u.to(DEV), qw.to(DEV)[:, :, 1:201].transpose(0, 1))
    assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])


def test_outputs_given():
    draft, p, u, q, _ = case(4, 2, 77, 6)
    tokens, kept = torch.full((6, 3), 99, dtype=I32, device=DEV), torch.full((6,), 99, dtype=I32, device=DEV)
    t, k = ssm.spec_verify(draft.to(DEV), p.to(DEV), u.to(DEV), q.to(DEV), tokens=tokens[1:5], n_kept=kept[1:5])
    want = verify_exact(draft, p, u, q)
    assert np.array_equal(tokens[1:5].cpu().numpy(), want[0]) and np.array_equal(kept[1:5].cpu().numpy(), want[1])
    assert (tokens[[0, 5]] == 99).all() and (kept[[0, 5]] == 99).all()


def test_no_requests():
    z = torch.zeros(0, 3, 8, device=DEV)
    t, k = ssm.spec_verify(torch.zeros(0, 2, dtype=I32, device=DEV), z, torch.zeros(0, 3, device=DEV))
    assert t.shape == (0, 3) and k.shape == (0,)


def test_tokens_have_the_targets_distribution():
    """Two tokens' share over 40000 requests with random numbers: within five standard deviations."""
    g = torch.Generator().manual_seed(8)
    n = 40000
    p, q = torch.tensor([0.5, 0.1, 0.3, 0.1]), torch.tensor([0.1, 0.4, 0.25, 0.25])
    draft = torch.multinomial(q.expand(n, 4), 1, generator=g).to(I32)
    tokens, _ = verify(draft, p.expand(n, 2, 4).contiguous(), torch.rand(n, 2, generator=g), q.expand(n, 1, 4).contiguous())
    share = np.bincount(tokens[:, 0], minlength=4) / n
    for i in range(4):
        e = float(p[i])
        assert abs(share[i] - e) <= 5 * (e * (1 - e) / n) ** 0.5


