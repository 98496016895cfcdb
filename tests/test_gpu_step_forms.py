"""Forms of the calls around the mixers that sizes choose and that need many rows or long ones: each against its definition in
64 bits, as in the tests of the small sizes."""
import numpy as np
import pytest
import torch

from _steps import NORM_REL, U, check_linear, check_norm, check_probs, half_step, norm64, probs64, to64, verify_exact
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, I32, U8 = torch.bfloat16, torch.float32, torch.int8, torch.int32, torch.uint8
INF, NAN = float("inf"), float("nan")


# ------------------------------------------------------------------ norm
# more than 304 groups (two for each SM): up to four vectors a thread, in blocks of 2, 4, 8, 16 and 32 warps
MANY = [(305, 1032, 1), (400, 2048, 1), (309, 2056, 1), (330, 4096, 1), (155, 8192, 2), (310, 4104, 1), (350, 7168, 1), (306, 8192, 1),
        (307, 8200, 1), (305, 16384, 1), (305, 16392, 1), (310, 32768, 1), (40, 16384, 8)]


@pytest.mark.parametrize("t,width,groups", MANY)
@pytest.mark.parametrize("x,res,out", [(BF16, None, BF16), (BF16, BF16, I8), (F32, None, F32), (BF16, F32, BF16), (F32, BF16, I8), (BF16, F32, I8),
                                       (F32, F32, I8), (F32, F32, F32)])
def test_norm_of_many_rows(t, width, groups, x, res, out):
    g = torch.Generator().manual_seed(t + width)
    xs = torch.randn(t, width, generator=g).to(x).to(DEV)
    rs = None if res is None else (3 * torch.randn(t, width, generator=g)).to(res).to(DEV)
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(DEV)
    o, r, s = ssm.norm_rms(xs, w, rs, n_groups=groups, out_dtype=out)
    check_norm(o, s, xs, w, rs, 1e-5, groups)
    if rs is not None:
        assert torch.equal(r, (xs.float() + rs.float()).to(res))
    again = ssm.norm_rms(xs, w, rs, n_groups=groups, out_dtype=out)
    assert all(a is None if b is None else torch.equal(a, b) for a, b in zip(again, (o, r, s)))


# A thread adds at most 32 squares (four vectors of eight), 5 steps join a warp's lanes and 5 its block's warps: 42
# additions, each U of the sum at most; r is off by U and its square, in the multiply-add, by no more: 45 U on the mean's
# sum, 2 for its division and eps, half of it on the root, the reciprocal root 4 U (two steps), three products.
TIGHT = (45 + 2) / 2 * U + 4 * U + 3 * U


@pytest.mark.parametrize("t,width", [(2, 8), (3, 264), (4, 4096), (330, 4096), (305, 8192), (2, 32768), (310, 32768), (1000, 1024)])
def test_norm_within_the_additions_that_a_thread_makes(t, width):
    assert TIGHT < NORM_REL / 2
    g = torch.Generator().manual_seed(width)
    x, res = (torch.randn(t, width, generator=g).to(DEV) for _ in range(2))
    for r in (None, res):
        o, _, _ = ssm.norm_rms(x, None, r, out_dtype=F32)
        # where r is a sum it is rounded once: relative to it, and so is y
        y, _ = norm64(x if r is None else x + r, None, None, float(np.float32(1e-5)), 1)
        got = to64(o).reshape(y.shape)
        assert (np.abs(got - y) <= np.abs(y) * TIGHT + 2.0 ** -126).all()
    assert half_step(F32) == U


# ------------------------------------------------------------------ probabilities
@pytest.mark.parametrize("r,v", [(700, 3001), (650, 5003), (400, 9001), (700, 17003), (320, 17003), (160, 33001), (80, 66001), (700, 9000), (40, 66001),
                                 (340, 40013)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_of_many_rows_of_medium_length(r, v, dtype):
    """Two to eight vectors a thread with one to four CTAs a row."""
    g = torch.Generator(device=DEV).manual_seed(r + v)
    x = (3 * torch.randn(r, v, generator=g, device=DEV)).to(dtype)
    t = (0.2 + 2 * torch.rand(r, generator=g, device=DEV))
    t[::7] = 0.0
    for temp in (None, t):
        got = ssm.spec_probs(x, temp)
        some = torch.cat([torch.arange(0, r, 13), torch.tensor([r - 1])]).to(DEV)
        check_probs(got[some], x[some], None if temp is None else temp[some])
        assert torch.isfinite(got).all()
        assert ((got.double().sum(-1) - 1).abs() < 1e-4).all()


@pytest.mark.parametrize("v", [262145, 300001, 600007])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_probs_of_rows_beyond_registers_masked_infinite_and_nan(v, dtype):
    g = torch.Generator().manual_seed(6)
    low = torch.finfo(dtype).min
    x = torch.randn(10, v, generator=g).to(dtype)
    x[0] = -INF
    x[1, 1:] = -INF
    x[2] = low
    x[3, ::2] = low
    x[4, v - 2] = INF
    x[5, v // 2] = NAN
    x[6, :] = -INF
    x[6, v - 1] = low
    x[8] = torch.finfo(dtype).max
    t = torch.tensor([1, 0.5, 2, 0.7, 1, 1, 0.3, NAN, 1, INF])
    x, t = x.to(DEV), t.to(DEV)
    o = ssm.spec_probs(x, t)
    check_probs(o, x, t)
    assert (o[0] == 0).all() and o[1, 0] == 1 and torch.isnan(o[4]).all() and torch.isnan(o[5]).all() and torch.isnan(o[7]).all()


@pytest.mark.parametrize("v", [200003, 262145, 300001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_greedy_takes_the_first_largest_of_long_rows(v, dtype):
    g = torch.Generator().manual_seed(v)
    x = torch.randint(0, 3, (6, v), generator=g).to(dtype)
    x[0] = 0.0
    x[1, v - 1] = 5
    x[2, v // 2], x[2, v // 2 + 1] = 5, 5
    x[3] = -INF
    x[4, v - 1], x[4, 3 * v // 4] = 7, 7
    x = x.to(DEV)
    for t in (0.0, -3.0):
        assert np.array_equal(ssm.spec_probs(x, torch.full((6,), t, device=DEV)).cpu().numpy(), probs64(x, np.full(6, t)))


# ------------------------------------------------------------------ verification
def same(draft, p, u, q=None, n=None, none=()):
    """As the definition says; the requests in `none` have no next token."""
    f = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    tokens, kept = ssm.spec_verify(f(draft), f(p), f(u), f(q), f(n))
    want = verify_exact(draft, p, u, q, n)
    for b in none:
        want[0][b, want[1][b]] = -1
    assert np.array_equal(kept.cpu().numpy(), want[1]), (kept, want[1])
    assert np.array_equal(tokens.cpu().numpy(), want[0]), (tokens, want[0])
    return want


def case(batch, n, vocab, seed, near=0.5):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(batch, n + 1, vocab, generator=g)
    p = torch.softmax(x, -1)
    q = torch.softmax(x[:, :n] + near * torch.randn(batch, n, vocab, generator=g), -1)
    draft = torch.stack([torch.multinomial(r, 1, generator=g) for r in q.reshape(-1, vocab)]).view(batch, n).to(I32)
    return draft, p, torch.rand(batch, n + 1, generator=g), q


LONG = [50021, 151937]                                # eight CTAs a request, several notes a warp


@pytest.mark.parametrize("vocab", LONG)
def test_empty_residuals_fall_back_across_a_cluster(vocab):
    """Refused with nothing left of p - q: the sums are taken again, of p, with words of their own."""
    draft, p, u, _ = case(3, 1, vocab, 1)
    u[:, 0] = 0.9999
    over = torch.clamp(p[:, :1] * 1.5 + 1e-6, max=1.0)
    u[:, 1] = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24])
    want = same(draft, p, u, over)
    assert (want[1] == 0).all()
    one = torch.zeros(3, 2, vocab)                    # a certain draft of a token with all of p, refused by its uniform number
    one[torch.arange(3), :, draft[:, 0].long()] = 0.5
    u[:, 0] = 0.75
    want = same(draft, one, u)
    assert (want[1] == 0).all() and (want[0][:, 0] == draft[:, 0].numpy()).all()


@pytest.mark.parametrize("vocab", LONG)
@pytest.mark.parametrize("with_q", [True, False])
def test_no_mass_and_values_that_are_none_across_a_cluster(vocab, with_q):
    draft, p, u, q = case(6, 1, vocab, 2)
    at = [3, vocab // 2, vocab - 1]
    p[0] = 0.0
    p[1][:, at] = NAN
    p[2][:, at] = -1.0
    p[3] = p[3] * 3.998                               # sums up to 3.99 and more over the row, in no CTA's part alone
    q[4][:, at] = NAN
    p[5][:, at[2]] = INF
    u[3, 0] = u[0, 0] = 0.999
    # the limit is 3.99 by the header; verify_exact knows the one of the integers, 4: 3.998 (1 +- 1e-3) is between them or above
    want = same(draft, p, u, q if with_q else None, none=[3])
    assert want[0][0, 0] == -1


@pytest.mark.parametrize("vocab", LONG)
def test_sums_at_the_limit_of_a_distribution_across_a_cluster(vocab):
    """Equal values whose sum is 3.9 or 4.1, whatever CTAs hold them: the first is drawn from, the second gives -1."""
    for total, none in ((3.9, False), (4.1, True)):
        p = torch.full((2, 1, vocab), total / vocab)
        u = torch.tensor([[0.3], [0.99]])
        tokens, kept = ssm.spec_verify(torch.zeros(2, 0, dtype=I32, device=DEV), p.to(DEV), u.to(DEV))
        assert (kept == 0).all() and bool((tokens == -1).all()) == none
        if not none:
            same(torch.zeros(2, 0, dtype=I32), p, u)


@pytest.mark.parametrize("vocab", LONG)
def test_masses_of_every_size_across_a_cluster(vocab):
    g = torch.Generator().manual_seed(6)
    p = (2.0 ** -torch.randint(0, 80, (4, 2, vocab), generator=g).double() * (1 + torch.rand(4, 2, vocab, generator=g, dtype=torch.float64)))
    p = (p / p.sum(-1, keepdim=True) * (0.5 + torch.rand(4, 2, 1, generator=g, dtype=torch.float64))).float()
    up, down = torch.nextafter(p[:, :1], torch.tensor(INF)), torch.nextafter(p[:, :1], torch.tensor(0.0))
    q = torch.where(torch.rand(4, 1, vocab, generator=g) < 0.5, up, down)
    draft = torch.randint(0, vocab, (4, 1), generator=g).to(I32)
    q[torch.arange(4), 0, draft[:, 0].long()] *= 2
    u = 0.6 + 0.4 * torch.rand(4, 2, generator=g)
    same(draft, p, u, q)
    same(draft, p, u)


@pytest.mark.parametrize("batch,vocab", [(310, 9001), (160, 17003), (330, 20011), (700, 5003)])
def test_many_requests_of_a_long_vocabulary(batch, vocab):
    """One or two CTAs a request: long stretches a warp, all its notes."""
    g = torch.Generator().manual_seed(batch)
    p = torch.softmax(2 * torch.randn(batch, 2, vocab, generator=g), -1)
    q = torch.softmax(2 * torch.randn(batch, 1, vocab, generator=g), -1)
    draft, u = torch.randint(0, vocab, (batch, 1), generator=g).to(I32), torch.rand(batch, 2, generator=g)
    f = lambda t: t.to(DEV)  # noqa: E731
    some = list(range(0, batch, 61)) + [batch - 1]
    for qs in (q, None):
        tokens, kept = ssm.spec_verify(f(draft), f(p), f(u), None if qs is None else f(qs))
        want = verify_exact(draft[some], p[some], u[some], None if qs is None else qs[some])
        assert np.array_equal(kept[some].cpu().numpy(), want[1]) and np.array_equal(tokens[some].cpu().numpy(), want[0])
        assert ((tokens[:, 0] >= 0) & (tokens[:, 0] < vocab)).all()


# ------------------------------------------------------------------ 4-bit weights
@pytest.mark.parametrize("m", [1, 6, 8, 9, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_no_output_of_a_row_with_an_infinity_or_nan_is_finite(m, group, zeros):
    """Few rows of x: every output of such a row, whatever the codes."""
    g = torch.Generator().manual_seed(m)
    n, k = 77, 384
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=U8).to(DEV)
    groups = k // group
    scales = torch.nn.functional.pad(0.02 * torch.randn(n, groups, generator=g), (0, -groups % 4)).to(DEV)[:, :groups]
    z = torch.nn.functional.pad(torch.randint(0, 16, (n, groups), generator=g, dtype=U8), (0, -groups % 16)).to(DEV)[:, :groups] if zeros else None
    x = torch.randn(m, k, generator=g).to(BF16).to(DEV)
    clean = ssm.w4_linear(x, codes, scales, z, out_dtype=F32)
    check_linear(clean, x, codes, scales, z, None)
    for value in (INF, -INF, NAN):
        for row in {0, m // 2, m - 1}:
            y = x.clone()
            y[row, (5 + 37 * row) % k] = value
            got = ssm.w4_linear(y, codes, scales, z, out_dtype=F32)
            assert not torch.isfinite(got[row]).any()
            rest = torch.arange(m, device=DEV) != row
            assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("m,k,n", [(128, 2048, 2048), (100, 2080, 2100), (20, 5120, 13824), (256, 1024, 3000)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_many_rows_whose_slices_go_by_the_group(m, k, n, group):
    """More slices for smaller groups, which take longer; the workspace is what the call's own plan asks for."""
    k = k // group * group
    g = torch.Generator(device=DEV).manual_seed(m)
    codes = torch.randint(0, 256, (n, -(-k // 32) * 16), generator=g, dtype=U8, device=DEV)[:, :k // 2]
    groups = k // group
    scales = torch.nn.functional.pad(0.02 * torch.randn(n, groups, generator=g, device=DEV), (0, -groups % 4))[:, :groups]
    zeros = torch.nn.functional.pad(torch.randint(0, 16, (n, groups), generator=g, dtype=U8, device=DEV), (0, -groups % 16))[:, :groups]
    x = torch.randn(m, k, generator=g, device=DEV).to(BF16)
    need = ssm.w4_linear_workspace_bytes(m, n, k, group)
    work = torch.full((need + 64,), 77, device=DEV, dtype=U8)
    got = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32, workspace=work[:need])
    check_linear(got, x, codes, scales, zeros, None)
    assert (work[need:] == 77).all()
    assert torch.equal(got, ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32))


def test_smaller_groups_have_at_least_as_many_slices():
    bytes_of = [ssm.w4_linear_workspace_bytes(128, 2048, 2048, group) for group in (128, 64, 32)]
    assert bytes_of == sorted(bytes_of) and bytes_of[1] > bytes_of[0]
