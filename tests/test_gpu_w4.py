"""4-bit weights: w4_quantize against its definition bit by bit, w4_linear against the product in 64 bits over
types, groups, odd sizes, strides and numbers of rows."""
import numpy as np
import pytest
import torch

from _steps import check_linear, quantise32, unpack
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


def weight(g, n, k, group, scale_dtype=BF16, zeros=False, pad=0):
    """A random 4-bit weight with every code and zero in it; rows padded to 16 bytes and by `pad` more."""
    groups = k // group
    codes = torch.randint(0, 256, (n, k // 2 + 16 * pad), generator=g, dtype=U8).to(DEV)[:, :k // 2]
    s = torch.full((n, -(-groups // 8) * 8 + 8 * pad), float("nan"))
    s[:, :groups] = 0.02 * torch.randn(n, groups, generator=g)
    z = torch.randint(0, 16, (n, -(-groups // 16) * 16 + 16 * pad), generator=g, dtype=U8).to(DEV)[:, :groups] if zeros else None
    return codes, s.to(scale_dtype).to(DEV)[:, :groups], z


def activations(g, m, k, dtype, blocks=1):
    if dtype == BF16:
        return torch.randn(m, k, generator=g).to(BF16).to(DEV), None
    x = torch.randint(-127, 128, (m, k), generator=g, dtype=I8).to(DEV)
    return x, (0.01 + torch.rand(m, blocks, generator=g)).to(DEV)


def run(m, n, k, group, x=BF16, blocks=1, scales=BF16, zeros=False, out=F32, seed=0, pad=0, **kw):
    g = torch.Generator().manual_seed(seed + m * 7 + n * 3 + k)
    xs, s = activations(g, m, k, x, blocks)
    w = weight(g, n, k, group, scales, zeros, pad)
    o = ssm.w4_linear(xs, *w, x_scale=s, out_dtype=out, **kw)
    check_linear(o, xs, *w, s)
    assert ssm.device_status() == 0
    return o


# one row to many; N around tiles of 8, 16 and 128; K from one group on, odd numbers of groups
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 16, 128), (2, 17, 256), (3, 33, 384), (7, 128, 640), (8, 129, 1152), (9, 250, 1024),
                                   (15, 100, 2048), (16, 48, 896), (17, 65, 1408), (24, 31, 512), (31, 144, 768), (32, 160, 2176),
                                   (33, 70, 1280), (47, 23, 640), (64, 320, 1536), (65, 40, 256), (130, 18, 384), (1, 4099, 512),
                                   (4, 2500, 4096), (1, 40, 16384), (8, 24, 8192), (12, 80, 8320)])
@pytest.mark.parametrize("group,x,zeros", [(128, BF16, False), (64, I8, True), (32, BF16, True), (128, I8, False)])
def test_sizes(m, n, k, group, x, zeros):
    run(m, n, k, group, x, 1, BF16 if zeros else F32, zeros, F32)


@pytest.mark.parametrize("k,group", [(32, 32), (96, 32), (64, 64), (192, 64), (160, 32), (4128, 32), (8160, 32), (7104, 64)])
@pytest.mark.parametrize("m", [1, 5, 20])
def test_short_and_odd_rows(m, k, group):
    run(m, 50, k, group, BF16, 1, BF16, True, BF16)
    run(m, 50, k, group, I8, 1, F32, False, F32)


@pytest.mark.parametrize("m,n,k", [(1, 48, 32768), (3, 33, 32768), (9, 20, 32768), (20, 40, 20480), (40, 17, 32512), (64, 50, 32768)])
def test_long_rows(m, n, k):
    run(m, n, k, 128, BF16, 1, F32, True, F32)


@pytest.mark.parametrize("blocks,k,group", [(1, 1024, 128), (2, 1024, 128), (8, 1024, 128), (4, 1536, 32), (64, 8192, 128), (3, 4608, 64)])
@pytest.mark.parametrize("m", [1, 8, 19, 64])
def test_blocks_of_activation_scales(m, blocks, k, group):
    run(m, 70, k, group, I8, blocks, BF16, False, F32)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("scales", [BF16, F32])
@pytest.mark.parametrize("m", [1, 13, 40])
def test_types_of_scales_and_outputs(m, scales, out):
    run(m, 77, 768, 64, I8, 2, scales, True, out)
    run(m, 77, 768, 64, BF16, 1, scales, False, out)


# many rows of x and a weight large enough for its tiles: sixteen rows and more times 2^24 products, or nine and a
# weight of three times that; rows at the borders of 16, 32 and 64, K from one group on and to the longest
@pytest.mark.parametrize("m,n,k,group", [(256, 33001, 32, 32), (250, 11001, 96, 32), (256, 6601, 160, 32), (241, 5501, 192, 64),
                                         (255, 16500, 64, 64), (200, 2703, 480, 32), (129, 1901, 992, 32), (65, 3301, 1024, 64),
                                         (64, 4099, 1152, 128), (33, 2803, 2048, 128), (32, 8300, 1024, 64), (17, 16700, 512, 128),
                                         (64, 257, 16512, 128), (33, 201, 28160, 64), (64, 130, 32768, 32), (24, 300, 28160, 128),
                                         (9, 12400, 4096, 128), (16, 1601, 32768, 64), (12, 50001, 1024, 32)])
@pytest.mark.parametrize("x,zeros", [(BF16, False), (I8, True)])
def test_tiles(m, n, k, group, x, zeros):
    run(m, n, k, group, x, 1, BF16 if zeros else F32, zeros, F32)


@pytest.mark.parametrize("blocks,k,group", [(2, 1024, 128), (32, 1024, 32), (3, 1152, 128), (8, 2560, 64)])
@pytest.mark.parametrize("m,scales,out", [(68, BF16, F32), (256, F32, BF16)])
def test_tiles_with_blocks_of_activation_scales(m, scales, out, blocks, k, group):
    run(m, 3701, k, group, I8, blocks, scales, True, out, pad=1)


def test_tiles_keep_to_their_rows_and_outputs():
    """Infinities, NaN and bad scales stay where they are; strided x; outputs inside a wider tensor; workspaces of
    exactly the asked size; the border between the two ways of a call agrees."""
    g = torch.Generator().manual_seed(17)
    m, n, k = 70, 901, 4096
    x = torch.randn(2 * m, k + 64, generator=g).to(BF16).to(DEV)[::2, 64:]
    codes, scales, zeros = weight(g, n, k, 64, F32, True, pad=1)
    clean = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32)
    check_linear(clean, x, codes, scales, zeros, None)
    need = ssm.w4_linear_workspace_bytes(m, n, k, 64)
    assert need > 128 * k * 2                          # x in its order, and the sums of slices
    for out in (BF16, F32):
        big = torch.full((m + 2, n + 20), 9.0, device=DEV, dtype=out)
        work = torch.full((need + 256,), 77, device=DEV, dtype=U8)
        got = ssm.w4_linear(x, codes, scales, zeros, out=big[1:-1, 7:7 + n], workspace=work[:need])
        assert torch.equal(got, clean.to(out)) and (work[need:] == 77).all()
        assert (big[:, :7] == 9).all() and (big[:, 7 + n:] == 9).all() and (big[0] == 9).all() and (big[-1] == 9).all()
    x[1, 5], x[4, 200], x[66, 1023] = float("inf"), float("nan"), float("-inf")
    scales[17, 3] = float("nan")
    got = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32)
    rows, cols = torch.ones(m, dtype=torch.bool, device=DEV), torch.ones(n, dtype=torch.bool, device=DEV)
    rows[[1, 4, 66]] = False
    cols[17] = False
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert not torch.isfinite(got[~rows]).any() and torch.isnan(got[:, 17]).all()


def test_slices_of_few_rows_with_a_given_workspace():
    g = torch.Generator().manual_seed(19)
    for m, n, k in ((1, 700, 16384), (8, 1000, 8192), (16, 700, 16384), (20, 300, 16384)):
        x = torch.randn(m, k, generator=g).to(BF16).to(DEV)
        codes, scales, _ = weight(g, n, k, 128, BF16)
        need = ssm.w4_linear_workspace_bytes(m, n, k, 128)
        assert need >= 2 * m * n * 4 and need % (m * n * 4) == 0
        work = torch.full((need + 64,), 77, device=DEV, dtype=U8)
        got = ssm.w4_linear(x, codes, scales, out_dtype=F32, workspace=work[:need])
        check_linear(got, x, codes, scales, None, None)
        assert (work[need:] == 77).all()


def test_strides_and_neighbours():
    """Slices of wider tensors; outputs in place, at odd offsets, and nothing around them touched."""
    g = torch.Generator().manual_seed(11)
    m, n, k = 5, 45, 512
    x = torch.randn(m, 3 * k, generator=g).to(BF16).to(DEV)[:, k:2 * k]
    codes, scales, zeros = weight(g, 3 * n, k, 64, F32, True, pad=2)
    w = (codes[n:2 * n], scales[n:2 * n], zeros[n:2 * n])
    for out in (BF16, F32):
        big = torch.full((m, n + 20), 9.0, device=DEV, dtype=out)
        o = ssm.w4_linear(x, *w, out=big[:, 7:7 + n])
        check_linear(o, x, *w, None)
        assert (big[:, :7] == 9).all() and (big[:, 7 + n:] == 9).all()
    # the rows' inner part: a slice of K at a group's and 16 bytes' border, as a tensor-parallel rank holds it
    part = (codes[:, 128:192], scales[:, 4:6].clone(), zeros[:, 4:6].clone())
    part = (part[0], torch.nn.functional.pad(part[1], (0, 2))[:, :2], torch.nn.functional.pad(part[2], (0, 14))[:, :2])
    xs = torch.randn(m, 128, generator=g).to(BF16).to(DEV)
    check_linear(ssm.w4_linear(xs, *part, out_dtype=F32), xs, *part, None)


def test_no_rows_and_every_second_row():
    g = torch.Generator().manual_seed(12)
    w = weight(g, 24, 256, 128)
    assert ssm.w4_linear(torch.empty(0, 256, device=DEV, dtype=BF16), *w).shape == (0, 24)
    x = torch.randn(12, 256, generator=g).to(BF16).to(DEV)
    assert torch.equal(ssm.w4_linear(x[::2], *w), ssm.w4_linear(x[::2].contiguous(), *w))


def test_infinities_and_nan_stay_in_their_rows():
    g = torch.Generator().manual_seed(13)
    w = weight(g, 40, 384, 128, F32)
    x = torch.randn(6, 384, generator=g).to(BF16).to(DEV)
    clean = ssm.w4_linear(x, *w, out_dtype=F32)
    x[1, 5] = float("inf")
    x[4, 200] = float("nan")
    got = ssm.w4_linear(x, *w, out_dtype=F32)
    for r in range(6):
        if r in (1, 4):
            assert not torch.isfinite(got[r]).all()
        else:
            assert torch.equal(got[r], clean[r])
    assert torch.isnan(got[4]).all()


def test_a_bad_scale_reaches_its_own_output_only():
    g = torch.Generator().manual_seed(14)
    codes, scales, zeros = weight(g, 50, 512, 64, F32, True)
    x = torch.randn(3, 512, generator=g).to(BF16).to(DEV)
    clean = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32)
    scales[17, 3] = float("nan")
    got = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32)
    assert torch.isnan(got[:, 17]).all()
    keep = torch.arange(50, device=DEV) != 17
    assert torch.equal(got[:, keep], clean[:, keep])


@pytest.mark.parametrize("m,n,k", [(1, 60, 1024), (8, 33, 640), (16, 70, 2048), (40, 24, 1024), (70, 901, 4096)])
@pytest.mark.parametrize("group", [32, 128])
def test_weights_that_are_mostly_zero(m, n, k, group):
    """One element of a group and the rest at its zero: the result is that element's, the errors those of the sums of
    x (16 + code) and x (16 + zero): at most 128 steps of 2 U and 4 U on sum 31 |x| scale, for each of the two."""
    g = torch.Generator().manual_seed(m + n)
    groups = k // group
    z = torch.randint(0, 16, (n, groups), generator=g, dtype=U8)
    c = z.repeat_interleave(group, 1)
    at = torch.arange(groups) * group + torch.randint(0, group, (n, groups), generator=g)
    c.scatter_(1, at, torch.randint(0, 16, (n, groups), generator=g, dtype=U8))
    codes = (c[:, ::2] | c[:, 1::2] << 4).to(DEV)
    zeros = torch.nn.functional.pad(z, (0, -groups % 16)).to(DEV)[:, :groups]
    scales = torch.nn.functional.pad(0.02 * torch.randn(n, groups, generator=g), (0, -groups % 4)).to(DEV)[:, :groups]
    x = torch.randn(m, k, generator=g).to(BF16).to(DEV)
    got = ssm.w4_linear(x, codes, scales, zeros, out_dtype=F32)
    w = ((c.double() - z.double().repeat_interleave(group, 1)) * scales.cpu().double().repeat_interleave(group, 1))
    ref = x.cpu().double() @ w.T
    mag = x.cpu().double().abs() @ (31 * scales.cpu().double().abs()).repeat_interleave(group, 1).T
    assert ((got.cpu().double() - ref).abs() <= 2 * 260 * 2.0 ** -24 * mag).all()


def test_zeros_count_by_their_low_half():
    g = torch.Generator().manual_seed(15)
    codes, scales, zeros = weight(g, 33, 256, 32, BF16, True)
    x = torch.randn(4, 256, generator=g).to(BF16).to(DEV)
    high = torch.nn.functional.pad(zeros | 0xa0, (0, 8))[:, :8]
    assert torch.equal(ssm.w4_linear(x, codes, scales, zeros), ssm.w4_linear(x, codes, scales, high))


def test_repeats_agree_bit_by_bit():
    g = torch.Generator().manual_seed(16)
    w = weight(g, 1000, 3328, 128, BF16, True)
    for m in (1, 8, 30, 64, 100):
        x = torch.randn(m, 3328, generator=g).to(BF16).to(DEV)
        a = ssm.w4_linear(x, *w, out_dtype=F32)
        for _ in range(4):
            assert torch.equal(a, ssm.w4_linear(x, *w, out_dtype=F32))


@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (5, 128, 128), (17, 192, 64), (40, 4096, 128), (3, 160, 32), (9, 640, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scales", [BF16, F32])
def test_quantize_is_its_definition(n, k, group, dtype, zeros, scales):
    g = torch.Generator().manual_seed(n + k)
    W = (torch.randn(n, k + 5, generator=g) * 0.05).to(dtype)
    W[0, :min(k, group)] = 0.0                                  # a group of zeros
    if n > 2:
        W[1] = W[1].abs()                                       # one sign only
        W[2] = 0.25                                             # all alike
    W = W.to(DEV)[:, 2:2 + k]                                   # rows at odd offsets
    codes, s, z = ssm.w4_quantize(W, group, zeros, scales)
    c, rs, rz = quantise32(W, group, zeros, scales)
    assert torch.equal(s.cpu(), rs)
    assert (z is None) == (not zeros) and (z is None or np.array_equal(z.cpu().numpy(), rz))
    assert np.array_equal(unpack(codes), c)
    assert codes.shape == (n, k // 2) and s.dtype == scales


def test_a_quantised_projection_is_near_the_projection():
    """Codes are off by half a scale at most, and amax / 7 by the bf16 scale's rounding at the ends."""
    g = torch.Generator().manual_seed(18)
    W = (torch.randn(200, 1024, generator=g) / 32).to(BF16).to(DEV)
    x = torch.randn(6, 1024, generator=g).to(BF16).to(DEV)
    for zeros in (False, True):
        codes, s, z = ssm.w4_quantize(W, 64, zeros)
        got = ssm.w4_linear(x, codes, s, z, out_dtype=F32)
        ref = x.double() @ W.double().T
        step = s.double().repeat_interleave(64, 1) * (0.5 + (15 if zeros else 7) * 2.0 ** -8 + (0.5 if zeros else 0))
        assert ((got - ref).abs() <= x.double().abs() @ step.T).all()
