"""norm_rms where squares leave the range of fp32: rows near its lowest and its largest values, with and without eps."""
import numpy as np
import pytest
import torch

from _steps import check_norm, norm64, to64
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8
# a warp's forms and a block's, few rows (a vector a thread) and many (up to four)
SIZES = [(6, 64, 2), (7, 264, 1), (4, 2048, 1), (2, 8200, 1), (2, 32768, 1), (330, 512, 1), (310, 2048, 1), (320, 4096, 2), (2, 16384, 1)]


def at(exponent, t, width, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    x = (1 + torch.rand(t, width, generator=g, dtype=torch.float64)) * (1 - 2 * torch.randint(0, 2, (t, width), generator=g))
    return (x * 2.0 ** exponent).to(dtype).to(DEV)


@pytest.mark.parametrize("t,width,groups", SIZES)
@pytest.mark.parametrize("exponent", [-148, -140, -127, -100, -76, -62, -50, 55, 63, 64, 100, 126])
@pytest.mark.parametrize("out", [BF16, F32, I8])
def test_rows_of_every_size(t, width, groups, exponent, out):
    x = at(exponent, t, width, t + width)
    g = torch.Generator().manual_seed(2)
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(DEV)
    o, _, s = ssm.norm_rms(x, w, eps=0.0, n_groups=groups, out_dtype=out)
    check_norm(o, s, x, w, None, 0.0, groups)
    assert np.abs(to64(o)).max() > 0.5                              # about 1, or codes


@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -130, 2.0 ** -102, 2.0 ** -40, 1.0, 2.0 ** 100, 2.0 ** 127])
@pytest.mark.parametrize("exponent", [-149, -130, -75, -50, -20, 50, 64, 120])
def test_eps_beside_them(eps, exponent):
    for t, width, groups in ((5, 128, 2), (3, 4096, 1), (310, 2048, 1)):
        x = at(exponent, t, width, width)
        o, _, _ = ssm.norm_rms(x, None, eps=eps, n_groups=groups, out_dtype=F32)
        check_norm(o, None, x, None, None, eps, groups)


@pytest.mark.parametrize("out", [BF16, F32, I8])
def test_each_group_has_its_own(out):
    """Groups of different sizes in a row, some of them of zeros, and values of all sizes in one group."""
    sizes = [-140, 0, 100, -75, 64, 3]
    x = torch.cat([at(e, 9, 256, e + 200) for e in sizes] + [torch.zeros(9, 256, device=DEV)], 1)
    mixed = torch.cat([at(e, 9, 32, e + 300) for e in (-149, -120, -90, -60, -30, 0, 30, 60)], 1)
    x = torch.cat([x, mixed, mixed * 2.0 ** -80, mixed * 2.0 ** 60], 1)
    o, _, s = ssm.norm_rms(x, None, eps=2.0 ** -60, n_groups=10, out_dtype=out)
    check_norm(o, s, x, None, None, 2.0 ** -60, 10)
    assert (o[:, 6 * 256:7 * 256] == 0).all()


@pytest.mark.parametrize("out", [BF16, F32])
def test_sums_with_a_residual(out):
    """r is x + residual, rounded once; it is what is normed, and what residual_out takes."""
    for e in (-140, -80, 70, 120):
        x, res = at(e, 4, 1024, 1), at(e, 4, 1024, 2)
        o, r, _ = ssm.norm_rms(x, None, res, eps=0.0, out_dtype=out)
        assert torch.equal(r, x + res)
        check_norm(o, None, r, None, None, 0.0, 1)


@pytest.mark.parametrize("e", [-100, 0, 100])
def test_infinities_zeros_and_nan_beside_large_and_small_values(e):
    x = at(e, 5, 64, 7)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 40] = float("nan")
    x[3, :32] = 0.0
    o, _, _ = ssm.norm_rms(x, None, n_groups=2, eps=0.0, out_dtype=F32)
    o = o.view(5, 2, 32)
    assert torch.isnan(o[0]).all() and torch.isnan(o[3, 0]).all()           # 0 / 0
    assert torch.isnan(o[1, 0, 3]) and (o[1, 0, :3] == 0).all() and (o[1, 0, 4:] == 0).all()
    assert torch.isnan(o[2, 1]).all()
    y, _ = norm64(x, None, None, 0.0, 2)
    for r, j in ((1, 1), (2, 0), (3, 1), (4, 0), (4, 1)):
        assert np.abs(to64(o[r, j]) - y[r, j]).max() <= 1e-5 * np.abs(y[r, j]).max()


def test_a_small_row_beside_zero_eps_of_the_largest_bf16_values():
    big = torch.finfo(BF16).max
    x = torch.tensor([[big, -big] * 32, [2.0 ** -133] * 64], dtype=BF16, device=DEV)
    o, _, _ = ssm.norm_rms(x, None, eps=0.0, out_dtype=F32)
    check_norm(o, None, x, None, None, 0.0, 1)
