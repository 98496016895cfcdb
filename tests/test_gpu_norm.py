"""norm_rms against its definition in 64 bits: types, groups, strides, sizes from one vector to the largest group,
rows of zeros, infinities and NaN, in-place residuals."""
import numpy as np
import pytest
import torch

from _steps import check_norm, norm64, to64
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def rows(g, t, w, dtype, spread=0.5):
    x = torch.randn(t, w, generator=g) * torch.exp(spread * torch.randn(w, generator=g))
    return x.to(dtype).to(DEV)


# (rows, width, groups): one vector of eight, widths around a warp's and a block's vectors, odd numbers of vectors,
# groups of one vector, the largest group
SIZES = [(1, 8, 1), (3, 16, 2), (5, 248, 1), (2, 256, 1), (7, 264, 1), (4, 1000, 5), (1, 1536, 1), (9, 2048, 8), (33, 2056, 1),
         (2, 5120, 8), (3, 7168, 1), (1, 8200, 1), (2, 16384, 1), (1, 32768, 1), (2, 65536, 2), (130, 640, 80), (1, 16, 2),
         (1000, 64, 1), (5, 4096, 2), (6, 12296, 1)]


@pytest.mark.parametrize("t,width,groups", SIZES)
@pytest.mark.parametrize("x,res,out", [(BF16, None, BF16), (BF16, BF16, I8), (F32, None, F32), (BF16, F32, BF16), (F32, BF16, I8),
                                       (F32, F32, I8), (F32, BF16, F32)])
def test_sizes_and_types(t, width, groups, x, res, out):
    g = torch.Generator().manual_seed(t * 31 + width)
    xs = rows(g, t, width, x)
    rs = None if res is None else 3 * rows(g, t, width, res)
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(DEV)
    o, r, s = ssm.norm_rms(xs, w, rs, eps=1e-5, n_groups=groups, out_dtype=out)
    assert o.dtype == out and o.shape == xs.shape and (s is None) == (out != I8) and (r is None) == (rs is None)
    check_norm(o, s, xs, w, rs, 1e-5, groups)
    if rs is not None:
        assert torch.equal(r, (xs.float() + rs.float()).to(res))
    assert ssm.device_status() == 0


@pytest.mark.parametrize("out", [BF16, I8])
def test_strides_and_neighbours(out):
    """Slices of wider rows are read and written in place; what lies around an output stays."""
    g = torch.Generator().manual_seed(3)
    wide = rows(g, 6, 96 + 520 + 40, BF16)
    x = wide[:, 96:96 + 520]
    res = rows(g, 12, 528, F32)[::2, :520]
    target = torch.full((6, 640), 7, dtype=out, device=DEV)
    kept = torch.full((6, 640), 7.0, device=DEV)
    scale = torch.empty(6, 1, device=DEV) if out == I8 else None
    o, r, s = ssm.norm_rms(x, None, res, out=target[:, 8:528], residual_out=kept[:, 16:536], out_scale=scale)
    check_norm(o, s, x, None, res, 1e-5, 1)
    assert torch.equal(kept[:, 16:536], x.float() + res)
    for t, a, b in ((target, 8, 528), (kept, 16, 536)):
        assert (t[:, :a] == 7).all() and (t[:, b:] == 7).all()


def test_residual_in_place_and_skipped():
    g = torch.Generator().manual_seed(4)
    x, res = rows(g, 5, 1024, BF16), rows(g, 5, 1024, BF16)
    want, r, _ = ssm.norm_rms(x, None, res)
    same = res.clone()
    got, r2, _ = ssm.norm_rms(x, None, same, residual_out=same)
    assert r2 is same and torch.equal(same, r) and torch.equal(got, want)
    got, r3, _ = ssm.norm_rms(x, None, res, residual_out=False)
    assert r3 is None and torch.equal(got, want)


@pytest.mark.parametrize("out", [BF16, F32, I8])
def test_zeros_infinities_and_nan_stay_in_their_group(out):
    g = torch.Generator().manual_seed(5)
    x = rows(g, 5, 64, F32)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 40] = float("nan")
    x[3, :] = 1e-30
    o, _, s = ssm.norm_rms(x, None, n_groups=2, eps=0.0 if out == F32 else 1e-5, out_dtype=out)
    o = o.float().view(5, 2, 32)
    clean = [(0, 1) if out != F32 else None, (1, 1), (2, 0), (3, 0), (4, 0), (4, 1)]
    for c in clean:
        if c and c[0] != 3:
            r, j = c
            check_norm((o[r, j][None]).to(out), None if s is None else s[r:r + 1, j:j + 1], x[r:r + 1, 32 * j:32 * j + 32], None, None,
                       0.0 if out == F32 else 1e-5, 1)
    if out == I8:
        # 1 / sqrt(inf) = 0: the finite ones 0, the infinite one NaN, whose code is 0
        assert (o[1, 0] == 0).all() and s[1, 0] == 0
        assert (o[2, 1] == 0).all() and s[2, 1] == 0        # all NaN: ignored by the maximum
        assert (o[0] == 0).all() and (s[0] == 0).all()
    else:
        assert torch.isnan(o[1, 0, 3]) and (o[1, 0, :3] == 0).all()
        assert torch.isnan(o[2, 1]).all()
        if out == F32:
            assert torch.isnan(o[0]).all()                  # 0 / 0 with eps 0
        else:
            assert (o[0] == 0).all()


def test_an_infinite_weight_gives_an_infinite_scale():
    x = torch.ones(1, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    w[5] = float("inf")
    o, _, s = ssm.norm_rms(x, w, out_dtype=I8)
    assert (o == 0).all() and torch.isinf(s).all()


def test_no_rows():
    x = torch.empty(0, 64, device=DEV, dtype=BF16)
    o, r, s = ssm.norm_rms(x, None, x, out_dtype=I8)
    assert o.shape == (0, 64) and r.shape == (0, 64) and s.shape == (0, 1)


def test_int8_rows_read_back():
    """Codes times scales are y within half a code."""
    g = torch.Generator().manual_seed(6)
    x = rows(g, 17, 512, BF16)
    o, _, s = ssm.norm_rms(x, None, n_groups=4, out_dtype=I8)
    y, _ = norm64(x, None, None, 1e-5, 4)
    back = to64(o).reshape(y.shape) * to64(s)[..., None]
    assert (np.abs(back - y) <= to64(s)[..., None] * 0.501).all()
    assert (to64(o).reshape(y.shape).__abs__().max(-1) == 127).all()


def test_many_rows_and_repeats():
    g = torch.Generator().manual_seed(7)
    x = rows(g, 5000, 768, BF16)
    res = rows(g, 5000, 768, F32)
    a = ssm.norm_rms(x, None, res, out_dtype=I8)
    check_norm(a[0], a[2], x, None, res, 1e-5, 1)
    for _ in range(3):
        for u, v in zip(ssm.norm_rms(x, None, res, out_dtype=I8), a):
            assert torch.equal(u, v)
