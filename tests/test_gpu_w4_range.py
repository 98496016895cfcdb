"""w4_quantize of weights near the ends of fp32's range: every finite weight is held to half a scale, or a little more."""
import pytest
import torch

from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("exponent", [-120, -100, 0, 100, 126, 127])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.bfloat16])
def test_weights_of_every_size(exponent, group, zeros, scale_dtype):
    """Off by half a scale; at the ends by up to the codes' range times the scale's own rounding (2^-8 for bf16, 2^-24 thrice
    for fp32); with zeros, by half a scale for the zero's."""
    g = torch.Generator().manual_seed(group)
    top = float(torch.finfo(torch.float32).max) if exponent == 127 else 2.0 ** exponent
    W = ((2 * torch.rand(9, 3 * group, generator=g, dtype=torch.float64) - 1) * top).float()
    W[0, 0], W[0, 1] = top, -top
    W[1] = W[1].abs()
    codes, s, z = ssm.w4_quantize(W.to(DEV), group, zeros, scale_dtype)
    assert torch.isfinite(s).all()
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(9, 3 * group).cpu().double()
    zero = z.cpu().double() if zeros else torch.full((9, 3), 8.0, dtype=torch.float64)
    step = s.cpu().double().repeat_interleave(group, 1)
    back = (c - zero.repeat_interleave(group, 1)) * step
    own = 2.0 ** -8 if scale_dtype == torch.bfloat16 else 3 * 2.0 ** -24
    limit = step * (0.5 + (15 if zeros else 7) * own * 1.01 + (0.5 if zeros else 0) + 1e-6)
    assert ((back - W.double()).abs() <= limit).all()
