"""spec_probs of logits whose differences pass the largest float, at temperatures up to infinity."""
import numpy as np
import pytest
import torch

from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = float(torch.finfo(torch.float32).max)


@pytest.mark.parametrize("v", [5, 3000, 50021, 300001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_whole_range_of_logits(v, dtype):
    """An infinite temperature counts as the largest float.  The exponent's parts are at most 2.9 there, with 21 bits or more
    of 1 / t (a subnormal): 2^-20 and what check_probs allows; sums of v terms, v / 512 + 32 additions in a thread."""
    top = float(torch.finfo(dtype).max)
    g = torch.Generator().manual_seed(v)
    x = ((2 * torch.rand(6, v, generator=g, dtype=torch.float64) - 1) * top).to(dtype)
    x[:, 0], x[:, v - 1] = -top, top
    t = torch.tensor([float("inf"), MOST, 3.1e38, 2.0e38, 1.0e37, 1.0])
    got = ssm.spec_probs(x.to(DEV), t.to(DEV)).cpu().double().numpy()
    xs = x.double().numpy()
    for r in range(6):
        d = (xs[r] - xs[r].max()) / min(float(t[r]), MOST)
        e = np.exp(d)
        want = e / e.sum()
        near = np.minimum(-d, 110.0)
        rel = near * 2.0 ** -20 + (16 + 4 * 20 + v / 512 + 32) * 2.0 ** -24
        assert (np.abs(got[r] - want) <= want * rel + 2.0 ** -125).all()
        assert got[r, 0] > 0 or r > 3
