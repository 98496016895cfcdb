"""Each of the library's bounded waits, made to run out by something that nobody does: it is reported, the kernel ends, and
the calls that use it work afterwards."""
import time

import pytest
import torch

from _steps import check_linear, check_probs
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_wait_that_runs_out_is_reported(which):
    ssm.device_status()
    t0 = time.perf_counter()
    ssm.selftest_expire_wait(50000, which=which)
    torch.cuda.synchronize()
    assert 0.045 <= time.perf_counter() - t0 < 1.0
    assert ssm.device_status() == ssm.DEV_WAIT_TIMEOUT and ssm.device_status() == 0
    g = torch.Generator().manual_seed(which)
    x = torch.randn(3, 50021, generator=g).cuda()                       # a cluster a row
    check_probs(ssm.spec_probs(x), x, None)
    w = ssm.w4_quantize((torch.randn(60, 512, generator=g) / 20).cuda(), 64)
    h = torch.randn(5, 512, generator=g).to(torch.bfloat16).cuda()
    check_linear(ssm.w4_linear(h, *w), h, *w, None)
    assert ssm.device_status() == 0


@pytest.mark.parametrize("which", [-1, 3])
def test_other_waits_are_refused(which):
    with pytest.raises(ssm.SSMError, match="which"):
        ssm.selftest_expire_wait(1000, which=which)
