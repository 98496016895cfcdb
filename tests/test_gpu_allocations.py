"""Outputs and workspaces that the attention calls and the calls around the mixers make: seen by dispatch modes and by the
profiler, and filled where torch is told to fill new memory."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import test_gpu_attention_streams as attention
import test_gpu_step_chain as step
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"
# outputs and workspaces that a call makes
CALLS = [(attention, "append", 2), (attention, "read", 2), (attention, "prefill", 2), (attention, "decode", 3),
         (step, "norm", 3), (step, "quantize", 3), (step, "linear", 1), (step, "slices", 2), (step, "tiles", 2), (step, "probs", 1), (step, "verify", 2)]
IDS = [f"{m.__name__[9:]}-{c}" for m, c, _ in CALLS]


class Made(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.seen.append(out)
        return out


@pytest.mark.parametrize("module,call,made", CALLS, ids=IDS)
def test_a_dispatch_mode_sees_them(module, call, made):
    s = module.Setup()
    want = [t.clone() for t in getattr(s, call)() if t is not None]
    with Made() as mode:
        got = [t for t in getattr(s, call)() if t is not None]
    assert len(mode.seen) == made
    assert {t.untyped_storage().data_ptr() for t in got} <= {t.untyped_storage().data_ptr() for t in mode.seen} | {s_ptr for s_ptr in _given(s)}
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def _given(s):
    return [t.untyped_storage().data_ptr() for t in vars(s).values() if isinstance(t, torch.Tensor)]


def test_a_profiler_sees_them():
    s = step.Setup()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
        s.norm()
    assert sum(e.name == "aten::empty" for e in p.events()) == 3


def test_unwritten_rows_are_filled_where_new_memory_is():
    """Rows behind the last sequence are left as they were: NaN, where new memory is filled."""
    s = attention.Setup()
    before = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    q = torch.cat([s.q, s.q])
    dirty = [torch.full_like(q, 3.0) for _ in range(4)]
    del dirty                                                           # what such memory is handed out as else
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        out, _ = ssm.attn_prefill(q, s.k, s.v, s.cu, s.cu, s.n)
        step_outs = step.Setup().norm()
    finally:
        torch.use_deterministic_algorithms(before[0])
        torch.utils.deterministic.fill_uninitialized_memory = before[1]
    assert torch.isnan(out[s.n:]).all() and torch.equal(out[:s.n], ssm.attn_prefill(s.q, s.k, s.v, s.cu, s.cu, s.n)[0])
    for a, b in zip(step_outs, step.Setup().norm()):
        assert torch.equal(a, b)
