"""Tensors of one attention call on different GPUs are refused on the host, and a call works on the
device of its tensors, not on the current one.  No GPU is needed: fake tensors carry the devices, and
every refusal comes before a pointer is taken."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from selective_state_space_prefill_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    build.build_calls()


def _t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, device="cuda:0", dtype=dtype)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


def _f(*shape):
    return _t(*shape, dtype=torch.float32)


def _i8(*shape):
    return _t(*shape, dtype=torch.int8)


# the tensors of each call, in the call's own names, and its other arguments
CALLS = {
    "attn_append": (lambda: dict(q=_t(4, 2, 64), k=_t(4, 1, 64), v=_t(4, 1, 64), positions=_i(4), cos=_f(9, 32), sin=_f(9, 32),
                                 k_cache=_i8(2, 1, 16, 64), v_cache=_i8(2, 1, 16, 64), slots=_i(4), k_scale=_f(2, 1, 16),
                                 v_scale=_f(2, 1, 16), q_out=_t(4, 2, 64), k_out=_t(4, 1, 64)), {}),
    "attn_cache_read": (lambda: dict(k_cache=_i8(2, 1, 16, 64), v_cache=_i8(2, 1, 16, 64), page_table=_i(1, 2), cu_len=_i(2),
                                     k_scale=_f(2, 1, 16), v_scale=_f(2, 1, 16), first=_i(1), k_out=_t(4, 1, 64),
                                     v_out=_t(4, 1, 64)), dict(n_tokens=4)),
    "attn_prefill": (lambda: dict(q=_t(4, 2, 64), k=_t(4, 1, 64), v=_t(4, 1, 64), cu_q=_i(2), cu_k=_i(2), out=_t(4, 2, 64),
                                  lse=_f(4, 2)), dict(max_q=4)),
    "attn_decode_step": (lambda: dict(q=_t(1, 2, 64), k_cache=_i8(2, 1, 16, 64), v_cache=_i8(2, 1, 16, 64), page_table=_i(1, 2),
                                      lens=_i(1), k_scale=_f(2, 1, 16), v_scale=_f(2, 1, 16), out=_t(1, 2, 64), lse=_f(1, 2),
                                      workspace=_t(64, dtype=torch.uint8)), dict(max_len=16)),
}
CASES = [(fn, name) for fn, names in {
    "attn_append": "q k v positions cos sin k_cache v_cache slots k_scale v_scale q_out k_out",
    "attn_cache_read": "k_cache v_cache page_table cu_len k_scale v_scale first k_out v_out",
    "attn_prefill": "q k v cu_q cu_k out lse",
    "attn_decode_step": "q k_cache v_cache page_table lens k_scale v_scale out lse workspace",
}.items() for name in names.split()]


@pytest.mark.parametrize("fn,name", CASES)
def test_a_tensor_on_another_gpu_is_refused(fn, name):
    make, rest = CALLS[fn]
    with FakeTensorMode():
        kw = make()
        assert name in kw
        x = kw[name]
        kw[name] = torch.empty(x.shape, dtype=x.dtype, device="cuda:1")
        with pytest.raises(ValueError, match=r"is on cuda:\d, other arguments on cuda:\d"):
            getattr(binding, fn)(**kw, **rest)


def test_every_tensor_argument_is_looked_at():
    """The lists above hold every tensor that the calls take."""
    with FakeTensorMode():
        for fn, (make, _) in CALLS.items():
            assert {n for f, n in CASES if f == fn} == set(make())


def test_rope_table_runs_on_its_tables_device(monkeypatch):
    seen, here = [], []

    class Lib:
        def attn_rope_table(self, *a):
            seen.append(list(here))
            return 0

    @contextlib.contextmanager
    def device(d):
        here.append(torch.device(d))
        yield
        here.pop()

    monkeypatch.setattr(binding, "load", lambda: Lib())
    monkeypatch.setattr(binding, "_ptr", lambda t: None)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: type("S", (), {"cuda_stream": 0})())
    with FakeTensorMode():
        cos, sin = binding.attn_rope_table([1.0, 0.5], 8, device="cuda:1")
    assert cos.device == sin.device == torch.device("cuda:1") and seen == [[torch.device("cuda:1")]]
