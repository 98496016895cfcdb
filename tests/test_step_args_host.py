"""The calls around a decode step's mixers: what they refuse, on the host and by name.  No GPU is needed: every
call is refused before a pointer is used."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from selective_state_space_prefill_gb300 import binding, build

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, -1, -2, -3
FAKE = 0x10000
F32, BF16, I8 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    build.build_step_calls()
    return binding.load()


NORM = dict(n_rows=2, width=64, n_groups=1, in_dtype=BF16, x=FAKE, x_stride=64, res_dtype=BF16, residual=FAKE, res_stride=64,
            residual_out=FAKE + 4096, ro_stride=64, weight=FAKE, eps=1e-5, out_dtype=BF16, out=FAKE, out_stride=64, out_scale=None,
            stream=None)
QUANT = dict(N=4, K=256, group=128, in_dtype=BF16, W=FAKE, ldw=256, codes=FAKE, ldc=128, scale_dtype=BF16, scales=FAKE, lds=8,
             zeros=FAKE, ldz=16, stream=None)
LINEAR = dict(M=2, N=4, K=256, group=128, x_dtype=BF16, x=FAKE, ldx=256, x_scale=None, x_blocks=1, codes=FAKE, ldc=128, scale_dtype=F32,
              scales=FAKE, lds=4, zeros=None, ldz=0, out_dtype=F32, out=FAKE, ldo=4, workspace=None, workspace_bytes=0, stream=None)
PROBS = dict(n_rows=2, vocab=10, in_dtype=BF16, logits=FAKE, ld_in=10, temperature=FAKE, probs=FAKE, ld_out=10, stream=None)
VERIFY = dict(batch=2, n_max=3, vocab=10, draft=FAKE, n_draft=FAKE, target_probs=FAKE, tp_sb=40, tp_st=10, draft_probs=FAKE, dp_sb=30,
              dp_st=10, u=FAKE, tokens=FAKE, n_kept=FAKE, stream=None)
REFUSED = [
    ("norm_rms", NORM, [
        (dict(n_rows=-1), INVALID), (dict(width=0), INVALID), (dict(n_groups=0), INVALID), (dict(n_groups=3), INVALID),
        (dict(n_groups=16), UNSUPPORTED), (dict(width=68, x_stride=72), UNSUPPORTED), (dict(width=32776), UNSUPPORTED),
        (dict(n_rows=1 << 31), UNSUPPORTED), (dict(n_rows=1 << 28, n_groups=8), UNSUPPORTED), (dict(in_dtype=2), INVALID),
        (dict(res_dtype=2), INVALID), (dict(out_dtype=3), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
        (dict(eps=float("inf")), INVALID), (dict(residual=None), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
        (dict(x_stride=56), INVALID), (dict(out_stride=56), INVALID), (dict(res_stride=60), INVALID), (dict(ro_stride=0), INVALID),
        (dict(x_stride=68), MISALIGNED), (dict(x=FAKE + 8), MISALIGNED), (dict(residual=FAKE + 2), MISALIGNED),
        (dict(out=FAKE + 8), MISALIGNED), (dict(weight=FAKE + 4), MISALIGNED), (dict(residual_out=FAKE, ro_stride=72), INVALID),
        (dict(out_scale=FAKE), INVALID), (dict(out_dtype=I8), INVALID), (dict(out_dtype=I8, out_scale=FAKE + 2), MISALIGNED),
        (dict(out_dtype=I8, out_scale=FAKE, out=FAKE + 4), MISALIGNED)]),
    ("w4_quantize", QUANT, [
        (dict(N=0), INVALID), (dict(N=(1 << 27) + 1), INVALID), (dict(K=0), INVALID), (dict(K=192), INVALID), (dict(group=16), UNSUPPORTED),
        (dict(group=256), UNSUPPORTED), (dict(K=32896, ldw=32896, ldc=16448, lds=520, ldz=528), UNSUPPORTED), (dict(in_dtype=2), INVALID),
        (dict(scale_dtype=2), INVALID), (dict(W=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
        (dict(ldw=255), INVALID), (dict(ldc=112), INVALID), (dict(lds=1), INVALID), (dict(ldz=1), INVALID), (dict(ldc=136), MISALIGNED),
        (dict(lds=4), MISALIGNED), (dict(ldz=8), MISALIGNED), (dict(codes=FAKE + 8), MISALIGNED), (dict(scales=FAKE + 8), MISALIGNED),
        (dict(zeros=FAKE + 4), MISALIGNED), (dict(W=FAKE + 1), MISALIGNED)]),
    ("w4_linear", LINEAR, [
        (dict(M=-1), INVALID), (dict(M=257), UNSUPPORTED), (dict(N=0), INVALID), (dict(K=192), INVALID), (dict(group=96), UNSUPPORTED),
        (dict(x_dtype=F32), UNSUPPORTED), (dict(x_dtype=5), INVALID), (dict(out_dtype=2), INVALID), (dict(x=None), INVALID),
        (dict(out=None), INVALID), (dict(ldx=248), INVALID), (dict(ldo=3), INVALID), (dict(ldx=260), MISALIGNED), (dict(x=FAKE + 8), MISALIGNED),
        (dict(x_scale=FAKE), INVALID), (dict(x_dtype=I8), INVALID), (dict(x_dtype=I8, x_scale=FAKE, x_blocks=0), INVALID),
        (dict(x_dtype=I8, x_scale=FAKE, x_blocks=4), INVALID), (dict(x_dtype=I8, x_scale=FAKE, x_blocks=65), INVALID),
        (dict(x_blocks=2), INVALID), (dict(x_dtype=I8, x_scale=FAKE, ldx=264), MISALIGNED), (dict(out=FAKE + 2), MISALIGNED),
        (dict(x_dtype=I8, x_scale=FAKE + 2), MISALIGNED), (dict(lds=5), MISALIGNED), (dict(zeros=FAKE, ldz=2), MISALIGNED),
        (dict(ldc=127), INVALID)]),
    ("spec_probs", PROBS, [
        (dict(n_rows=-1), INVALID), (dict(n_rows=1 << 28), INVALID), (dict(vocab=0), INVALID), (dict(vocab=(1 << 24) + 1), INVALID),
        (dict(in_dtype=2), INVALID), (dict(logits=None), INVALID), (dict(probs=None), INVALID), (dict(ld_in=9), INVALID),
        (dict(ld_out=9), INVALID), (dict(logits=FAKE + 1), MISALIGNED), (dict(probs=FAKE + 2), MISALIGNED),
        (dict(temperature=FAKE + 2), MISALIGNED)]),
    ("spec_verify", VERIFY, [
        (dict(batch=-1), INVALID), (dict(batch=65536), INVALID), (dict(n_max=-1), INVALID), (dict(n_max=1025), INVALID),
        (dict(vocab=0), INVALID), (dict(vocab=(1 << 24) + 1), INVALID), (dict(draft=None), INVALID), (dict(target_probs=None), INVALID),
        (dict(u=None), INVALID), (dict(tokens=None), INVALID), (dict(n_kept=None), INVALID), (dict(tp_st=9), INVALID),
        (dict(tp_sb=9), INVALID), (dict(dp_st=9), INVALID), (dict(dp_sb=9), INVALID), (dict(u=FAKE + 2), MISALIGNED),
        (dict(draft=FAKE + 1), MISALIGNED), (dict(target_probs=FAKE + 2), MISALIGNED), (dict(tokens=FAKE + 2), MISALIGNED)]),
]


@pytest.mark.parametrize("fn,base,change,code", [(f, b, c, r) for f, b, rows in REFUSED for c, r in rows])
def test_library_refuses(lib, fn, base, change, code):
    a = dict(base)
    assert set(change) <= set(a)
    a.update(change)
    assert getattr(lib, fn)(*a.values()) == code
    assert lib.ssm_last_error().decode().startswith(fn)


def test_linear_wants_a_workspace_for_long_rows(lib):
    need = lib.w4_linear_workspace_bytes(2, 4, 32768, 128)
    assert need >= 8 * 2 * 4 * 4 and need % (2 * 4 * 4) == 0                # at least eight slices' sums
    long = dict(LINEAR, K=32768, ldx=32768, ldc=16384, lds=256)
    for more, code in ((dict(), INVALID), (dict(workspace=FAKE, workspace_bytes=need - 1), INVALID),
                       (dict(workspace=FAKE + 8, workspace_bytes=need), MISALIGNED)):
        assert lib.w4_linear(*{**long, **more}.values()) == code
        assert "workspace" in lib.ssm_last_error().decode()
    assert lib.w4_linear_workspace_bytes(8, 16384, 4096, 128) == 0          # 4096 elements are one slice
    for bad in ((0, 4, 128, 128), (257, 4, 128, 128), (1, 0, 128, 128), (1, 4, 192, 128), (1, 4, 128, 16), (1, 4, 32896, 128)):
        assert lib.w4_linear_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("fn,base,change", [("norm_rms", NORM, dict(n_rows=0, x=None, out=None)), ("w4_linear", LINEAR, dict(M=0, x=None, out=None)),
                                            ("spec_probs", PROBS, dict(n_rows=0, logits=None, probs=None)),
                                            ("spec_verify", VERIFY, dict(batch=0, target_probs=None, u=None))])
def test_nothing_to_do_is_no_error(lib, fn, base, change):
    assert getattr(lib, fn)(*{**base, **change}.values()) == OK


# ------------------------------------------------------------------ the binding
def _t(*shape, dtype=torch.bfloat16, device="cuda:0"):
    return torch.empty(*shape, device=device, dtype=dtype)


def _f(*shape):
    return _t(*shape, dtype=torch.float32)


def _u8(*shape):
    return _t(*shape, dtype=torch.uint8)


def _i(*shape):
    return _t(*shape, dtype=torch.int32)


CALLS = {
    "norm_rms": lambda: dict(x=_t(4, 64), weight=_f(64), residual=_t(4, 64), out=_t(4, 64, dtype=torch.int8), residual_out=_t(4, 64),
                             out_scale=_f(4, 1)),
    "w4_quantize": lambda: dict(W=_t(8, 256)),
    "w4_linear": lambda: dict(x=_t(4, 256, dtype=torch.int8), codes=_u8(8, 128), scales=_f(8, 4), zeros=_u8(8, 4), x_scale=_f(4), out=_t(4, 8),
                              workspace=_u8(64)),
    "spec_probs": lambda: dict(logits=_t(4, 100), temperature=_f(4), out=_f(4, 100)),
    "spec_verify": lambda: dict(draft=_i(2, 3), target_probs=_f(2, 4, 10), u=_f(2, 4), draft_probs=_f(2, 3, 10), n_draft=_i(2), tokens=_i(2, 4),
                                n_kept=_i(2)),
}
NAMES = [(fn, name) for fn, names in {
    "norm_rms": "x weight residual out residual_out out_scale", "w4_linear": "x codes scales zeros x_scale out workspace",
    "spec_probs": "logits temperature out", "spec_verify": "draft target_probs u draft_probs n_draft tokens n_kept",
}.items() for name in names.split()]


@pytest.mark.parametrize("fn,name", NAMES)
def test_a_tensor_on_another_gpu_is_refused(lib, fn, name):
    with FakeTensorMode():
        kw = CALLS[fn]()
        x = kw[name]
        kw[name] = torch.empty(x.shape, dtype=x.dtype, device="cuda:1")
        with pytest.raises(ValueError, match=r"is on cuda:\d, other arguments on cuda:\d"):
            getattr(binding, fn)(**kw)


def test_every_tensor_argument_is_looked_at():
    with FakeTensorMode():
        for fn, make in CALLS.items():
            assert {n for f, n in NAMES if f == fn} == (set(make()) if fn != "w4_quantize" else set())


def on_cpu(fn):
    with FakeTensorMode():
        like = {n: (tuple(t.shape), t.dtype) for n, t in CALLS[fn]().items()}
    return {n: torch.zeros(s, dtype=d) for n, (s, d) in like.items()}


@pytest.mark.parametrize("fn", CALLS)
def test_cpu_tensors_are_refused(lib, fn):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        getattr(binding, fn)(**on_cpu(fn))


@pytest.mark.parametrize("fn,change,error", [
    ("norm_rms", dict(x=3), "x must be a tensor"), ("w4_linear", dict(x=None), "x must be a tensor"),
    ("spec_probs", dict(logits=[1.0]), "logits must be a tensor"), ("spec_probs", dict(top=1), "unexpected keyword"),
    ("spec_verify", dict(target_probs="p"), "target_probs must be a tensor"), ("w4_quantize", dict(W=1), "W must be a tensor")])
def test_other_objects_are_refused(lib, fn, change, error):
    with pytest.raises((TypeError, ValueError), match=error):
        getattr(binding, fn)(**{**on_cpu(fn), **change})


def test_the_wrong_number_of_arguments_is_refused(lib):
    with pytest.raises(TypeError, match="10 arguments expected, 1 given"):
        binding.step_calls().norm(1)
