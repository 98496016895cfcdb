"""Host-side checks of the attention calls that need no GPU: every refusal comes before a CUDA call
(the pointers are fake), the binding's own checks, and the rope frequencies."""
import ctypes
import math

import pytest
import torch

from selective_state_space_prefill_gb300 import binding, build
from selective_state_space_prefill_gb300.rope import rope_frequencies

INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    build.build_calls()
    return binding.load()


def _refused(lib, fn, base, kw, code):
    assert set(kw) <= set(base), kw
    assert getattr(lib, fn)(*dict(base, **kw).values()) == code, kw
    assert lib.ssm_last_error().decode().startswith(fn)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), INVALID), (dict(half=0), INVALID), (dict(half=65), INVALID), (dict(freq=None), INVALID),
    (dict(cos=None), INVALID), (dict(scale=math.inf), INVALID), (dict(sin=FAKE + 2), MISALIGNED),
])
def test_rope_table_refusals(lib, kw, code):
    arr = (ctypes.c_double * 64)(*([1.0] * 64))
    base = dict(n=16, half=32, freq=ctypes.cast(arr, ctypes.c_void_p), scale=1.0, cos=FAKE, sin=FAKE, stream=None)
    _refused(lib, "attn_rope_table", base, kw, code)


APPEND = dict(n=4, H=8, Hk=2, D=64, rot=64, inter=0, q=FAKE, qt=512, qh=64, k=FAKE, kt=128, kh=64, v=FAKE, vt=128,
              vh=64, pos=FAKE, cos=FAKE, sin=FAKE, n_pos=100, slots=FAKE, dtype=2, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
              pages=4, page=16, qo=2 * FAKE, qot=512, qoh=64, ko=None, kot=0, koh=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(H=7), INVALID), (dict(Hk=0), INVALID), (dict(D=72), UNSUPPORTED),
    (dict(D=144), UNSUPPORTED), (dict(rot=72), INVALID), (dict(rot=12), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), MISALIGNED), (dict(kt=132), MISALIGNED), (dict(qh=32), INVALID), (dict(qo=None), INVALID),
    (dict(qot=64), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(cos=FAKE + 4), MISALIGNED),
    (dict(n_pos=0), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(dtype=9), INVALID), (dict(ks=None), INVALID),
    (dict(dtype=1), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=8192), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(pages=1 << 30), UNSUPPORTED), (dict(kc=FAKE + 4), MISALIGNED), (dict(qo=FAKE, qot=1024), INVALID),
    (dict(ko=FAKE, kot=256, koh=64), INVALID),
])
def test_append_refusals(lib, kw, code):
    _refused(lib, "attn_append", APPEND, kw, code)


READ = dict(batch=2, n=8, Hk=2, D=64, dtype=2, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pages=4, page=16, table=FAKE, ts=4,
            nt=4, cu=FAKE, first=None, odt=1, k=FAKE, v=FAKE, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(n=-1), INVALID), (dict(D=8), UNSUPPORTED), (dict(odt=2), INVALID),
    (dict(table=None), INVALID), (dict(ts=3), INVALID), (dict(nt=0), INVALID), (dict(cu=None), INVALID),
    (dict(k=None), INVALID), (dict(v=FAKE + 8), MISALIGNED), (dict(first=FAKE + 2), MISALIGNED), (dict(vs=None), INVALID),
])
def test_read_refusals(lib, kw, code):
    _refused(lib, "attn_cache_read", READ, kw, code)


PREFILL = dict(batch=1, tq=4, tk=4, max_q=4, H=8, Hk=2, D=64, idt=1, odt=1, q=FAKE, qt=512, qh=64, k=FAKE, kt=128, kh=64,
               v=FAKE, vt=128, vh=64, cuq=FAKE, cuk=FAKE, scale=0.125, out=FAKE, ot=512, oh=64, lse=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(tq=-1), INVALID), (dict(max_q=-1), INVALID), (dict(H=3), INVALID),
    (dict(D=200), UNSUPPORTED), (dict(idt=0), UNSUPPORTED), (dict(idt=2), INVALID), (dict(odt=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(cuq=None), INVALID), (dict(q=None), INVALID), (dict(kt=100), MISALIGNED), (dict(vh=16), INVALID),
    (dict(out=None), INVALID), (dict(ot=64), INVALID), (dict(out=FAKE + 2), MISALIGNED), (dict(lse=FAKE + 2), MISALIGNED),
    (dict(batch=65535, tq=1 << 26, max_q=1 << 20), UNSUPPORTED),
])
def test_prefill_refusals(lib, kw, code):
    _refused(lib, "attn_prefill", PREFILL, kw, code)


DECODE = dict(batch=2, H=8, Hk=2, D=64, idt=1, odt=1, q=FAKE, qt=512, qh=64, dtype=2, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
              pages=4, page=16, table=FAKE, ts=4, nt=4, lens=FAKE, max_len=64, scale=0.125, out=FAKE, ot=512, oh=64,
              lse=None, ws=FAKE, wsb=1 << 40, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(max_len=0), INVALID), (dict(idt=0), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(q=FAKE + 8), MISALIGNED), (dict(lens=None), INVALID), (dict(nt=0), INVALID), (dict(ks=None), INVALID),
    (dict(out=None), INVALID), (dict(ot=256), INVALID), (dict(D=24), UNSUPPORTED), (dict(page=0), INVALID),
])
def test_decode_refusals(lib, kw, code):
    _refused(lib, "attn_decode_step", DECODE, kw, code)


def test_decode_short_workspace_is_refused(lib):
    need = lib.attn_decode_workspace_bytes(1, 8, 2, 64, 1 << 20)
    base = dict(DECODE, batch=1, max_len=1 << 20)
    if need:
        _refused(lib, "attn_decode_step", base, dict(wsb=need - 1), INVALID)
        _refused(lib, "attn_decode_step", base, dict(ws=None), INVALID)
        _refused(lib, "attn_decode_step", base, dict(ws=FAKE + 8), MISALIGNED)
    assert lib.attn_decode_workspace_bytes(0, 8, 2, 64, 64) == 0
    assert lib.attn_decode_workspace_bytes(1, 8, 3, 64, 64) == 0


def test_calls_without_tokens_do_nothing(lib):
    assert lib.attn_append(*dict(APPEND, n=0, k=None, v=None, q=None, qo=None, slots=None).values()) == 0
    assert lib.attn_cache_read(*dict(READ, n=0, k=None, v=None).values()) == 0
    assert lib.attn_prefill(*dict(PREFILL, tq=0, q=None, out=None).values()) == 0


def test_binding_checks_come_first(lib):
    """CPU tensors, wrong shapes and types are refused by the binding itself."""
    bf = torch.bfloat16
    x = torch.zeros(4, 2, 64, dtype=bf)
    i32 = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):
        binding.attn_append(None, x, x, None, None, None, cache, cache, i32)
    with pytest.raises(TypeError):
        binding.attn_append(None, x, x, None, None, None, cache.float(), cache.float(), i32)
    with pytest.raises(ValueError):
        binding.attn_prefill(x, x, x, i32, i32, 4)
    with pytest.raises(ValueError):
        binding.attn_prefill(x[0], x, x, i32, i32, 4)
    with pytest.raises(ValueError):
        binding.attn_decode_step(x, cache, cache, i32[None], i32, 16)
    with pytest.raises(ValueError):
        binding.attn_cache_read(cache, cache, i32[None], i32, 4)


def test_rope_frequencies():
    f, s = rope_frequencies(8, 10000.0)
    assert s == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001])
    assert rope_frequencies(8, 10000.0, "linear", 4.0)[0] == pytest.approx([x / 4 for x in f])
    n, s = rope_frequencies(64, 10000.0, "ntk", 8.0)
    base = rope_frequencies(64)[0]
    assert s == 1.0 and n[0] == base[0] and n[-1] == pytest.approx(base[-1] / 8.0)
    y, s = rope_frequencies(64, 10000.0, "yarn", 8.0, original_len=4096)
    assert s == pytest.approx(0.1 * math.log(8.0) + 1.0)
    turns = [4096 * b / (2 * math.pi) for b in base]
    for a, b, t in zip(y, base, turns):
        assert b / 8.0 * 0.999999 <= a <= b * 1.000001
        if t > 32:
            assert a == pytest.approx(b)
        if t < 1:
            assert a == pytest.approx(b / 8.0)
    for bad in (dict(rot_dim=3), dict(rot_dim=8, factor=0.5), dict(rot_dim=8, scaling="cubic"),
                dict(rot_dim=8, scaling="yarn", factor=2.0), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            rope_frequencies(**bad)
