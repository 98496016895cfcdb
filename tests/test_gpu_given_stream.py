"""The mixer, projection and reduction calls on a stream given by the caller: the bits of the current one,
outputs and workspaces that no other pending work uses."""
import pytest
import torch

from selective_state_space_prefill_gb300 import binding as ssm
from selective_state_space_prefill_gb300.inputs import (make_mixer_inputs, make_partials, make_ssd_inputs, make_ssd_states,
                                                        make_states)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 100_000_000            # cycles: some 50 ms


def _copies(states, stream=None):
    """States to advance in place, copied on the stream that the call runs on."""
    with torch.cuda.stream(stream):
        return [t.clone() for t in states]


def _call(name):
    """A function of `stream` that makes one call with outputs (and workspace) made by the binding."""
    if name in ("prefill", "prefill_segmented", "decode_step", "decode_tokens"):
        m = make_mixer_inputs(2, 256, 64, seed=3, dtype=torch.bfloat16).to(DEV)
        tok = (m.x, m.z, m.dt, m.B, m.C)
        par = (m.A, m.D, m.dt_bias, m.conv_w, m.conv_b)
        states = [t.to(DEV) for t in make_states(2, 64, seed=4)]
        if name == "decode_step":
            one = [t[:, 0].contiguous() for t in tok]
            return lambda **kw: ssm.decode_step(*one, *par, *_copies(states, **kw), **kw)
        if name == "decode_tokens":
            few = [t[:, :4].contiguous() for t in tok]
            return lambda **kw: ssm.decode_tokens(*few, *par, *_copies(states, **kw), **kw)
        seg = 64 if name == "prefill_segmented" else None
        return lambda **kw: ssm.prefill(*tok, *par, seg_len=seg, **kw)
    if name in ("ssd_prefill", "ssd_decode_step"):
        s = make_ssd_inputs(2, 300, 4, n_groups=1, seed=5).to(DEV)
        par = (s.conv_w, s.conv_b, s.A, s.D, s.dt_bias, 4, 1)
        if name == "ssd_prefill":
            return lambda **kw: ssm.ssd_prefill(s.xBC, s.z, s.dt, *par, **kw)
        states = [t.to(DEV) for t in make_ssd_states(2, 4, 64, 64, s.channels, seed=6)]
        one = [t[:, 0].contiguous() for t in (s.xBC, s.z, s.dt)]
        return lambda **kw: ssm.ssd_decode_step(*one, *par, *_copies(states, **kw), **kw)
    if name == "out_proj":
        g = torch.Generator(device=DEV).manual_seed(7)
        y, w = (torch.randn(n, 256, generator=g, device=DEV).to(torch.bfloat16) for n in (128, 256))
        return lambda **kw: ssm.out_proj_partial(y, w, **kw)
    parts = [p.to(DEV) for p in make_partials(4, (1000,), seed=8)]
    amax = ssm.q8_block_absmax(parts[0])
    codes, scales = ssm.q8_quantize_shared(parts[0], amax)
    return {"q8_reduce": lambda **kw: ssm.q8_reduce(parts, **kw),
            "q8_block_absmax": lambda **kw: ssm.q8_block_absmax(parts[0], **kw),
            "q8_quantize_shared": lambda **kw: ssm.q8_quantize_shared(parts[0], amax, **kw),
            "q8_sum_dequant": lambda **kw: ssm.q8_sum_dequant([codes, codes], scales, **kw)}[name]


CALLS = ["prefill", "prefill_segmented", "decode_step", "decode_tokens", "ssd_prefill", "ssd_decode_step", "out_proj",
         "q8_reduce", "q8_block_absmax", "q8_quantize_shared", "q8_sum_dequant"]


def _outs(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("name", CALLS)
def test_a_given_stream_takes_its_own_memory(name):
    """Blocks freed on the current stream with reads of them still pending there are not written by the call,
    and its own are not handed out on the current stream before it has run."""
    call = _call(name)
    want = [t.clone() for t in _outs(call())]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    held = [torch.full_like(t, 3) for t in want]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in held]
    places = {t.data_ptr() for t in held}
    held.clear()
    got = _outs(call(stream=side))
    assert not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the call held back on its stream while the current one fills whatever memory is free there
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = _outs(call(stream=side))
    junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in (1 << s for s in range(9, 24)) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 60


def test_given_outputs_are_returned_and_positional_streams_work():
    side = torch.cuda.Stream()
    x = torch.randn(1000, device=DEV).to(torch.bfloat16)
    out = torch.empty(8, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    assert ssm.q8_block_absmax(x, 128, out, side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ssm.q8_block_absmax(x))
