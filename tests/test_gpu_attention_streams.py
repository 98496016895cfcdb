"""Attention calls on a stream given by the caller: the same bits as on the current one, and memory made for
them that no pending work of another stream still uses."""
import pytest
import torch

from _attn import cu, heads
from selective_state_space_prefill_gb300 import binding as ssm
from selective_state_space_prefill_gb300.rope import rope_frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 100_000_000            # cycles: some 50 ms


class Setup:
    """700 tokens of one request, cached; every call with outputs made by the binding."""

    def __init__(self, i8=True, n=700, H=8, Hk=2, D=64, page=64, max_len=9000):
        g = torch.Generator().manual_seed(5)
        self.n, self.H, self.Hk, self.D, self.max_len = n, H, Hk, D, max_len
        self.q, self.k, self.v = (heads(g, n, h, D).to(DEV) for h in (H, Hk, Hk))
        self.cos, self.sin = ssm.attn_rope_table(rope_frequencies(D)[0], n)
        pages = -(-n // page)
        self.kc, self.vc = (torch.zeros(pages, Hk, page, D, dtype=torch.int8 if i8 else torch.bfloat16, device=DEV) for _ in range(2))
        self.ks, self.vs = ((torch.zeros(pages, Hk, page, device=DEV) for _ in range(2)) if i8 else (None, None))
        self.table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
        self.pos = torch.arange(n, dtype=torch.int32, device=DEV)
        self.cu, self.lens = cu([n]).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
        self.append()
        torch.cuda.synchronize()

    def append(self, **kw):
        return ssm.attn_append(self.q, self.k, self.v, self.pos, self.cos, self.sin, self.kc, self.vc, self.pos, self.ks,
                               self.vs, k_out=True, **kw)

    def read(self, **kw):
        return ssm.attn_cache_read(self.kc, self.vc, self.table, self.cu, self.n, self.ks, self.vs, **kw)

    def prefill(self, **kw):
        return ssm.attn_prefill(self.q, self.k, self.v, self.cu, self.cu, self.n, lse=True, **kw)

    def decode(self, **kw):
        return ssm.attn_decode_step(self.q[:1], self.kc, self.vc, self.table, self.lens, self.max_len, self.ks, self.vs,
                                    lse=True, **kw)

    def rope(self, **kw):
        return ssm.attn_rope_table(rope_frequencies(self.D)[0], self.n, **kw)


CALLS = ["append", "read", "prefill", "decode", "rope"]


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("call", CALLS)
def test_a_given_stream_gives_the_same_bits(call, i8):
    s = Setup(i8)
    assert ssm.attn_decode_workspace_bytes(1, s.H, s.Hk, s.D, s.max_len) > 0       # decode: pieces, workspace and join
    want = getattr(s, call)()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = getattr(s, call)(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.cuda.current_stream() != side and ssm.device_status() == 0


@pytest.mark.parametrize("call", CALLS)
def test_memory_still_read_on_the_current_stream_is_not_overwritten(call):
    """A block freed on the current stream may be handed out again there, as later work follows the reads
    that are still pending.  A call on another stream follows nothing of that and takes other memory."""
    s = Setup()
    shapes = [(t.shape, t.dtype) for t in getattr(s, call)()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()
    held = [torch.full(shape, 3, dtype=dtype, device=DEV) for shape, dtype in shapes]
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in held]
    places = {t.data_ptr() for t in held}
    held.clear()
    got = getattr(s, call)(stream=side)
    assert not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies)


@pytest.mark.parametrize("call", CALLS)
def test_an_output_still_read_on_the_current_stream_is_not_handed_out_again(call):
    """The other way: an output made on the given stream and dropped while the current one still reads it."""
    s = Setup()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = [t.clone() for t in getattr(s, call)()]
    torch.cuda.synchronize()
    first = getattr(s, call)(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in first]
    places = {t.data_ptr() for t in first}
    del first
    with torch.cuda.stream(side):
        again = [torch.full_like(t, 7) for t in want]
    assert not places & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


def test_what_is_not_a_stream_is_refused():
    s = Setup()
    with pytest.raises((TypeError, AttributeError)):
        s.read(stream="side")
    with pytest.raises(TypeError):
        s.read(stream=type("S", (), {"cuda_stream": "0"})())
