"""The calls around a decode step's mixers as a served model uses them: on a caller's stream, captured into a
graph, on memory that other work still reads, and one after another behind a mixer's block of drafted tokens."""
import numpy as np
import pytest
import torch

from _steps import activations64, check_linear, check_norm, check_probs, verify_exact, weight64
from selective_state_space_prefill_gb300 import binding as ssm
from selective_state_space_prefill_gb300.inputs import make_mixer_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 100_000_000            # cycles: some 50 ms


class Setup:
    def __init__(self, seed=0, m=6, k=1024, n=700, drafts=3):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(m, k, generator=g).to(torch.bfloat16).to(DEV)
        self.res = torch.randn(m, k, generator=g).to(DEV)
        self.W = (torch.randn(n, k, generator=g) / k ** 0.5).to(DEV)
        self.w = ssm.w4_quantize(self.W, 64, True)
        self.logits = (3 * torch.randn(m, n, generator=g)).to(DEV)
        self.t = torch.rand(m, generator=g).to(DEV)
        p = torch.softmax(2 * torch.randn(m, drafts + 1, n, generator=g), -1)
        self.p, self.q = p.to(DEV), torch.softmax(2 * torch.randn(m, drafts, n, generator=g), -1).to(DEV)
        self.draft = torch.randint(0, n, (m, drafts), generator=g, dtype=torch.int32).to(DEV)
        self.u = torch.rand(m, drafts + 1, generator=g).to(DEV)
        # rows split into slices: few rows of x, and many of them against a larger weight
        self.xs = torch.randn(m, 8192, generator=g).to(torch.bfloat16).to(DEV)
        self.ws = ssm.w4_quantize((torch.randn(n, 8192, generator=g) / 90).to(DEV), 128)[:2]
        self.xm = torch.randn(150, 4096, generator=g).to(torch.bfloat16).to(DEV)
        self.wm = ssm.w4_quantize((torch.randn(600, 4096, generator=g) / 64).to(DEV), 64, True)
        torch.cuda.synchronize()

    def norm(self, **kw):
        return ssm.norm_rms(self.x, None, self.res, out_dtype=torch.int8, n_groups=2, **kw)

    def quantize(self, **kw):
        return ssm.w4_quantize(self.W, 64, True, **kw)

    def linear(self, **kw):
        return (ssm.w4_linear(self.x, *self.w, out_dtype=torch.float32, **kw),)

    def slices(self, **kw):
        return (ssm.w4_linear(self.xs, *self.ws, out_dtype=torch.float32, **kw),)

    def tiles(self, **kw):
        return (ssm.w4_linear(self.xm, *self.wm, out_dtype=torch.float32, **kw),)

    def probs(self, **kw):
        return (ssm.spec_probs(self.logits, self.t, **kw),)

    def verify(self, **kw):
        return ssm.spec_verify(self.draft, self.p, self.u, self.q, **kw)


CALLS = ["norm", "quantize", "linear", "slices", "tiles", "probs", "verify"]


def test_the_calls_split_rows_as_meant():
    assert ssm.w4_linear_workspace_bytes(6, 700, 8192, 128) >= 2 * 6 * 700 * 4
    assert ssm.w4_linear_workspace_bytes(150, 600, 4096, 64) >= 192 * 4096 * 2 + 2 * 150 * 600 * 4


@pytest.mark.parametrize("call", CALLS)
def test_a_given_stream_gives_the_same_bits(call):
    s = Setup()
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
    """A block freed on the current stream is not handed to a call on another while the reads are to come."""
    s = Setup()
    want = [t.clone() for t in getattr(s, call)()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = sorted({t.numel() * t.element_size() for t in want})
    held = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    sums = [t.to(torch.int64).sum() for t in held]                 # reads them once the sleep is over
    del held
    got = getattr(s, call)(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert [int(v) for v in sums] == [7 * n for n in sizes for _ in range(2)]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("call", CALLS)
def test_captured_calls_replay_on_new_inputs(call):
    a, b = Setup(0), Setup(1)
    want = [[t.clone() for t in getattr(s, call)()] for s in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        getattr(a, call)()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = getattr(a, call)()
    for turn in range(3):
        if turn == 1:
            for name in ("x", "res", "W", "logits", "t", "p", "q", "draft", "u", "xs", "xm"):
                getattr(a, name).copy_(getattr(b, name))
            for mine, other in zip(a.w + a.ws + a.wm, b.w + b.ws + b.wm):
                mine.copy_(other)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want[min(turn, 1)]):
            assert torch.equal(o, w)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("rows,inner", [(3, 512), (20, 512), (200, 1024)])
def test_each_call_reads_what_the_one_before_wrote(rows, inner, graph):
    """Kernels start before the one before them ends.  Steps in which every call reads what the one before it wrote, and
    writes over what others read, weights among it, with torch's kernels between them, give the bits that they
    give one at a time."""
    vocab, steps = 2600, 12
    g = torch.Generator().manual_seed(rows)
    x0 = torch.randn(rows, inner, generator=g).to(torch.bfloat16).to(DEV)
    W0 = (torch.randn(vocab, inner, generator=g) / inner ** 0.5).to(DEV)
    u = torch.rand(1, rows, generator=g).to(DEV)
    fixed = dict(x=x0.clone(), W=W0.clone(), y=torch.empty_like(x0, dtype=torch.int8), s=torch.empty(rows, 1, device=DEV),
                 l=torch.empty(rows, vocab, device=DEV), p=torch.empty(1, rows, vocab, device=DEV))
    work = torch.empty(max(1, ssm.w4_linear_workspace_bytes(rows, vocab, inner, 64)), dtype=torch.uint8, device=DEV)

    def step(wait):
        f, seen = fixed, []
        w = ssm.w4_quantize(f["W"], 64, True)
        wait()
        ssm.norm_rms(f["x"], out=f["y"], out_scale=f["s"], out_dtype=torch.int8)
        wait()
        ssm.w4_linear(f["y"], *w, x_scale=f["s"], out=f["l"], workspace=work)
        wait()
        ssm.spec_probs(f["l"], out=f["p"][0])
        wait()
        best = f["l"][:rows - 1].argmax(-1).to(torch.int32)[None].contiguous()
        seen += [t.clone() for t in ssm.spec_verify(best, f["p"], u)]
        wait()
        f["W"].mul_(1.0 + f["p"][0, 0, :1])
        nxt = ssm.w4_linear(f["x"], *ssm.w4_quantize(f["W"][:inner], 32), workspace=None)
        wait()
        ssm.norm_rms(nxt, residual=f["x"], out=f["x"], residual_out=False)      # over its own residual
        wait()
        return seen + [f["l"].clone(), f["x"].clone()]

    def run(wait):
        fixed["x"].copy_(x0), fixed["W"].copy_(W0)
        return [t for _ in range(steps) for t in step(wait)]

    want = [t.cpu() for t in run(torch.cuda.synchronize)]
    assert all(torch.isfinite(t.float()).all() for t in want)
    if not graph:
        for _ in range(3):
            got = run(lambda: None)
            torch.cuda.synchronize()
            assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
        return
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.graph(captured, stream=side):
        got = run(lambda: None)
    for _ in range(3):
        captured.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    assert ssm.device_status() == 0


@pytest.mark.parametrize("capture", [False, True])
def test_branches_that_meet(capture):
    """A step forked over two streams and joined: calls behind an event, behind two kernels, a copy and a fill."""
    g = torch.Generator().manual_seed(21)
    m, k, n = 40, 512, 3000
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).to(DEV)
    pinned = torch.empty(m, k, dtype=torch.bfloat16, device=DEV)
    w = [ssm.w4_quantize((torch.randn(n, k, generator=g) / 20).to(DEV), 64, z) for z in (True, False)]
    other = torch.cuda.Stream()

    def run(x):
        main = torch.cuda.current_stream()
        pinned.copy_(x)                                             # a copy, then a call
        h = ssm.norm_rms(pinned)[0]
        other.wait_stream(main)
        with torch.cuda.stream(other):                              # behind an event
            b = ssm.w4_linear(h[:6], *w[1], out_dtype=torch.float32)
            p2 = ssm.spec_probs(b)
        a = ssm.w4_linear(h, *w[0], out_dtype=torch.float32)
        p1 = ssm.spec_probs(a)
        main.wait_stream(other)
        both = ssm.norm_rms(a[:6, :2992], residual=b[:, :2992])[0]  # behind two kernels
        zero = torch.full((6, 2992), 9.0, device=DEV)
        zero.zero_()                                                # a fill, then a call
        z = ssm.norm_rms(zero, residual=both, out_dtype=torch.float32)[0]
        other.wait_stream(main)
        return h, a, b, p1, p2, both, z

    want = [t.clone() for t in run(x)]
    torch.cuda.synchronize()
    check_linear(want[1], want[0], *w[0], None)
    check_linear(want[2], want[0][:6], *w[1], None)
    check_norm(want[5], None, want[1][:6, :2992], None, want[2][:, :2992], 1e-5, 1)
    check_probs(want[4], want[2], None)
    if capture:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run(x)
        for _ in range(3):
            for o in outs:
                o.zero_()
            graph.replay()
    else:
        for _ in range(20):
            outs = run(x)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    assert ssm.device_status() == 0


def test_two_streams_at_once():
    """Calls that overlap share nothing: each gives what it gives alone."""
    s = [Setup(i, m=8, k=4096, n=5000) for i in range(2)]
    want = [[t.clone() for c in CALLS for t in getattr(x, c)()] for x in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i] = [t for c in CALLS for t in getattr(s[i], c)(stream=streams[i])]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


def test_a_block_of_drafted_tokens_from_mixer_to_verification():
    """Blocks of drafted tokens through a mixer's decode, its grouped norm in int8, a 4-bit head, probabilities and
    verification; each step against its definition, and the tokens against the definition on the step's own
    probabilities."""
    batch, drafts, d, vocab = 5, 3, 256, 1001
    inp = make_mixer_inputs(batch, 20 + drafts + 1, d, seed=3, device=DEV)
    pre, block = inp.token_slice(0, 20), inp.token_slice(20, 24)
    args = (inp.A, inp.D, inp.dt_bias, inp.conv_w, inp.conv_b)
    out, conv, state = ssm.prefill(pre.x, pre.z, pre.dt, pre.B, pre.C, *args)
    y = ssm.decode_tokens(block.x, block.z, block.dt, block.B, block.C, *args, conv, state)
    rows = y.reshape(batch * (drafts + 1), d)
    g = torch.Generator().manual_seed(9)
    weight = (1 + 0.1 * torch.randn(d, generator=g)).to(DEV)
    res = torch.randn(rows.shape, generator=g).to(torch.bfloat16).to(DEV)
    head = (0.3 * torch.randn(vocab, d, generator=g)).to(DEV)
    codes, scales, zeros = ssm.w4_quantize(head, 32, True)
    h, stream, hs = ssm.norm_rms(rows, weight, res, n_groups=4, out_dtype=torch.int8)
    check_norm(h, hs, rows, weight, res, 1e-5, 4)
    logits = ssm.w4_linear(h, codes, scales, zeros, x_scale=hs, out_dtype=torch.float32)
    check_linear(logits, h, codes, scales, zeros, hs)
    assert np.isfinite(activations64(h, hs) @ weight64(codes, scales, zeros).T).all()
    temperature = torch.tensor([0.0, 0.7, 1.0, 1.3], device=DEV).repeat(batch)
    p = ssm.spec_probs(logits, temperature)
    check_probs(p, logits, temperature)
    p = p.view(batch, drafts + 1, vocab)
    # drafts from probabilities near the target's; request 4 has two of them only
    q = ssm.spec_probs(logits.to(torch.bfloat16).view(batch, drafts + 1, vocab)[:, :drafts].reshape(-1, vocab),
                       temperature.view(batch, -1)[:, :drafts].clamp(min=0.8).reshape(-1)).view(batch, drafts, vocab)
    draft = torch.multinomial(q.reshape(-1, vocab).cpu(), 1, generator=g).view(batch, drafts).to(torch.int32)
    u, count = torch.rand(batch, drafts + 1, generator=g), torch.tensor([3, 3, 3, 3, 2], dtype=torch.int32)
    for qs in (q, None):
        tokens, kept = ssm.spec_verify(draft.to(DEV), p, u.to(DEV), qs, count.to(DEV))
        want = verify_exact(draft, p, u, qs, count)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])
    # greedy drafts of the target itself are kept, and the token after them is its own
    best = p.argmax(-1).to(torch.int32)
    one = ssm.spec_probs(logits, torch.zeros_like(temperature)).view(batch, drafts + 1, vocab)
    tokens, kept = ssm.spec_verify(best[:, :drafts].contiguous(), one, u.to(DEV))
    assert (kept == drafts).all() and torch.equal(tokens, best)
    assert ssm.device_status() == 0
