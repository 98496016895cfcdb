"""attn_prefill and attn_decode_step against the 64-bit softmax.

The bounds (tests/_attn.py) are those of the documented arithmetic: scores from fp32 sums, weights
rounded for the second product, fp32 accumulation, one rounding of the output.
"""
import numpy as np
import pytest
import torch

from _attn import W_DECODE, W_PREFILL, attend64, check_attention, cu, heads, out_bound, paged, to64
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cat(refs):
    return tuple(np.concatenate([r[i] for r in refs]) for i in range(4))


def _prefill_ref(q, k, v, ql, kl, scale):
    refs, aq, ak = [], 0, 0
    for n, m in zip(ql, kl):
        refs.append(attend64(to64(q[aq:aq + n]), to64(k[ak:ak + m]), to64(v[ak:ak + m]), scale, m - n))
        aq, ak = aq + n, ak + m
    return _cat(refs)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ql,kl,H,Hk,D", [
    ([1], [1], 1, 1, 16), ([77], [77], 6, 6, 64), ([128], [128], 2, 1, 128), ([129, 127], [129, 127], 4, 2, 64),
    ([5, 0, 300, 1, 64], [5, 0, 300, 1, 64], 6, 2, 80), ([130, 40], [391, 640], 7, 1, 128),
    ([200, 3, 50, 9], [60, 3, 0, 140], 4, 4, 96), ([1, 1, 1], [257, 1, 128], 12, 3, 112), ([513], [513], 3, 1, 32),
    ([384, 256, 255, 257], [384, 256, 511, 1025], 2, 2, 128),
])
def test_prefill(ql, kl, H, Hk, D, out_dtype):
    g = torch.Generator().manual_seed(sum(ql) + D)
    q = heads(g, sum(ql), H, D, 1.5)
    kv = heads(g, sum(kl), 2 * Hk, D)
    k, v = kv[:, :Hk], kv[:, Hk:]
    out, lse = ssm.attn_prefill(q.to(DEV), kv.to(DEV)[:, :Hk], kv.to(DEV)[:, Hk:], cu(ql).to(DEV), cu(kl).to(DEV),
                                max(ql), out_dtype=out_dtype, lse=True)
    torch.cuda.synchronize()
    ref = _prefill_ref(q, k, v, ql, kl, D ** -0.5)
    check_attention(out, lse, ref, D, out_dtype, W_PREFILL, f"prefill {ql} {kl}")
    empty = np.isneginf(ref[1])
    assert (to64(out)[empty] == 0).all()
    assert ssm.device_status() == 0


@pytest.mark.parametrize("scale,gain", [(1.0, 3.0), (0.02, 1.0), (1e-3, 0.1)])
def test_prefill_score_ranges(scale, gain):
    """Sharp softmaxes (scores of hundreds, whose maximum moves from tile to tile) and flat ones."""
    g = torch.Generator().manual_seed(7)
    n, D = 400, 64
    q, k, v = heads(g, n, 2, D, gain), heads(g, n, 1, D, gain), heads(g, n, 1, D)
    k *= torch.linspace(0.2, 1.5, n)[:, None, None].to(torch.bfloat16)      # later keys score higher
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu([n]).to(DEV), cu([n]).to(DEV), n, scale=scale,
                                out_dtype=torch.float32, lse=True)
    check_attention(out, lse, _prefill_ref(q, k, v, [n], [n], scale), D, torch.float32, W_PREFILL)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_layouts(D):
    """[heads][tokens] order, rows inside wider buffers, an output inside a wider one: the same values
    as contiguous tensors, and nothing written beside them."""
    g = torch.Generator().manual_seed(1)
    n, H, Hk = 200, 4, 2
    q, k, v = heads(g, n, H, D).to(DEV), heads(g, n, Hk, D).to(DEV), heads(g, n, Hk, D).to(DEV)
    c = cu([150, 50]).to(DEV)
    ref, _ = ssm.attn_prefill(q, k, v, c, c, 150)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    kw = torch.full((n, Hk, D + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    kw[..., 8:8 + D] = k
    wide = torch.full((n, H + 2, D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    out, _ = ssm.attn_prefill(qt, kw[..., 8:8 + D], v, c, c, 150, out=wide[:, 1:-1, :D])
    assert torch.equal(out, ref)
    wide[:, 1:-1, :D] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,n", [(64, 300), (128, 300), (128, 90), (128, 1500)])
def test_prefill_unseen_values_do_not_leak(D, n, bad):
    """Non-finite keys and values at a token reach only the rows that see it; the neighbours in the
    packing are untouched."""
    g = torch.Generator().manual_seed(2)
    lens = [60, n, 70]
    at = 60 + n // 2 + 3
    q, k, v = heads(g, sum(lens), 2, D), heads(g, sum(lens), 1, D), heads(g, sum(lens), 1, D)
    c = cu(lens).to(DEV)
    clean, cl = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), c, c, n, lse=True, out_dtype=torch.float32)
    # one value: its column in the rows that see it, nothing else
    v2 = v.clone()
    v2[at, 0, 5] = bad
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v2.to(DEV), c, c, n, lse=True, out_dtype=torch.float32)
    sees = torch.zeros(sum(lens), dtype=torch.bool)
    sees[at:60 + n] = True
    hit = out[sees.to(DEV)][:, :, 5]
    assert bool(hit.isnan().all()) if bad != bad else bool((hit == bad).all())
    rest = out.clone()
    rest[sees.to(DEV), :, 5] = clean[sees.to(DEV), :, 5]
    assert torch.equal(rest, clean) and torch.equal(lse, cl)
    # a whole key and value row of it: the rows before, and the other sequences, keep their bits
    k2 = k.clone()
    k2[at], v2[at] = bad, bad
    out, _ = ssm.attn_prefill(q.to(DEV), k2.to(DEV), v2.to(DEV), c, c, n, out_dtype=torch.float32)
    assert torch.equal(out[~sees.to(DEV)], clean[~sees.to(DEV)])


@pytest.mark.parametrize("ql,kl,H,Hk,D", [
    ([1], [5000], 8, 2, 128), ([8, 3, 1], [2200, 0, 999], 4, 1, 64), ([257, 300], [2000, 1700], 3, 3, 80),
    ([700], [900], 2, 1, 128), ([40], [3001], 12, 4, 64), ([1, 0, 2], [1, 4000, 130], 5, 5, 96),
    ([70, 0, 129], [2500, 2600, 2049], 3, 1, 128), ([2, 2], [4200, 4097], 6, 2, 64),
])
def test_prefill_few_rows_over_many_keys(ql, kl, H, Hk, D):
    """Items too few for the GPU: their keys are shared out between the CTAs of a cluster."""
    g = torch.Generator().manual_seed(sum(kl) + H)
    q = heads(g, sum(ql), H, D, 1.5)
    k, v = heads(g, sum(kl), Hk, D), heads(g, sum(kl), Hk, D)
    for out_dtype in (torch.bfloat16, torch.float32):
        out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu(ql).to(DEV), cu(kl).to(DEV), max(ql),
                                    out_dtype=out_dtype, lse=True)
        check_attention(out, lse, _prefill_ref(q, k, v, ql, kl, D ** -0.5), D, out_dtype, W_PREFILL, f"{ql} {kl}")
    assert ssm.device_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefill_split_keys_do_not_leak(bad):
    """The same where a cluster shares the keys: a bad value in the last CTA's share reaches only the
    rows that see it."""
    g = torch.Generator().manual_seed(6)
    lq, lk, D = 300, 5000, 64
    q, k, v = heads(g, lq, 3, D).to(DEV), heads(g, lk, 1, D).to(DEV), heads(g, lk, 1, D).to(DEV)
    cq, ck = cu([lq]).to(DEV), cu([lk]).to(DEV)
    clean, cl = ssm.attn_prefill(q, k, v, cq, ck, lq, lse=True, out_dtype=torch.float32)
    v2 = v.clone()
    v2[4850, 0, 7] = bad                        # row i sees keys up to i + 4700
    out, lse = ssm.attn_prefill(q, k, v2, cq, ck, lq, lse=True, out_dtype=torch.float32)
    hit = out[150:, :, 7]
    assert bool(hit.isnan().all()) if bad != bad else bool((hit == bad).all())
    out[150:, :, 7] = clean[150:, :, 7]
    assert torch.equal(out, clean) and torch.equal(lse, cl)


def test_prefill_max_q_and_empty_calls():
    g = torch.Generator().manual_seed(3)
    q, k, v = heads(g, 40, 2, 64).to(DEV), heads(g, 40, 2, 64).to(DEV), heads(g, 40, 2, 64).to(DEV)
    c = cu([40]).to(DEV)
    ref, _ = ssm.attn_prefill(q, k, v, c, c, 40)
    big, _ = ssm.attn_prefill(q, k, v, c, c, 5000)              # a loose bound is only a bound
    assert torch.equal(big, ref)
    none, _ = ssm.attn_prefill(q[:0], k, v, cu([0]).to(DEV), c, 0)
    assert none.shape == (0, 2, 64)
    out, lse = ssm.attn_prefill(q, k[:0], v[:0], c, cu([0]).to(DEV), 40, lse=True)      # no keys at all
    assert bool((out == 0).all()) and bool(lse.isneginf().all())


def test_prefill_chunks_equal_the_whole_prompt():
    """A prompt in three chunks, each over the keys so far, against the 64-bit whole."""
    g = torch.Generator().manual_seed(4)
    n, H, Hk, D = 500, 4, 2, 128
    q, k, v = heads(g, n, H, D), heads(g, n, Hk, D), heads(g, n, Hk, D)
    ref = _prefill_ref(q, k, v, [n], [n], D ** -0.5)
    outs, lses = [], []
    for a, e in ((0, 130), (130, 431), (431, 500)):
        o, l = ssm.attn_prefill(q[a:e].to(DEV), k[:e].to(DEV), v[:e].to(DEV), cu([e - a]).to(DEV), cu([e]).to(DEV),
                                e - a, lse=True)
        outs.append(o)
        lses.append(l)
    check_attention(torch.cat(outs), torch.cat(lses), ref, D, torch.bfloat16, W_PREFILL)


# ------------------------------------------------------------------------------ decode
def _decode_ref(q, c, lens, scale):
    refs, at = [], 0
    for b, n in enumerate(lens):
        refs.append(attend64(to64(q[b:b + 1]), c["k64"][at:at + n], c["v64"][at:at + n], scale, n - 1))
        at += n
    return _cat(refs)


def _decode(q, c, lens, max_len=None, **kw):
    dev = {n: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    return ssm.attn_decode_step(q.to(DEV), dev["k_cache"], dev["v_cache"], dev["table"],
                                torch.tensor(lens, dtype=torch.int32, device=DEV), max_len or max(max(lens), 1),
                                dev["k_scale"], dev["v_scale"], **kw)


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,H,Hk,D,page", [
    ([1], 1, 1, 16, 16), ([0, 1, 15, 16, 17], 4, 2, 64, 16), ([700], 32, 8, 128, 64), ([33, 250, 0, 64], 7, 1, 128, 48),
    ([1100, 5], 12, 1, 80, 256), ([129, 640, 31], 24, 24, 64, 32), ([90], 40, 2, 112, 16), ([513], 17, 1, 96, 80),
])
def test_decode(lens, H, Hk, D, page, i8, out_dtype):
    g = torch.Generator().manual_seed(sum(lens) + H)
    T = sum(lens)
    c = paged(torch.randn(T, Hk, D, generator=g), torch.randn(T, Hk, D, generator=g), lens, page, i8)
    q = heads(g, len(lens), H, D, 1.5)
    out, lse = _decode(q, c, lens, out_dtype=out_dtype, lse=True)
    ref = _decode_ref(q, c, lens, D ** -0.5)
    check_attention(out, lse, ref, D, out_dtype, W_DECODE, f"decode {lens}")
    assert (to64(out)[np.isneginf(ref[1])] == 0).all()
    # a loose bound of the lengths only changes how the work is cut
    loose, _ = _decode(q, c, lens, max_len=(max(lens) + 1) * 9, out_dtype=out_dtype)
    check_attention(loose, None, ref, D, out_dtype, W_DECODE, f"decode {lens}, loose bound")
    assert ssm.device_status() == 0


@pytest.mark.parametrize("i8", [True, False])
def test_decode_long_and_sharp(i8):
    """One long sequence cut into many pieces; keys that stand out far from the end; rows whose scales
    differ by 2^40."""
    g = torch.Generator().manual_seed(11)
    n, H, Hk, D = 9001, 8, 2, 64
    k, v = torch.randn(n, Hk, D, generator=g), torch.randn(n, Hk, D, generator=g)
    k[100] *= 6
    k[5000] *= 9
    v[::7] *= 2.0 ** -20
    v[3::7] *= 2.0 ** 20
    c = paged(k, v, [n], 64, i8)
    q = heads(g, 1, H, D, 2.0)
    out, lse = _decode(q, c, [n], out_dtype=torch.float32, lse=True)
    check_attention(out, lse, _decode_ref(q, c, [n], D ** -0.5), D, torch.float32, W_DECODE)


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("gain", [2.0 ** -60, 2.0 ** 40])
def test_decode_query_and_value_ranges(i8, gain):
    """Queries, keys and values far from 1: nothing overflows a narrower type on the way."""
    g = torch.Generator().manual_seed(12)
    n, D = 200, 128
    c = paged(torch.randn(n, 1, D, generator=g) / gain, torch.randn(n, 1, D, generator=g) * gain, [n], 16, i8)
    q = heads(g, 1, 4, D, gain)
    out, lse = _decode(q, c, [n], out_dtype=torch.float32, lse=True)
    check_attention(out, lse, _decode_ref(q, c, [n], D ** -0.5), D, torch.float32, W_DECODE)


@pytest.mark.parametrize("i8", [True, False])
def test_decode_reports_bad_pages_and_lengths(i8):
    g = torch.Generator().manual_seed(13)
    lens = [40, 40]
    c = paged(torch.randn(80, 1, 64, generator=g), torch.randn(80, 1, 64, generator=g), lens, 16, i8)
    q = heads(g, 2, 2, 64)
    ssm.device_status(clear=True)
    good, _ = _decode(q, c, lens, out_dtype=torch.float32)
    assert ssm.device_status(clear=True) == 0
    c["table"][0, 2] = -5                       # request 0 loses its last page's keys; request 1 keeps its bits
    out, lse = _decode(q, c, lens, out_dtype=torch.float32, lse=True)
    assert ssm.device_status(clear=True) == ssm.DEV_BAD_INDEX
    ref = attend64(to64(q[:1]), c["k64"][:32], c["v64"][:32], 64 ** -0.5, 31)
    check_attention(out[:1], lse[:1], ref, 64, torch.float32, W_DECODE)
    assert torch.equal(out[1], good[1])
    cut, _ = _decode(q, c, [-3, 4000], max_len=40, out_dtype=torch.float32)
    assert ssm.device_status(clear=True) == ssm.DEV_BAD_INDEX
    assert bool((cut[0] == 0).all())
    check_attention(cut[1:], None, attend64(to64(q[1:]), c["k64"][40:], c["v64"][40:], 64 ** -0.5, 39), 64, torch.float32, W_DECODE)


@pytest.mark.parametrize("i8", [True, False])
def test_append_read_prefill_decode_agree(i8):
    """A prompt appended, attended over and continued token by token equals the whole sequence attended
    at once, on a side stream and replayed from a CUDA graph."""
    g = torch.Generator().manual_seed(21)
    n, extra, H, Hk, D, page = 150, 3, 8, 2, 64, 16
    N = n + extra
    qkv = heads(g, N, H + 2 * Hk, D).to(DEV)
    from selective_state_space_prefill_gb300.rope import rope_frequencies
    cos, sin = ssm.attn_rope_table(rope_frequencies(D)[0], N)
    pages = -(-N // page)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].to(DEV)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    slots = (table[0, pos.long() // page] * page + pos % page).to(torch.int32)
    shape = (pages, Hk, page, D)
    kc, vc = (torch.zeros(shape, dtype=torch.int8 if i8 else torch.bfloat16, device=DEV) for _ in range(2))
    ks, vs = ((torch.zeros(shape[:3], device=DEV) for _ in range(2)) if i8 else (None, None))

    def append(a, e):
        x = qkv[a:e]
        return ssm.attn_append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], pos[a:e], cos, sin, kc, vc, slots[a:e], ks, vs)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q = [append(0, n)]
        k, v = ssm.attn_cache_read(kc, vc, table, cu([n]).to(DEV), n, ks, vs)
        outs = [ssm.attn_prefill(q[0], k, v, cu([n]).to(DEV), cu([n]).to(DEV), n)[0]]
        for t in range(n, N):
            q.append(append(t, t + 1))
            lens = torch.tensor([t + 1], dtype=torch.int32, device=DEV)
            outs.append(ssm.attn_decode_step(q[-1], kc, vc, table, lens, N, ks, vs)[0])
    side.synchronize()
    k, v = ssm.attn_cache_read(kc, vc, table, cu([N]).to(DEV), N, ks, vs, out_dtype=torch.float32)
    ref = attend64(to64(torch.cat(q)), to64(k), to64(v), D ** -0.5, 0)
    out, _ = torch.cat(outs), None
    # the prompt's rows attend over keys and values rounded to bf16 on reading an int8 cache
    extra_v = W_PREFILL * ref[2] + W_PREFILL * 2.1 * ref[3][..., None] * ref[2]
    bound = out_bound(ref[0], ref[2], ref[3], D, torch.bfloat16, W_PREFILL) + 1.1 * extra_v
    assert (np.abs(to64(out) - ref[0]) <= bound).all()
    # the decode step captured in a graph: replays give the same bits
    lens = torch.tensor([N], dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, ssm.attn_decode_workspace_bytes(1, H, Hk, D, N)), dtype=torch.uint8, device=DEV)
    buf = torch.empty_like(outs[-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.attn_decode_step(q[-1], kc, vc, table, lens, N, ks, vs, out=buf, workspace=ws)
    for _ in range(2):
        buf.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, outs[-1])


def test_decode_workspace_is_kept_inside():
    """Guard bytes around the workspace and the output stay as they were."""
    g = torch.Generator().manual_seed(31)
    lens, H, Hk, D = [3000, 700], 16, 2, 128
    c = paged(torch.randn(3700, Hk, D, generator=g), torch.randn(3700, Hk, D, generator=g), lens, 64, True)
    q = heads(g, 2, H, D)
    need = ssm.attn_decode_workspace_bytes(2, H, Hk, D, 3000)
    buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    obuf = torch.full((2, H + 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
    out, _ = _decode(q, c, lens, workspace=buf[256:256 + need] if need else buf[256:257], out=obuf[:, 1:-1])
    torch.cuda.synchronize()
    assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + need:] == 0xA5).all())
    assert bool((obuf[:, 0] == 7.0).all()) and bool((obuf[:, -1] == 7.0).all())
    check_attention(out, None, _decode_ref(q, c, lens, D ** -0.5), D, torch.bfloat16, W_DECODE)


@pytest.mark.parametrize("rows,keys,H,Hk", [(700, 700, 8, 2), (8, 4008, 8, 2)])
def test_prefill_gives_the_same_bits_again(rows, keys, H, Hk):
    """No atomics and a fixed order of the joins: calls on the same inputs agree bit by bit, whether one
    CTA takes an item's keys or a cluster shares them."""
    g = torch.Generator().manual_seed(rows)
    q, k, v = (heads(g, n, h, 128).to(DEV) for n, h in ((rows, H), (keys, Hk), (keys, Hk)))
    first, *rest = [ssm.attn_prefill(q, k, v, cu([rows]).to(DEV), cu([keys]).to(DEV), rows, lse=True) for _ in range(4)]
    for out, lse in rest:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("lens", [[900, 33], [9000, 1, 4097]])
def test_decode_gives_the_same_bits_again(lens, i8):
    g = torch.Generator().manual_seed(sum(lens))
    c = paged(torch.randn(sum(lens), 2, 128, generator=g), torch.randn(sum(lens), 2, 128, generator=g), lens, 64, i8)
    q = heads(g, len(lens), 16, 128)
    first, *rest = [_decode(q, c, lens, lse=True) for _ in range(4)]
    for out, lse in rest:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
