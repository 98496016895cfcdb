"""The forms that the attention calls choose between by their sizes, each run and compared with 64 bits:
decode's one piece, cluster, and pieces with either join, at both padded widths and both head groups;
strided queries and page tables; prompts whose keys a cluster shares at padded widths; weights as bf16
pairs; long prompts; the two-kernel decode in a graph."""
import numpy as np
import pytest
import torch

from _attn import W_DECODE, W_PREFILL, attend64, check_attention, cu, heads, paged, to64
from selective_state_space_prefill_gb300 import binding as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cat(refs):
    return tuple(np.concatenate([r[i] for r in refs]) for i in range(4))


def _to_dev(c):
    return {n: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}


def _decode(q, c, lens, max_len, table=None, **kw):
    c = _to_dev(c)
    return ssm.attn_decode_step(q, c["k_cache"], c["v_cache"], c["table"] if table is None else table,
                                torch.tensor(lens, dtype=torch.int32, device=DEV), max_len, c["k_scale"], c["v_scale"], **kw)


def _decode_ref(q, c, lens, scale):
    refs, at = [], 0
    for b, n in enumerate(lens):
        refs.append(attend64(to64(q[b:b + 1]), c["k64"][at:at + n], c["v64"][at:at + n], scale, n - 1))
        at += n
    return _cat(refs)


def _pair_weight(keys):
    """Weights as bf16 pairs: the high part keeps 8 bits of w, the low part 8 bits of a rest below 2^-7 w, so
    2^-9 x 2^-7 of w is lost; beside it the fp32 accumulation of 2 products a 16 keys, 2^-23 each."""
    return 2.0 ** -16 + (keys / 8 + 8) * 2.0 ** -23


SHORT = [2048, 1, 192, 193, 0, 700, 1500, 191, 384, 65]
# lens, max_len, kv heads; a join takes a warp a head for up to 16 pieces, a block for more
FORMS = {
    "one piece": ([64, 1, 0, 33], 64, 2),
    "one piece, many requests": ([(13 * i) % 101 for i in range(300)], 100, 1),
    "cluster": ([900, 65, 64, 0], 1024, 2),
    "warp join": (SHORT, 2048, 8),
    "block join": ([5000, 4097, 3], 5000, 2),
}


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("D,group", [(64, 2), (64, 12), (96, 1), (128, 2), (128, 12)])
@pytest.mark.parametrize("form", FORMS)
def test_decode_forms(form, D, group, i8):
    lens, max_len, Hk = FORMS[form]
    H = Hk * group
    g = torch.Generator().manual_seed(sum(lens) + D + group)
    T = sum(lens)
    c = paged(torch.randn(T, Hk, D, generator=g), torch.randn(T, Hk, D, generator=g), lens, 64, i8)
    q = heads(g, len(lens), H, D, 1.5).to(DEV)
    need = ssm.attn_decode_workspace_bytes(len(lens), H, Hk, D, max_len)
    # pieces x (outputs, maximum, sum) of fp32
    pieces = need // (len(lens) * H * ((64 if D <= 64 else 128) + 2) * 4)
    assert {"one piece": need == 0, "one piece, many requests": need == 0, "cluster": need == 0,
            "warp join": 1 < pieces <= 16, "block join": pieces > 16}[form], pieces
    out, lse = _decode(q, c, lens, max_len, out_dtype=torch.float32, lse=True)
    ref = _decode_ref(q, c, lens, D ** -0.5)
    check_attention(out, lse, ref, D, torch.float32, W_DECODE, form)
    empty = np.isneginf(ref[1])
    assert (to64(out)[empty] == 0).all() and ssm.device_status() == 0
    if not i8:
        check_attention(out, lse, ref, D, torch.float32, _pair_weight(max(lens)), form + ", weights as pairs")


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("D,max_len", [(64, 700), (128, 700), (80, 5000)])
def test_decode_strided_query_and_table(D, max_len, i8):
    """The query as a slice of a fused projection's rows, and the table as columns of a wider one: the
    bits of contiguous ones."""
    lens, H, Hk = [700, 17], 6, 2
    g = torch.Generator().manual_seed(D)
    c = paged(torch.randn(717, Hk, D, generator=g), torch.randn(717, Hk, D, generator=g), lens, 16, i8)
    qkv = heads(g, 2, H + 2 * Hk, D).to(DEV)
    want, _ = _decode(qkv[:, :H].contiguous(), c, lens, max_len)
    wide = torch.full((2, c["table"].shape[1] + 7), -9, dtype=torch.int32, device=DEV)
    wide[:, 3:-4] = c["table"].to(DEV)
    got, _ = _decode(qkv[:, :H], c, lens, max_len, table=wide[:, 3:-4])
    assert torch.equal(got, want) and ssm.device_status() == 0


@pytest.mark.parametrize("i8", [True, False])
def test_decode_pieces_and_join_in_a_graph(i8):
    """Both kernels of a long call captured (the join's launch overlaps the pieces'): replays follow lens and
    queries written in between, and give the bits of direct calls."""
    H, Hk, D, n, max_len = 8, 2, 128, 3000, 6000
    g = torch.Generator().manual_seed(9)
    c = _to_dev(paged(torch.randn(n, Hk, D, generator=g), torch.randn(n, Hk, D, generator=g), [n], 64, i8))
    need = ssm.attn_decode_workspace_bytes(1, H, Hk, D, max_len)
    assert need > 0
    q, lens = torch.zeros(1, H, D, dtype=torch.bfloat16, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty(1, H, D, device=DEV), torch.empty(1, H, device=DEV)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def step():
        ssm.attn_decode_step(q, c["k_cache"], c["v_cache"], c["table"], lens, max_len, c["k_scale"], c["v_scale"], out=out,
                             lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for m in (n, 1, 0, 2047):
        q.copy_(heads(g, 1, H, D))
        lens.fill_(m)
        step()
        want = out.clone(), lse.clone()
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        check_attention(out, lse, attend64(to64(q), c["k64"][:m], c["v64"][:m], D ** -0.5, m - 1), D, torch.float32, W_DECODE)


def _prefill_ref(q, k, v, ql, kl, scale):
    refs, aq, ak = [], 0, 0
    for n, m in zip(ql, kl):
        refs.append(attend64(to64(q[aq:aq + n]), to64(k[ak:ak + m]), to64(v[ak:ak + m]), scale, m - n))
        aq, ak = aq + n, ak + m
    return _cat(refs)


@pytest.mark.parametrize("ql,kl,H,Hk,D", [
    ([3], [4400], 2, 1, 80), ([130], [5000], 2, 2, 112), ([1, 2], [4500, 4300], 4, 2, 96), ([300], [4100], 2, 1, 96),
    ([90], [4097], 4, 1, 48),
])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_prefill_shared_keys_at_padded_widths(ql, kl, H, Hk, D, out_dtype):
    """Keys shared by a cluster where head_dim is less than the width of a part; the output lies in a wider
    buffer, and nothing is written beside it."""
    g = torch.Generator().manual_seed(sum(kl) + D)
    q = heads(g, sum(ql), H, D, 1.5)
    k, v = heads(g, sum(kl), Hk, D), heads(g, sum(kl), Hk, D)
    wide = torch.full((sum(ql), H, D + 16), 7.0, dtype=out_dtype, device=DEV)
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu(ql).to(DEV), cu(kl).to(DEV), max(ql),
                                out=wide[..., 8:8 + D], lse=True)
    check_attention(out, lse, _prefill_ref(q, k, v, ql, kl, D ** -0.5), D, out_dtype, W_PREFILL, f"{ql} {kl}")
    assert bool((wide[..., :8] == 7.0).all()) and bool((wide[..., 8 + D:] == 7.0).all())


@pytest.mark.parametrize("rows,keys,H,Hk,D", [
    (1, 2, 4, 1, 64), (30, 40, 2, 2, 128), (64, 700, 4, 1, 80), (9, 4400, 8, 2, 128), (2, 5000, 3, 1, 64),
])
def test_prefill_few_rows_keep_16_bits(rows, keys, H, Hk, D):
    """256 rows x heads or fewer: the weights are bf16 pairs, whether or not the keys are shared out; sharp
    softmaxes, so that few weights matter and their rounding does not average out."""
    assert rows * H <= 256
    g = torch.Generator().manual_seed(keys)
    q, k, v = heads(g, rows, H, D, 3.0), heads(g, keys, Hk, D), heads(g, keys, Hk, D)
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu([rows]).to(DEV), cu([keys]).to(DEV), rows,
                                out_dtype=torch.float32, lse=True)
    check_attention(out, lse, _prefill_ref(q, k, v, [rows], [keys], D ** -0.5), D, torch.float32, _pair_weight(keys))


def test_prefill_mixed_batch():
    """One long chunk beside single rows over contexts of all lengths."""
    ql, kl, H, Hk, D = [600] + [1] * 9 + [0, 3], [900, 1, 127, 128, 129, 2000, 1500, 255, 256, 257, 40, 3], 4, 2, 128
    g = torch.Generator().manual_seed(8)
    q, k, v = heads(g, sum(ql), H, D), heads(g, sum(kl), Hk, D), heads(g, sum(kl), Hk, D)
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu(ql).to(DEV), cu(kl).to(DEV), max(ql),
                                out_dtype=torch.float32, lse=True)
    check_attention(out, lse, _prefill_ref(q, k, v, ql, kl, D ** -0.5), D, torch.float32, W_PREFILL)


@pytest.mark.parametrize("n,context,H,Hk,D", [(6001, 0, 4, 2, 128), (5000, 0, 2, 2, 64), (2500, 7001, 4, 1, 96)])
def test_prefill_long_prompt_at_sampled_rows(n, context, H, Hk, D):
    """Long prompts, and a chunk over a long context, at rows around tile and block edges and at random ones."""
    g = torch.Generator().manual_seed(n)
    q, k, v = heads(g, n, H, D, 1.5), heads(g, n + context, Hk, D), heads(g, n + context, Hk, D)
    out, lse = ssm.attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu([n]).to(DEV), cu([n + context]).to(DEV), n,
                                out_dtype=torch.float32, lse=True)
    rows = sorted({0, 1, 127, 128, 255, 256, 257, 1023, 2047, 2048, n - 129, n - 128, n - 2, n - 1,
                   *torch.randint(0, n, (20,), generator=g).tolist()})
    k64, v64 = to64(k), to64(v)
    ref = _cat([attend64(to64(q[i:i + 1]), k64, v64, D ** -0.5, i + context) for i in rows])
    check_attention(out[rows], lse[rows], ref, D, torch.float32, W_PREFILL)
