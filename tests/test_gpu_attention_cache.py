"""attn_rope_table, attn_append and attn_cache_read against plain evaluations.

Rotated values: within three fp32 roundings of the 64-bit rotation (plus half a bf16 ulp); int8 codes
and scales and bf16 rows bit for bit those of an IEEE fp32 evaluation of the documented steps, and
within half a step of the 64-bit rotation; cache reads bit for bit code * scale.
"""
import numpy as np
import pytest
import torch

from _attn import cu, heads, paged, quantise32, rotate32, rotate64, to64
from selective_state_space_prefill_gb300 import binding as ssm
from selective_state_space_prefill_gb300.rope import rope_frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_rope_table_matches_64_bits(scaling):
    freq, scale = rope_frequencies(64, 10000.0, scaling, 1.0 if scaling is None else 8.0, original_len=4096)
    cos, sin = ssm.attn_rope_table(freq, 40001, scale)
    angle = np.arange(40001)[:, None] * np.asarray(freq)
    # one rounding to fp32 (2^-24 relative) of values whose angle is exact to 2^-50
    for got, ref in ((cos, scale * np.cos(angle)), (sin, scale * np.sin(angle))):
        assert np.max(np.abs(to64(got) - ref) - 2.0 ** -24 * np.abs(ref)) <= 1e-10


def _append_case(T, H, Hk, D, rot, interleaved, i8, page, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = heads(g, T, H + 2 * Hk, D, spread).to(DEV)          # strided views of one projection's rows
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    n_pos = 5 * T + 70
    pos = torch.randperm(n_pos, generator=g)[:T].to(torch.int32).to(DEV)
    n_pages = -(-T // page) + 2
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32).to(DEV)
    cos = sin = None
    if rot:
        f, s = rope_frequencies(rot)
        cos, sin = ssm.attn_rope_table(f, n_pos, s)
    shape = (n_pages, Hk, page, D)
    if i8:
        kc, vc = (torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).to(DEV) for _ in range(2))
        ks, vs = (torch.rand(shape[:3], generator=g).to(DEV) for _ in range(2))
    else:
        kc, vc = (torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        ks = vs = None
    return q, k, v, pos, cos, sin, kc, vc, slots, ks, vs


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("T,H,Hk,D,rot,interleaved,page", [
    (1, 1, 1, 16, 8, False, 16), (1, 32, 8, 128, 128, False, 16), (3, 7, 7, 64, 64, True, 32),
    (77, 24, 4, 64, 32, False, 48), (130, 12, 2, 80, 40, False, 64), (65, 5, 5, 96, 48, True, 16),
    (1500, 56, 8, 128, 64, True, 64), (1031, 6, 1, 112, 112, False, 80), (33, 4, 2, 32, 0, False, 16),
])
def test_append(T, H, Hk, D, rot, interleaved, page, i8):
    q, k, v, pos, cos, sin, kc, vc, slots, ks, vs = _append_case(T, H, Hk, D, rot, interleaved, i8, page, T + D)
    before = [t.clone() if t is not None else None for t in (kc, vc, ks, vs)]
    qo, ko = ssm.attn_append(q, k, v, pos, cos, sin, kc, vc, slots, ks, vs, interleaved=interleaved, k_out=True)
    torch.cuda.synchronize()
    p, sl = pos.cpu().numpy(), slots.cpu().numpy()
    for x, got, cache, scale, b_c, b_s, out in ((q, qo, None, None, None, None, qo), (k, ko, kc, ks, before[0], before[2], ko),
                                                (v, None, vc, vs, before[1], before[3], None)):
        x64 = to64(x)
        turned = rot > 0 and x is not v
        r64 = rotate64(x64, to64(cos), to64(sin), p, interleaved) if turned else x64
        r32 = rotate32(x64, cos.cpu().numpy(), sin.cpu().numpy(), p, interleaved) if turned else x64.astype(np.float32)
        if out is not None:
            # bit for bit the fp32 evaluation rounded to bf16, and near the 64-bit one
            assert torch.equal(out.cpu(), torch.from_numpy(r32).to(torch.bfloat16))
            partner = np.abs(x64).max(-1, keepdims=True)
            assert np.all(np.abs(to64(out) - r64) <= 2.0 ** -8 * np.abs(r64) + 2.0 ** -22 * partner)
        if cache is None:
            continue
        want = b_c.cpu().clone()
        pg, off = sl // page, sl % page
        if i8:
            codes, sc = quantise32(r32)
            want[pg, :, off] = torch.from_numpy(codes)
            want_s = b_s.cpu().clone()
            want_s[pg, :, off] = torch.from_numpy(sc)
            assert torch.equal(scale.cpu(), want_s)
            held = codes.astype(np.float64) * sc.astype(np.float64)[..., None]
            assert np.all(np.abs(held - r64) <= 0.5001 * sc[..., None] + 2.0 ** -22 * np.abs(x64).max(-1, keepdims=True))
        else:
            want[pg, :, off] = torch.from_numpy(r32).to(torch.bfloat16)
        assert torch.equal(cache.cpu(), want), "rows written, and rows left alone"
    assert ssm.device_status() == 0


def test_append_in_place_and_without_q():
    q, k, v, pos, cos, sin, kc, vc, slots, ks, vs = _append_case(40, 8, 2, 128, 128, False, True, 16, 5)
    ref_q, ref_k = ssm.attn_append(q, k, v, pos, cos, sin, kc, vc, slots, ks, vs, k_out=True)
    kc2, ks2 = torch.zeros_like(kc), torch.zeros_like(ks)
    vc2, vs2 = torch.zeros_like(vc), torch.zeros_like(vs)
    k2 = k.clone()
    none, ko = ssm.attn_append(None, k2, v, pos, cos, sin, kc2, vc2, slots, ks2, vs2, k_out=k2)
    assert none is None and ko is k2 and torch.equal(k2, ref_k)
    pg, off = slots.long() // 16, slots.long() % 16
    assert torch.equal(kc2[pg, :, off], kc[pg, :, off]) and torch.equal(vs2[pg, :, off], vs[pg, :, off])
    q2 = q.clone()
    qo, ko = ssm.attn_append(q2, k, v, pos, cos, sin, kc, vc, slots, ks, vs, q_out=q2)
    assert qo is q2 and ko is None and torch.equal(q2, ref_q)


def test_append_padding_and_bad_tokens_are_skipped():
    T = 12
    q, k, v, pos, cos, sin, kc, vc, slots, ks, vs = _append_case(T, 4, 2, 64, 64, False, True, 16, 9)
    keep = [t.clone() for t in (kc, vc, ks, vs)]
    ssm.device_status(clear=True)
    for bad_slot, bad_pos, status in ((-1, 0, 0), (-1, 10 ** 9, 0), (-2, 0, ssm.DEV_BAD_INDEX),
                                      (kc.shape[0] * 16, 0, ssm.DEV_BAD_INDEX), (3, -1, ssm.DEV_BAD_INDEX),
                                      (3, cos.shape[0], ssm.DEV_BAD_INDEX)):
        s2, p2 = torch.full_like(slots, bad_slot), torch.full_like(pos, bad_pos)
        qo = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        ssm.attn_append(q, k, v, p2, cos, sin, kc, vc, s2, ks, vs, q_out=qo)
        assert ssm.device_status(clear=True) == status, (bad_slot, bad_pos)
        assert bool((qo == 7.0).all())
        assert all(torch.equal(a, b) for a, b in zip(keep, (kc, vc, ks, vs)))
    ssm.attn_append(q[:0], k[:0], v[:0], pos[:0], cos, sin, kc, vc, slots[:0], ks, vs)      # no tokens
    assert all(torch.equal(a, b) for a, b in zip(keep, (kc, vc, ks, vs)))


def test_append_non_finite_and_zero_rows():
    T, Hk, D = 5, 1, 64
    k = torch.randn(T, Hk, D).to(torch.bfloat16)
    k[0] = 0
    k[1, 0, 3] = float("nan")
    k[2, 0, 5] = float("inf")
    k[3] = float("nan")
    kc, vc = (torch.full((1, Hk, 16, D), 9, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((1, Hk, 16), 9.0, device=DEV) for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    ssm.attn_append(None, k.to(DEV), k.to(DEV), None, None, None, kc, vc, slots, ks, vs)
    codes, sc = quantise32(k.float().numpy())
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(c.cpu().numpy()[0, 0, :T], codes[:, 0])
        assert np.array_equal(s.cpu().numpy()[0, 0, :T], sc[:, 0])
    assert sc[0, 0] == 0 and np.isinf(sc[2, 0]) and sc[3, 0] == 0
    kr, _ = ssm.attn_cache_read(kc, vc, torch.zeros(1, 1, dtype=torch.int32, device=DEV), cu([T]).to(DEV), T, ks, vs)
    assert bool(kr[2].isnan().all()) and bool((kr[0] == 0).all()) and bool(kr[4].isfinite().all())


@pytest.mark.parametrize("i8", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hk,D,page", [
    ([1], 1, 16, 16), ([777], 8, 128, 64), ([0, 5, 0, 0, 33, 1, 0], 3, 80, 48), ([300, 17, 256], 5, 64, 256),
    (list(range(0, 70)), 1, 112, 16),
])
def test_cache_read(lens, Hk, D, page, i8, out_dtype):
    g = torch.Generator().manual_seed(len(lens))
    T = sum(lens)
    c = paged(torch.randn(T, Hk, D, generator=g), torch.randn(T, Hk, D, generator=g), lens, page, i8)
    dev = {n: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    k, v = ssm.attn_cache_read(dev["k_cache"], dev["v_cache"], dev["table"], cu(lens).to(DEV), T, dev["k_scale"],
                               dev["v_scale"], out_dtype=out_dtype)
    for got, name in ((k, "k64"), (v, "v64")):
        want = torch.from_numpy(c[name]).float().to(out_dtype)      # an int8 code times an fp32 scale, rounded once
        assert torch.equal(got.cpu(), want)
    # a range of each sequence: its second half
    first = [n // 2 for n in lens]
    half = [n - f for n, f in zip(lens, first)]
    k, _ = ssm.attn_cache_read(dev["k_cache"], dev["v_cache"], dev["table"], cu(half).to(DEV), sum(half), dev["k_scale"],
                               dev["v_scale"], first=torch.tensor(first, dtype=torch.int32, device=DEV), out_dtype=out_dtype)
    at = np.concatenate([[0], np.cumsum(lens)])
    rows = np.concatenate([np.arange(at[b] + first[b], at[b + 1]) for b in range(len(lens))]).astype(int)
    assert torch.equal(k.cpu(), torch.from_numpy(c["k64"][rows]).float().to(out_dtype))
    assert ssm.device_status() == 0


def test_cache_read_bad_page_is_reported():
    c = paged(torch.randn(40, 2, 64), torch.randn(40, 2, 64), [40], 16, True)
    dev = {n: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    dev["table"][0, 1] = c["n_pages"]
    out = torch.full((40, 2, 64), 7.0, device=DEV)
    ssm.device_status(clear=True)
    k, _ = ssm.attn_cache_read(dev["k_cache"], dev["v_cache"], dev["table"], cu([40]).to(DEV), 40, dev["k_scale"],
                               dev["v_scale"], k_out=out)
    assert ssm.device_status(clear=True) == ssm.DEV_BAD_INDEX
    assert bool((k[16:32] == 7.0).all()) and torch.equal(k[:16].cpu().double(), torch.from_numpy(c["k64"][:16]).float().double())


def test_cache_rows_past_two_gib():
    """A cache whose rows lie past 2^31 bytes: the last pages written and read back."""
    Hk, D, page = 8, 128, 64
    n_pages = (5 << 29) // (Hk * D * page * 2) + 1                    # 2.5 GiB per bf16 cache
    kc, vc = (torch.zeros(n_pages, Hk, page, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    k, v = heads(g, 70, Hk, D).to(DEV), heads(g, 70, Hk, D).to(DEV)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    pos = torch.arange(70, device=DEV)
    slots = (table[0, pos // page] * page + pos % page).to(torch.int32)
    ssm.attn_append(None, k, v, None, None, None, kc, vc, slots)
    kr, vr = ssm.attn_cache_read(kc, vc, table, cu([70]).to(DEV), 70)
    assert torch.equal(kr, k) and torch.equal(vr, v)
    assert bool((kc[: n_pages - 2] == 0).all())
