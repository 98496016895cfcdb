"""Plain 64-bit forms of the attention operators, on the CPU, and seeded inputs for them."""
from __future__ import annotations

import numpy as np
import torch

from _gpu import half_ulp_bf16

F64 = np.float64


def to64(t):
    return t.detach().cpu().double().numpy()


def rotate64(x, cos, sin, pos, interleaved):
    """x [T, heads, D] float64; cos, sin [n_pos, half]."""
    half = cos.shape[1]
    c, s = cos[pos][:, None, :], sin[pos][:, None, :]
    y = x.copy()
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def rotate32(x, cos, sin, pos, interleaved):
    """The same with every product and sum rounded to float32."""
    half = cos.shape[1]
    c, s = cos[pos][:, None, :], sin[pos][:, None, :]
    y = x.astype(np.float32).copy()
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def quantise32(x):
    """(codes, scale) of float32 rows [..., D]; NaN ignored by the maximum, code 0."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(x), np.float32(0), np.abs(x)), -1)
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
        r = np.rint(x * inv[..., None])
        r = np.where(np.isnan(r), 0, np.clip(r, -127, 127))
        return r.astype(np.int8), (amax / np.float32(127)).astype(np.float32)


def attend64(q, k, v, scale, first):
    """q [r, H, D], k and v [n, Hk, D] float64; row i sees keys 0 .. first + i (first may be negative).
    Returns out, lse, and per row and head what the error bounds need: sum_j p_j |v_j| [r, H, D] and
    the largest scale * sum_d |q_d k_jd| over the visible keys [r, H]."""
    r, H, D = q.shape
    n, Hk, _ = k.shape
    out, absum = np.zeros((r, H, D)), np.zeros((r, H, D))
    lse, mag = np.full((r, H), -np.inf), np.zeros((r, H))
    for h in range(H):
        kh, vh = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        for i in range(r):
            see = min(n, first + i + 1)
            if see <= 0:
                continue
            s = scale * (kh[:see] @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            p /= l
            out[i, h] = p @ vh[:see]
            absum[i, h] = p @ np.abs(vh[:see])
            lse[i, h] = m + np.log(l)
            mag[i, h] = scale * (np.abs(kh[:see]) @ np.abs(q[i, h])).max()
    return out, lse, absum, mag


def score_error(mag, D):
    """A bound of the error of a score: D products summed in fp32, the scale in units of log 2 and the
    hardware exponential's and its argument's rounding."""
    return (D + 8) * 2.0 ** -24 * mag + 2.0 ** -20


# Unit roundoff of the softmax weights as the second product takes them: bf16 has 8 significant bits
# (attn_prefill), fp16 has 11 and a bf16 pair 16 (attn_decode_step).
W_PREFILL, W_DECODE = 2.0 ** -8, 2.0 ** -11


def out_bound(out, absum, mag, D, out_dtype, weight):
    """Bound of |kernel - 64-bit|: each softmax weight is off by its score's error twice (itself and the
    sum) and by its rounding; fp32 accumulation; then the output's rounding (half a bf16 ulp)."""
    e = score_error(mag, D)[..., None]
    b = absum * (weight * 1.01 + 2.1 * e + 2.0 ** -18) + 1e-30
    if out_dtype == torch.bfloat16:
        b = b + half_ulp_bf16(np.abs(out) + b)
    return b


def check_attention(got, lse, ref, D, out_dtype, weight, what=""):
    out, rl, absum, mag = ref
    g = to64(got)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    ratio = np.abs(g - out) / out_bound(out, absum, mag, D, out_dtype, weight)
    assert ratio.max(initial=0) <= 1.0, f"{what}: error {ratio.max():.3g} of the bound at {np.unravel_index(ratio.argmax(), ratio.shape)}"
    if lse is not None:
        gl = to64(lse)
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty), f"{what}: lse of empty rows"
        e = np.abs(gl[~empty] - rl[~empty])
        b = (score_error(mag, D) + 2.0 ** -22 * np.abs(rl))[~empty]
        assert (e <= b).all(), f"{what}: lse error {(e / b).max():.3g} of its bound"


def heads(g, t, h, d, gain=1.0):
    return (torch.randn(t, h, d, generator=g) * gain).to(torch.bfloat16)


def paged(rows_k, rows_v, lens, page, i8, seed=0, spare=3, junk=float("nan")):
    """Sequences' rows (packed [T, Hk, D] float32 tensors) laid into a shuffled paged cache whose unwritten
    rows hold `junk`.  Returns dict of CPU tensors: k_cache, v_cache, k_scale, v_scale, table, and the
    values the cache stands for (k64, v64)."""
    g = torch.Generator().manual_seed(seed)
    Hk, D = rows_k.shape[1:]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lens), max(1, max(need)) + 1), 2 ** 31 - 1, dtype=torch.int32)
    shape = (n_pages, Hk, page, D)
    out = {}
    if i8:
        caches = [torch.randint(-128, 128, shape, generator=g, dtype=torch.int8) for _ in range(2)]
        scales = [torch.full(shape[:3], junk) for _ in range(2)]
    else:
        caches = [torch.full(shape, junk, dtype=torch.bfloat16) for _ in range(2)]
        scales = [None, None]
    values = [torch.empty(rows_k.shape, dtype=torch.float64) for _ in range(2)]
    at = pg = 0
    for b, n in enumerate(lens):
        ids = order[pg:pg + need[b]]
        pg += need[b]
        table[b, :need[b]] = ids.to(torch.int32)
        for j in range(n):
            p, o = int(ids[j // page]), j % page
            for x, (c, s, val) in zip((rows_k, rows_v), zip(caches, scales, values)):
                row = x[at + j].float()
                if i8:
                    codes, sc = quantise32(row.numpy())
                    c[p, :, o], s[p, :, o] = torch.from_numpy(codes), torch.from_numpy(sc)
                    val[at + j] = torch.from_numpy(codes.astype(F64) * sc.astype(F64)[:, None])
                else:
                    c[p, :, o] = row.to(torch.bfloat16)
                    val[at + j] = row.to(torch.bfloat16).double()
        at += n
    out.update(k_cache=caches[0], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1], table=table,
               k64=values[0].numpy(), v64=values[1].numpy(), n_pages=n_pages)
    return out


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
