"""Plain 64-bit forms of the operators around a decode step's mixers, on the CPU, and the error bounds of fp32
evaluations of them, each derived beside it."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

F64 = np.float64
U = 2.0 ** -24                                      # half a step of fp32, relative


def to64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    """The rounding of an output, relative to its value."""
    return {torch.float32: U, torch.bfloat16: 2.0 ** -8}[dtype]


# ------------------------------------------------------------------ norm
def norm64(x, weight, residual, eps, groups):
    """(y [rows, groups, n], r [rows, width]) in 64 bits."""
    r = to64(x) + (to64(residual) if residual is not None else 0.0)
    g = r.reshape(r.shape[0], groups, -1)
    with np.errstate(all="ignore"):
        y = g / np.sqrt((g ** 2).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * to64(weight).reshape(1, groups, -1)
    return y, r


# A row's fp32 sum of squares goes through at most 128 additions in a thread (32768 channels over 256 threads) and
# 16 across threads, each off by U of the sum at most, and r and its square by 3 U: 147 U on the mean, half of it on
# its root; the reciprocal root (2 steps, 4 U), two products and the sum with eps: below 80 U in all.
NORM_REL = 80 * U


def check_norm(out, scale, x, weight, residual, eps, groups):
    y, _ = norm64(x, weight, residual, eps, groups)
    rows, _, n = y.shape
    if out.dtype != torch.int8:
        got = to64(out).reshape(y.shape)
        tiny = 2.0 ** -126                          # results below the normal range
        bad = np.abs(got - y) > np.abs(y) * (NORM_REL + half_step(out.dtype) * 1.01) + tiny
        assert not bad.any(), (np.argwhere(bad)[0], got[bad][0], y[bad][0])
        return
    amax = np.abs(y).max(-1)
    s = to64(scale)
    assert s.shape == (rows, groups)
    assert (np.abs(s - amax / 127) <= (amax / 127) * (NORM_REL + 2 * U) + 2.0 ** -149).all()
    c = out.cpu().numpy().reshape(y.shape).astype(F64)
    with np.errstate(all="ignore"):
        t = np.where(amax[..., None] > 0, y * 127 / amax[..., None], 0.0)
    # a code is the nearest whole number; next to a tie the value's own error (both y's and amax's) decides
    assert (np.abs(c - t) <= 0.5 + 127 * (2 * NORM_REL + 4 * U)).all()
    assert np.abs(c).max(initial=0) <= 127


# ------------------------------------------------------------------ 4-bit weights
def unpack(codes):
    """[N, K] codes of [N, K / 2] bytes."""
    b = codes.cpu().numpy()
    return np.stack([b & 15, b >> 4], -1).reshape(b.shape[0], -1).astype(F64)


def weight64(codes, scales, zeros):
    c = unpack(codes)
    n, k = c.shape
    s = to64(scales)
    group = k // s.shape[1]
    z = (zeros.cpu().numpy() & 15).astype(F64) if zeros is not None else np.full(s.shape, 8.0)
    return (c - np.repeat(z, group, 1)) * np.repeat(s, group, 1)


def quantise32(W, group, zeros, scale_dtype):
    """The definition of w4_quantize, every operation rounded to fp32: (codes [N, K], scales, zeros or None)."""
    w = W.detach().cpu().float().numpy()
    n, k = w.shape
    g = w.reshape(n, k // group, group)
    lo, hi = np.minimum(g.min(-1), 0), np.maximum(g.max(-1), 0)
    s = (hi - lo) / np.float32(15) if zeros else np.maximum(-lo, hi) / np.float32(7)
    s = torch.from_numpy(s.astype(np.float32)).to(scale_dtype)
    sf = s.float().numpy()
    with np.errstate(all="ignore"):
        q = np.rint((g / sf[..., None]).astype(np.float32))
        z = np.where(sf > 0, np.clip(np.rint((-lo / sf).astype(np.float32)), 0, 15), 8) if zeros else np.full(sf.shape, 8.0)
        c = np.where(sf[..., None] > 0, np.clip(q + z[..., None], 0 if zeros else 1, 15), 8)
    return c.reshape(n, k).astype(np.uint8), s, (z.astype(np.uint8) if zeros else None)


def activations64(x, x_scale):
    v = to64(x)
    if x_scale is None:
        return v
    s = to64(x_scale).reshape(v.shape[0], -1)
    return v * np.repeat(s, v.shape[1] // s.shape[1], 1)


def check_linear(out, x, codes, scales, zeros, x_scale):
    """Products are exact.  Their sum goes through no more than 128 steps in sequence (a matrix instruction's own
    sum counted as two), each cut off (2 U) or rounded at the size of sum |x w|; the scales' products add 4 U.
    Where a thread adds all groups of a row one after another, each addition is rounded (U): that many U, at most
    16 steps (2 U) inside a group, 8 U for the sum of slices and 4 U."""
    xv, w = activations64(x, x_scale), weight64(codes, scales, zeros)
    ref, mag = xv @ w.T, np.abs(xv) @ np.abs(w).T
    got = to64(out)
    assert got.shape == ref.shape
    bad = np.abs(got - ref) > mag * (max(260, scales.shape[1] + 44) * U) + np.abs(ref) * half_step(out.dtype) * 1.01 + 2.0 ** -126
    assert not bad.any(), (np.argwhere(bad)[0], got[bad][0], ref[bad][0], mag[bad][0])


# ------------------------------------------------------------------ probabilities
def probs64(logits, temperature):
    x = to64(logits)
    out = np.zeros(x.shape)
    for r in range(x.shape[0]):
        t = 1.0 if temperature is None else float(temperature[r])
        m = x[r].max(initial=-np.inf) if not np.isnan(x[r]).any() else np.nan
        if np.isnan(m) or m == np.inf or np.isnan(t):
            out[r] = np.nan
        elif m == -np.inf:
            continue
        elif t <= 2.0 ** -100:
            out[r, int(np.argmax(x[r]))] = 1.0
        else:
            e = np.exp((x[r] - m) / min(t, 3.0e38))
            out[r] = e / e.sum()
    return out


def check_probs(got, logits, temperature):
    """The exponent d = (x - m) / t in base 2 is off by 4 U of itself, the power by 2^-22 more (4 U) and the sum of
    positive terms by U for each addition in sequence (at most vocab / 512 and 32) and as the powers are."""
    ref, x = probs64(logits, temperature), to64(logits)
    g = to64(got)
    assert (np.isnan(g) == np.isnan(ref)).all()
    with np.errstate(all="ignore"):
        d = np.abs(x - x.max(-1, keepdims=True))
        if temperature is not None:
            d = d / np.maximum(to64(temperature), 2.0 ** -100)[:, None]
    d = np.where(np.isfinite(d), d, 0.0)
    near = np.minimum(d, 110.0)                      # further away the result is below 2^-149
    rel = (4 * near + 16 + 4 * 20 + x.shape[1] / 512 + 32) * U
    ok = np.isnan(ref) | (np.abs(g - ref) <= ref * rel + 2.0 ** -125)
    assert ok.all(), (np.argwhere(~ok)[0], g[~ok][0], ref[~ok][0])


# ------------------------------------------------------------------ verification
def _whole(p):
    """A probability as Fraction; negative ones and NaN are 0."""
    return Fraction(2) ** 200 if p == np.inf else Fraction(float(p)) if p > 0 else Fraction(0)


def _units(p):
    """The same in whole units of 2^-62, cut off."""
    return int(_whole(p) * 2 ** 62)


def verify_exact(draft, target, u, draft_probs=None, n_draft=None):
    """The definition in exact fractions: (tokens [batch, n + 1], n_kept [batch])."""
    target, u, draft = target.cpu().numpy(), u.cpu().numpy(), draft.cpu().numpy()
    q = None if draft_probs is None else draft_probs.cpu().numpy()
    batch, places, vocab = target.shape
    tokens, kept = np.full((batch, places), -1, np.int32), np.zeros(batch, np.int32)

    def uniform(v):
        return Fraction(float(min(v, np.float32(1 - 2.0 ** -24)))) if v > 0 else Fraction(0)

    for b in range(batch):
        n = places - 1 if n_draft is None else min(max(int(n_draft[b]), 0), places - 1)
        a = 0
        while a < n:
            d = int(draft[b, a])
            inside = 0 <= d < vocab
            pd = _whole(target[b, a, d]) if inside else Fraction(0)
            qd = Fraction(1) if q is None else _whole(q[b, a, d]) if inside else Fraction(0)
            if not uniform(u[b, a]) * qd < pd:
                break
            tokens[b, a] = d
            a += 1
        mass = [_units(v) for v in target[b, a]]
        if a < n:
            if q is None:
                less = list(mass)
                if 0 <= int(draft[b, a]) < vocab:
                    less[int(draft[b, a])] = max(0, less[int(draft[b, a])] - 2 ** 62)
            else:
                less = [max(0, p - _units(v)) for p, v in zip(mass, q[b, a])]
            if sum(less) > 0:
                mass = less
        total, at = sum(mass), 0
        if 0 < total < 4 * 2 ** 62:
            border, run = uniform(u[b, places - 1]) * total, 0
            for at, m in enumerate(mass):
                run += m
                if run > border:
                    break
            tokens[b, a] = at
        kept[b] = a
    return tokens, kept

