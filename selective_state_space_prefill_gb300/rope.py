"""Frequencies of rotary positions, plain or scaled for contexts longer than the model was trained on.

``rope_frequencies`` gives what ``binding.attn_rope_table`` takes: the angle per position of each pair
of rotated dimensions, and the factor on the cosines and sines.
"""
from __future__ import annotations

import math


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int | None = None, alpha: float = 1.0, beta: float = 32.0):
    """(inv_freq [rot_dim / 2] floats, table scale).

    scaling None      inv_freq_i = base ** (-2 i / rot_dim)
            "linear"  positions interpolated: inv_freq / factor
            "ntk"     the base grown so that the slowest pair is interpolated by factor and the fastest
                      kept: base * factor ** (rot_dim / (rot_dim - 2))
            "yarn"    by parts (Peng et al., "YaRN", 2023): with r = original_len * inv_freq / 2 pi turns
                      over the original context and ramp = clamp((r - alpha) / (beta - alpha), 0, 1),
                      inv_freq * (ramp + (1 - ramp) / factor); the table is scaled by 0.1 ln(factor) + 1
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in (None, "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling == "yarn":
        if original_len is None or not beta > alpha:
            raise ValueError("yarn scaling needs original_len and beta > alpha")
        out = []
        for f in freq:
            ramp = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - alpha) / (beta - alpha)))
            out.append(f * (ramp + (1.0 - ramp) / factor))
        return out, 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    raise ValueError(f"unknown scaling {scaling!r}")
