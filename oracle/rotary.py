"""Float64 oracle of rotary positions -- test infrastructure only.

Pair i of a head's first ``rot`` values, (x, y) at i and i + rot / 2 (half) or
at 2 i and 2 i + 1 (interleaved), turned by a = t f_i and multiplied by the gain;
``transpose`` turns by -a.  With ``bounds`` the largest error of fp32 arithmetic
on exactly reduced angles, rounded once to bf16:

    the angle: t f_i / 2 pi is off by t (2^-52 f_i / 2 pi + 2^-65) turns from the
    rounded steps (and by as much here), its fp32 fraction and that times pi by
    2 * 2^-24 of at most pi: da = 2 t (2^-52 f_i + 2^-62) + 2^-21
    cos and sin: da + 2^-22 (a few units in the last place), times gain 2^-23
    two products and a sum: 3 * 2^-24 of |x| + |y|
    the rounding to bf16: 2^-8 of the result
"""

from __future__ import annotations

import numpy as np

from .attention import _f64


def rotary(x, positions, inv_freq, rot, interleaved=False, gain=1.0, transpose=False, bounds=False):
    """x [T, H, D] -> the turned values (float64), or (values, bounds)."""
    x = _f64(x)
    t = np.asarray(positions, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = rot // 2
    first, second = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    a = t[:, None] * f * (-1.0 if transpose else 1.0)
    c, s = gain * np.cos(a)[:, None], gain * np.sin(a)[:, None]
    y, b = x.copy(), np.zeros_like(x)
    p, q = x[..., first], x[..., second]
    y[..., first], y[..., second] = p * c - q * s, p * s + q * c
    if not bounds:
        return y
    da = 2.0 * np.abs(t)[:, None] * (2.0 ** -52 * np.abs(f) + 2.0 ** -62) + 2.0 ** -21
    off = abs(gain) * (da + 2.0 ** -22 + 2.0 ** -23 + 3 * 2.0 ** -24)[:, None] * (np.abs(p) + np.abs(q)) * 1.01
    for at in (first, second):
        b[..., at] = off + 2.0 ** -8 * np.abs(y[..., at]) + 2.0 ** -133
    return y, b
