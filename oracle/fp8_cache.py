"""The 8-bit paged KV cache in float64 NumPy: the code formats by their
definition, the quantising write, and the values a cache stands for.

Independent of the library and of any float8 type: a code is an integer 0 to
255, its value comes from its sign, exponent and fraction bits, and rounding
is a search among the values of all codes.
"""

from __future__ import annotations

import numpy as np

E4M3, E5M2 = "e4m3", "e5m2"


def code_values(kind: str) -> np.ndarray:
    """The value of each of the 256 codes.  e4m3 (the "fn" variant): 4 exponent
    bits, bias 7, no infinities, fraction and exponent all ones is NaN; e5m2:
    5 exponent bits, bias 15, infinities and NaN as in IEEE formats."""
    exps, bias = (4, 7) if kind == E4M3 else (5, 15)
    frac = 7 - exps
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> frac) & ((1 << exps) - 1), c & ((1 << frac) - 1)
        v = f * 2.0 ** (1 - bias - frac) if e == 0 else (2 ** frac + f) * 2.0 ** (e - bias - frac)
        if kind == E4M3 and c & 127 == 127:
            v = np.nan
        if kind == E5M2 and e == 31:
            v = np.nan if f else np.inf
        out[c] = -v if c & 128 else v
    return out


def quantise_rows(x, kind: str):
    """x [..., D] float64 -> (codes uint8 [..., D], exponent bytes uint8
    [...]): e = the least integer >= -126 with max |x| <= c_max 2^e over the
    finite values of a row, codes the nearest to x / 2^e (ties to the even
    code), NaN where x is not finite."""
    x = np.asarray(x, dtype=np.float64)
    pos = code_values(kind)[:128]
    pos = pos[np.isfinite(pos)]
    fine = np.isfinite(x)
    most = np.where(fine, np.abs(x), 0.0).max(-1, initial=0.0)
    e = np.full(most.shape, -126, dtype=np.int64)
    while np.any(up := most > pos[-1] * np.exp2(e.astype(np.float64))):
        e[up] += 1
    a = np.where(fine, np.abs(x), 0.0) / np.exp2(e.astype(np.float64))[..., None]
    hi = np.clip(np.searchsorted(pos, a), 0, pos.size - 1)  # pos[hi - 1] < a <= pos[hi]
    lo = np.maximum(hi - 1, 0)
    mid = (pos[lo] + pos[hi]) / 2
    code = np.where(a > mid, hi, np.where(a < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == pos[hi], hi, code)
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(fine, code, 127).astype(np.uint8), (e + 127).astype(np.uint8)


def stands_for(codes, exponents, kind: str) -> np.ndarray:
    """float64 values of a cache: codes [2, nb, bs, Hkv, D], exponent bytes
    [2, nb, Hkv, bs] -> [2, nb, bs, Hkv, D]."""
    e = np.asarray(exponents).astype(np.float64) - 127.0
    return code_values(kind)[np.asarray(codes)] * np.exp2(e).transpose(0, 1, 3, 2)[..., None]


def kv_cache_write_fp8(key, value, slot_mapping, codes, exponents, kind: str):
    """Tokens in order into copies of (codes, exponents); a negative slot
    stores nothing, one past the cache is an error."""
    codes, exponents = np.array(codes), np.array(exponents)
    _, nb, bs, _, _ = codes.shape
    for half, x in enumerate((key, value)):
        c, e = quantise_rows(x, kind)
        for t, slot in enumerate(np.asarray(slot_mapping).astype(np.int64)):
            if slot < 0:
                continue
            if slot >= nb * bs:
                raise ValueError(f"slot {slot} is past the cache")
            codes[half, slot // bs, slot % bs] = c[t]
            exponents[half, slot // bs, :, slot % bs] = e[t]
    return codes, exponents
