"""Float64 oracle of the attention gradients -- test infrastructure only.

The plain definition, score matrix materialised, for one document and all its
heads: with p_ij = exp(scale q_i.k_j - lse_i) over the visible pairs and
delta_i = dout_i.out_i - dlse_i,

    dv_j = sum_i p_ij dout_i
    ds_ij = p_ij (dout_i.v_j - delta_i)
    dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i

(out and lse as they are given; dk and dv summed over the query heads of a KV
head; key j visible to row i under causal masking iff j <= i + Lk - Lq).  With
``bounds`` the largest error that fp32 sums and bf16-rounded p, ds and results
can make comes beside each gradient, term by term:

    u = 2^-8 (rounding to bf16), f = 2^-23 (an fp32 operation, with room for
    truncating adders),
    p is off by r_ij = f ((D + 8) scale |q_i|.|k_j| + 4 |lse_i| + 8) of itself
    (scores of D terms, the exponent's rounding, 2^x),
    ds by e_ij = r_ij |ds_ij| + f (D + 8) p_ij (|dout_i|.|v_j| + |dout_i|.|out_i| + |dlse_i|),
    a sum of n terms x y by u |x||y| (x rounded) and f n |x||y|.
"""

from __future__ import annotations

import numpy as np

from .attention import _f64, visible_mask

U, F = 2.0 ** -8, 2.0 ** -23


def attention_gradients(q, k, v, out, lse, dout, scale, causal, dlse=None, bounds=False):
    """q, out, dout [Lq, Hq, D], k, v [Lk, Hkv, D], lse, dlse [Hq, Lq] ->
    (dq, dk, dv), or ((dq, bound), (dk, bound), (dv, bound))."""
    q, k, v, out, lse, dout = map(_f64, (q, k, v, out, lse, dout))
    Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[:2]
    group = Hq // Hkv
    dlse = np.zeros((Hq, Lq)) if dlse is None else _f64(dlse)
    seen = visible_mask(Lq, Lk, causal)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    rounded = 1.0 + U  # a rounded operand
    for h in range(Hq):
        g = h // group
        Q, K, V, O, G = q[:, h], k[:, g], v[:, g], out[:, h], dout[:, h]
        L = lse[h]
        live = np.isfinite(L)
        vis = seen & live[:, None]
        Q0, O0, G0 = (np.where(live[:, None], x, 0.0) for x in (Q, O, G))  # rows without a key give nothing
        s = scale * (Q0 @ K.T) - np.where(live, L, 0.0)[:, None]
        p = np.where(vis, np.exp(np.where(vis, s, 0.0)), 0.0)
        c = np.where(live, dlse[h], 0.0)
        delta = np.sum(G0 * O0, axis=1) - c
        ds = p * (G0 @ V.T - delta[:, None])
        dv[:, g] += p.T @ G0
        dq[:, h] = scale * (ds @ K)
        dk[:, g] += scale * (ds.T @ Q0)
        if bounds:
            r = F * ((D + 8) * scale * (np.abs(Q0) @ np.abs(K).T) + 4 * np.abs(np.where(live, L, 0.0))[:, None] + 8)
            size = np.abs(G0) @ np.abs(V).T + np.sum(np.abs(G0 * O0), axis=1)[:, None] + np.abs(c)[:, None]
            e = r * np.abs(ds) + F * (D + 8) * p * size
            nq, nk = Lq * group, Lk
            ep = (r * rounded + U + F * nq) * p
            bv[:, g] += ep.T @ np.abs(G0)
            bq[:, h] = scale * ((e * rounded + (U + F * nk) * np.abs(ds)) @ np.abs(K))
            bk[:, g] += scale * ((e * rounded + (U + F * nq) * np.abs(ds)).T @ np.abs(Q0))
    if not bounds:
        return dq, dk, dv
    tiny = 2.0 ** -133  # half of bf16's least subnormal
    return tuple((x, b * rounded + U * np.abs(x) + tiny) for x, b in ((dq, bq), (dk, bk), (dv, bv)))
