"""Conditioning: norms and rotation of Q and K in place, attention to states of another length.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* qk_norm_rope: RMSNorm of every head, then every pair turned by its row of
  the table; interleaved pairs (2i, 2i + 1) or halves (i, i + D/2).  A position
  outside the table turns nothing.
* conditioned: every query of batch b attends to the keys of one or more
  segments one behind the other.  A segment is a list of sets; batch b of B
  reads set b // (B // n_sets), query head h reads head h // (H // H_kv).  Each
  set is given as its rows [l, H_kv, D] that count.  No key: o = 0, lse = -inf.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64, attention


def qk_norm_rope(x, gamma=None, eps=1e-6, table=None, pos=None, pairing="interleaved"):
    """x [n, H, D] -> fp64 [n, H, D]."""
    x = _f64(x)
    D = x.shape[-1]
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    if gamma is not None:
        y = y * _f64(gamma)
    if table is None:
        return y
    table = _f64(table).reshape(-1, D // 2, 2)
    out = y.copy()
    for n, p in enumerate(np.asarray(pos)):
        if not 0 <= p < len(table):
            continue
        c, s = table[p, :, 0], table[p, :, 1]
        i0, i1 = (slice(0, D, 2), slice(1, D, 2)) if pairing == "interleaved" else (slice(0, D // 2), slice(D // 2, D))
        a, b = y[n, :, i0], y[n, :, i1]
        out[n, :, i0], out[n, :, i1] = a * c - b * s, a * s + b * c
    return out


def conditioned(q, segments, scale=None):
    """q [B, T, S, H, D]; segments: per segment a list of (k, v) rows [l, H_kv, D] per set.

    Returns o [B, T, S, H, D], lse [B, T, H, S] and the weighted mean of |v|
    (same shape as o), the magnitude that rounding errors of the weights scale
    with."""
    q = _f64(q)
    B, T, S, H, D = q.shape
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.zeros((B, T, H, S))
    for b in range(B):
        parts = [seg[b // (B // len(seg))] for seg in segments]
        k = np.concatenate([_f64(p[0]) for p in parts])
        v = np.concatenate([_f64(p[1]) for p in parts])
        for h in range(H):
            hk = h // (H // k.shape[1])
            qh = q[b, :, :, h].reshape(T * S, D)
            oh, lh = attention(qh, k[:, hk], v[:, hk], scale)
            o[b, :, :, h] = oh.reshape(T, S, D)
            lse[b, :, h] = lh.reshape(T, S)
            mag[b, :, :, h] = attention(qh, k[:, hk], np.abs(v[:, hk]), scale)[0].reshape(T, S, D)
    return o, lse, mag
