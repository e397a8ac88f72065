"""Float64 CPU oracle for the 4-bit KV cache, decodes with weights, and eviction.

TEST INFRASTRUCTURE ONLY (see ``oracle/parallax.py``).

A cached row x of d values is held as d four-bit codes and (s, z):

    lo = min(0, min x), hi = max(0, max x)
    s = the smallest bf16 value >= (hi - lo) / 15,  z = rint(-lo / s)
    c = min(15, rint(x / s) + z)                    (ties to even)

and stands for s (c - z).  The rounding decisions are taken in exact rational
arithmetic here, the values in float64.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .parallax import decode_gqa_ref, softmax_weights_row


def _bf16_value(bits: int) -> float:
    return float(np.array([bits << 16], dtype=np.uint32).view(np.float32)[0])


def smallest_bf16_at_or_above(x: Fraction) -> float:
    """Smallest non-negative bf16 value >= x (x >= 0, below the largest bf16)."""
    if x == 0:
        return 0.0
    lo, hi = 0, 0x7F7F  # bit patterns of non-negative finite bf16 are ordered like their values
    while lo < hi:
        mid = (lo + hi) // 2
        if Fraction(_bf16_value(mid)) >= x:
            hi = mid
        else:
            lo = mid + 1
    return _bf16_value(lo)


def kv_quantize_int4_ref(X: np.ndarray):
    """Rows X[..., d] (values that bf16 holds) -> (codes uint8 [..., d/2], scales, zero points float64 [...])."""
    X = np.asarray(X, dtype=np.float64)
    d = X.shape[-1]
    rows = X.reshape(-1, d)
    codes = np.zeros(rows.shape, dtype=np.uint8)
    s = np.zeros(len(rows))
    z = np.zeros(len(rows))
    for i, x in enumerate(rows):
        if not np.isfinite(x).all():
            s[i] = math.nan
            continue
        lo, hi = min(0.0, x.min()), max(0.0, x.max())
        s[i] = smallest_bf16_at_or_above((Fraction(hi) - Fraction(lo)) / 15)
        if s[i] == 0:
            continue
        step = Fraction(s[i])
        z[i] = round(Fraction(-lo) / step)  # Fraction rounds ties to even
        codes[i] = [min(15, round(Fraction(v) / step) + int(z[i])) for v in x]
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return packed.reshape(*X.shape[:-1], d // 2), s.reshape(X.shape[:-1]), z.reshape(X.shape[:-1])


def kv_dequantize_int4_ref(codes: np.ndarray, s: np.ndarray, z: np.ndarray) -> np.ndarray:
    """The float64 values s (c - z) that 4-bit rows stand for."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1).astype(np.float64)
    return np.asarray(s)[..., None] * (c - np.asarray(z)[..., None])


def decode_weights_ref(q, r, K, V, seqlens, weights):
    """(out [B, H, d], weights + the softmax weights of every visible key summed over its KV head's query heads)."""
    B, H, _ = q.shape
    Hkv = K.shape[1]
    G = H // Hkv
    total = np.array(weights, dtype=np.float64)
    for b in range(B):
        n = int(seqlens[b])
        for h in range(H):
            total[b, h // G, :n] += softmax_weights_row(q[b, h], K[b, h // G, :n])
    return decode_gqa_ref(q, r, K, V, seqlens), total


def decode_magnitude(q, r, K, V, seqlens) -> np.ndarray:
    """sum_j p_j (1 + |t_j| + |tbar|) |v_j| of every output [B, H, d]: what rounding errors relative to each
    term of out = sum_j p_j (1 - t_j + tbar) v_j scale with."""
    B, H, d = q.shape
    G = H // K.shape[1]
    out = np.zeros((B, H, d))
    for b in range(B):
        n = int(seqlens[b])
        for h in range(H):
            k, v = K[b, h // G, :n], V[b, h // G, :n]
            p = softmax_weights_row(q[b, h], k)
            t = k @ r[b, h]
            out[b, h] = (p * (1 + np.abs(t) + abs(p @ t))) @ np.abs(v)
    return out


def evict_ref(weights, n: int, budget: int, sinks: int, recent: int) -> np.ndarray:
    """Positions, ascending, of the rows that one KV head of a sequence of n rows keeps."""
    if n <= budget:
        return np.arange(n)
    middle = sorted(range(sinks, n - recent),
                    key=lambda j: (math.isnan(weights[j]), 0.0 if math.isnan(weights[j]) else -weights[j], j))
    return np.array(sorted([*range(sinks), *middle[:budget - sinks - recent], *range(n - recent, n)]), dtype=np.int64)
