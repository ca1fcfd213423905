"""Plain float64 CPU oracle of the 4-bit key/value cache and of attention.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports, calls or links
this module; it shares no code, header, table or constant generator with the
HIP library.

    kept value  (q - z)·s per group x of channels, with
                s = the smallest bf16 with 15·s >= max x - min x, 4096·s >= max|x|, s >= 2^-100,
                z = -rint(min x / s), q = clamp(rint(x / s) + z, 0, 15)
    attention   Y_i = Σ_{j <= last_i} softmax_j(scale·q_i·k_j)·v_j; no j: zeros
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def smallest_bf16(need: Fraction) -> Fraction:
    """The smallest number of eight significant bits that is at least `need` > 0."""
    e = 0
    while Fraction(2) ** e * 256 < need * 1:
        e += 1
    while Fraction(2) ** (e - 1) * 255 >= need:
        e -= 1
    unit = Fraction(2) ** e
    return -(-need // unit) * unit


def kv_group(x) -> tuple:
    """(s, z, kept values) of one group; s is nan if it holds what cannot be kept."""
    x = [float(v) for v in x]
    if not all(abs(v) <= 2.0 ** 64 for v in x):
        return float("nan"), 0, [float("nan")] * len(x)
    f = [Fraction(v) for v in x]
    lo, hi, a = min(f), max(f), max(abs(v) for v in f)
    s = smallest_bf16(max((hi - lo) / 15, a / 4096, Fraction(2) ** -100))
    z = -round(lo / s)          # round() of a Fraction goes to even
    q = [min(max(round(v / s) + z, 0), 15) for v in f]
    return float(s), z, [float((c - z) * s) for c in q]


def kv_kept(x, group) -> np.ndarray:
    """What the cache keeps of x [..., dim], group channels to a scale."""
    x = np.asarray(x, dtype=np.float64)
    flat = x.reshape(-1, group)
    return np.array([kv_group(r)[2] for r in flat]).reshape(x.shape)


def attention(q, k, v, scale, last) -> np.ndarray:
    """q [n, heads, dim], k and v [t, kv_heads, dim], last[i]: the last position
    that token i sees (-1: none).  float64."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, heads, dim = q.shape
    share = heads // k.shape[1]
    y = np.zeros((n, heads, v.shape[2]))
    for h in range(heads):
        for i in range(n):
            seen = int(last[i]) + 1
            if seen <= 0:
                continue
            x = scale * (k[:seen, h // share] @ q[i, h])
            p = np.exp(x - x.max())
            y[i, h] = (p / p.sum()) @ v[:seen, h // share]
    return y
