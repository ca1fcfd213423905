"""Plain float64 CPU oracle of the layers on the quantizer's 2/3/4-bit weights.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports, calls or links
this module; it shares no code, header, table or constant generator with the
HIP library.

    linear  Y = act(X·Ŵᵀ + b) + R
    glu     Y = act(X·Ŵgᵀ + bg) ⊙ (X·Ŵuᵀ + bu)
    moe     p = softmax(x·Rᵀ); the top_k largest (ties: the lower expert);
            y = Σ_j w_j·Ŵd_e(act(Ŵg_e·x) ⊙ (Ŵu_e·x)) + residual
with Ŵ the dequantized weight, all in float64 from the bytes the GPU reads.
"""
from __future__ import annotations

import math

import numpy as np

from .quantized_matmul import dequant_matmul

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(x, name):
    x = np.asarray(x, dtype=np.float64)
    if name == "none":
        return x
    if name == "relu":
        return np.maximum(x, 0.0)
    if name == "silu":
        with np.errstate(over="ignore"):
            return x / (1.0 + np.exp(-x))
    if name == "gelu":
        return 0.5 * x * _erfc(-x / math.sqrt(2.0))
    if name == "gelu_tanh":
        with np.errstate(over="ignore"):
            return x / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    raise ValueError(name)


def linear(X, w, n, bits, bias=None, activation="none", residual=None):
    """w = (qweight, scales, zeros, g_idx)."""
    y = dequant_matmul(X, *w, n, bits)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    y = activate(y, activation)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def glu(X, gate, up, n, bits, activation="silu", gate_bias=None, up_bias=None):
    return linear(X, gate, n, bits, gate_bias, activation) * linear(X, up, n, bits, up_bias)


def route(X, router, top_k, renormalize):
    """(ids [T, k], weights [T, k]): the largest softmax values, largest first."""
    logits = np.asarray(X, dtype=np.float64) @ np.asarray(router, dtype=np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    w = np.take_along_axis(e, ids, axis=1)
    return ids, w / (w if renormalize else e).sum(axis=1, keepdims=True)


def moe(X, router, experts, hidden, inter, bits, top_k, activation="silu", renormalize=True, residual=None):
    """experts: a list of (gate, up, down), each (qweight, scales, zeros, g_idx)."""
    X = np.asarray(X, dtype=np.float64)
    ids, wts = route(X, router, top_k, renormalize)
    y = np.zeros((X.shape[0], hidden))
    for e in np.unique(ids):
        gate, up, down = experts[e]
        t, j = np.nonzero(ids == e)
        mid = glu(X[t], gate, up, hidden, bits, activation)
        y[t] += wts[t, j][:, None] * dequant_matmul(mid, *down, inter, bits)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
    return y, ids, wts
