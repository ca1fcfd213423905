"""Inputs, references and error bounds of the layers on packed weights.

Bounds, from the kernels' arithmetic (u = 2^-24, S = Σ_k s_g(k)·|x_k|).  A
group of at most 128 positions is two fp32 chains, Σ x·(16 + q) and Σ x, of
products that are exact; each addition rounds once, to at most 2u of the
chain's absolute sum whatever the matrix core's internal rounding is, and the
offset is taken off in one fused step:
    |error of a group| <= s·Σ|x|·((16 + q) + (16 + z))·(2·128 + 2)·u
                       <= 16100·u·s·Σ|x|          for q, z <= 15,
and every fold of a group or of a wave's share adds at most u of the sum so
far, at most 16·S: F = n/32 + 16 folds.  Together
    E = u·(16100 + 16·F)·S                         (zbig: zero points beyond 15
                                                   scale it by (16 + |z|)/31).
These are worst cases.  In the root mean square the same chain of some eight
roundings at a magnitude of at most (16 + q)/|q - z| <= 20 times the result
(2-bit codes) gives sqrt(8)·20·u = 3.4e-6: REL holds the relative Frobenius
error of fp32 results before an activation to 4e-6.

An activation has slope at most 1.13 and its own fp32 evaluation errs by at
most 16u·|x|.  A result in bf16 adds half a step, 2^-8 of its value.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

U = 2.0 ** -24
REL = 4e-6
TDT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def pack_words(Q):
    """Codes [m, n] -> int32 words, column 8w+i in bits [4i, 4i+4)."""
    m, n = Q.shape
    nw = (n + 7) // 8
    P = np.zeros((m, nw * 8), dtype=np.uint64)
    P[:, :n] = Q
    out = np.zeros((m, nw), dtype=np.uint64)
    for i in range(8):
        out |= P[:, i::8] << np.uint64(4 * i)
    return out.astype(np.uint32).view(np.int32)


def group_index(n, g, rng, act_order):
    gw = n if g == -1 else g
    gidx = np.zeros(n, dtype=np.int32)
    gidx[rng.permutation(n) if act_order else np.arange(n)] = np.arange(n) // gw
    return gidx


def weight(m, n, bits, g, rng, gidx, exact=False, zero_lo=0, zero_hi=None):
    """(qweight, scales, zeros, g_idx) of a random quantized weight."""
    G = 1 if g == -1 else -(-n // g)
    Q = rng.integers(0, 2 ** bits, size=(m, n))
    zeros = rng.integers(zero_lo, 2 ** bits if zero_hi is None else zero_hi, size=(m, G)).astype(np.int32)
    if exact:
        scales = (2.0 ** -rng.integers(0, 4, size=(m, G))).astype(np.float32)
    else:
        scales = rng.uniform(0.002, 0.05, size=(m, G)).astype(np.float32)
    return pack_words(Q), scales, zeros, gidx


def gpu(w):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in w]


def activations(tokens, n, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, n, generator=g) * scale).to(torch.bfloat16)


def vector(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(TDT[dtype])


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def product_bound(X, w, n, planes=1):
    """E of every output of X·Ŵᵀ (X float64, the exact values the GPU reads)."""
    _, scales, zeros, gidx = w
    S = np.abs(X) @ np.abs(scales).astype(np.float64)[:, gidx].T
    zmax = max(31.0, 16.0 + float(np.abs(zeros).max())) / 31.0 if zeros.size else 1.0
    return U * planes * (16100 * zmax + 16 * zmax * (n / 32 + 16)) * S


def act_bound(x, e):
    """Error bound of act(x ± e) evaluated in fp32."""
    return 1.13 * e + 16 * U * (np.abs(x) + e)


def rounded(y, e, dtype):
    """Bound after the last fp32 steps and the rounding to the result's type."""
    e = e + 4 * U * (np.abs(y) + e)
    return e + (2.0 ** -8 * (np.abs(y) + e) if dtype == "bf16" else 0.0) + 1e-37


def linear_ref(X, w, n, bits, bias=None, act="none", residual=None, out="fp32"):
    """(reference, bound) of gptq_w4a16_linear."""
    pre = oracle.linear(X, w, n, bits, bias)
    e = product_bound(X, w, n)
    y = oracle.activate(pre, act)
    e = act_bound(pre, e)
    if residual is not None:
        y = y + residual
        e = e + U * np.abs(y)
    return y, rounded(y, e, out)


def glu_ref(X, gate, up, n, bits, act, gate_bias=None, up_bias=None):
    """(reference, bound before the last rounding)."""
    g = oracle.linear(X, gate, n, bits, gate_bias)
    u = oracle.linear(X, up, n, bits, up_bias)
    eg = act_bound(g, product_bound(X, gate, n) + U * np.abs(g))
    eu = product_bound(X, up, n) + U * np.abs(u)
    a = oracle.activate(g, act)
    return a * u, np.abs(a) * eu + np.abs(u) * eg + eg * eu + 2 * U * np.abs(a * u)


def moe_ref(X, router, experts, hidden, inter, bits, top_k, act, renorm, residual=None, out="fp32"):
    """(reference, bound, ids, weights) of gptq_w4a16_moe."""
    y, ids, wts = oracle.moe(X, router, experts, hidden, inter, bits, top_k, act, renorm, residual)
    e = np.zeros_like(y)
    size = np.zeros_like(y)
    for x in np.unique(ids):
        gate, up, down = experts[x]
        t, j = np.nonzero(ids == x)
        a, ea = glu_ref(X[t], gate, up, hidden, bits, act)
        ea = ea + 2.0 ** -16 * (np.abs(a) + ea)              # two bf16 parts at least
        Wd = oracle.dequantized_weight(*down, inter, bits)
        part = np.abs(a @ Wd.T)
        ed = ea @ np.abs(Wd).T + product_bound(np.abs(a) + ea, down, inter, planes=3)
        w = wts[t, j][:, None]
        e[t] += w * (ed + 2 * U * part)
        size[t] += w * part
    e += U * (top_k + 1) * size                              # the weighted sum
    if residual is not None:
        e += U * np.abs(y)
    return y, rounded(y, e, out), ids, wts


def check(got, ref, bound, what, out="fp32", rel=None):
    g = got.detach().cpu().to(torch.float64).numpy()
    err = np.abs(g - ref)
    fro = float(np.linalg.norm(g - ref) / max(np.linalg.norm(ref), 1e-300)) if ref.size else 0.0
    worst = float(np.max(err / bound)) if ref.size else 0.0
    print(f"{what}: worst error {worst:.3f} of its bound, rel frob {fro:.3e}", flush=True)
    assert g.shape == ref.shape
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    assert np.all(err <= bound), f"{what}: {int(np.sum(err > bound))} outputs beyond the bound ({worst:.2f}x)"
    if rel is not None:
        assert fro <= rel + (2.0 ** -8 if out == "bf16" else 0.0), f"{what}: relative Frobenius error {fro:.3e}"
