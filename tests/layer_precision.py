"""What the bounds of layer_helpers, which are worst cases, do not notice: an
operand held in too few bits.

Relative Frobenius errors.  A product is off by at most H.REL (layer_helpers).
A gated half act(g)·u: g and u are each off by REL of their size; act's slope
is at most 1.13 and rms(act(g)) at least rms(g)/√2 for g of both signs (less
where |g| < 1, where the slope is as much smaller), so act(g) is off by 1.6 REL
and the half by 2.6: GLU = 4 REL.  An expert's sum adds its down product: MOE =
5 REL, and the hidden activation's bf16 parts, 2^-17 for two of them (a bf16
result), nothing for three (fp32).  A hidden activation of one bf16 would be off
by 2^-9 to 2^-8 of each value, evenly spread: 1e-3 and more.

bf16 results.  Their own rounding, up to 2^-8, hides such an error in a norm; but
a result that is off by d of a value rounds otherwise than the reference only
where a rounding border lies between, and borders are 2^-8 of a value apart or
more: with d = MOE + 2^-17 = 2.8e-5 that is 0.7 % of the results of the mean
size, and with the smaller ones of a normal distribution, for which the error is
the larger part, up to 4 %.  OFF = 5 %, plus three standard deviations of the
count.  One bf16 part of the hidden activation moves a third of the results.
"""
from __future__ import annotations

import numpy as np
import torch

import layer_helpers as H
import oracle

GLU, MOE, OFF = 4 * H.REL, 5 * H.REL, 0.05


def errors(got, ref, out):
    """(relative Frobenius error, share of results off the rounded reference)."""
    g = got.detach().cpu().to(torch.float64).numpy()
    fro = float(np.linalg.norm(g - ref) / np.linalg.norm(ref))
    rounded = torch.from_numpy(np.ascontiguousarray(ref)).to(H.TDT[out]).to(torch.float64).numpy()
    return fro, float(np.mean(g != rounded))


def within(fro, off, size, out, rel):
    if out == "fp32":
        return fro <= rel
    return fro <= rel + 2.0 ** -8 + 2.0 ** -17 and off <= OFF + 3 * (OFF / size) ** 0.5


def parts(v, planes):
    """v as the sum of `planes` bf16 parts, largest first, each rounded to nearest."""
    v = torch.from_numpy(np.ascontiguousarray(v)).to(torch.float32)
    total = torch.zeros_like(v)
    for _ in range(planes):
        p = (v - total).to(torch.bfloat16).to(torch.float32)
        total = total + p
    return total.to(torch.float64).numpy()


def moe_with_parts(X, router, experts, hidden, inter, bits, top_k, act, renorm, residual, planes):
    """oracle.moe with the hidden activation held in `planes` bf16 parts."""
    ids, wts = oracle.route(X, router, top_k, renorm)
    y = np.zeros((X.shape[0], hidden))
    for e in np.unique(ids):
        gate, up, down = experts[e]
        t, j = np.nonzero(ids == e)
        mid = parts(oracle.glu(X[t], gate, up, hidden, bits, act), planes)
        y[t] += wts[t, j][:, None] * oracle.dequant_matmul(mid, *down, inter, bits)
    return y if residual is None else y + residual


def exact_moe(tokens, inter, g, out, seed):
    """An expert layer whose result every step holds exactly: integer
    activations, scales of 1, one row of gate that is not zero, so the down
    product has one term per output, up to 15·2^20 < 2^24.  Of the seeds from
    `seed` the first whose hidden values are below 2^16 for a bf16 result (two
    parts hold them) or 2^20 for an fp32 one (three), and need all their parts.
    Returns (experts, X, router, ids, hidden activation, Y)."""
    E, h, planes = 3, 256, 2 if out == "bf16" else 3
    while True:
        rng = np.random.default_rng(seed)
        seed += 1000
        experts, row = [], int(rng.integers(inter))
        for _ in range(E):
            gi, gm = H.group_index(h, g, rng, True), H.group_index(inter, g, rng, True)
            gate, up, down = (H.weight(*s, 4, g, rng, i) for s, i in (((inter, h), gi), ((inter, h), gi), ((h, inter), gm)))
            words, zeros = np.zeros_like(gate[0]), np.zeros_like(gate[2])
            words[row], zeros[row] = gate[0][row], gate[2][row]
            experts.append(tuple((w[0], np.ones_like(w[1]), w[2], w[3]) for w in ((words, gate[1], zeros, gi), up, down)))
        top = 1 if out == "bf16" else 6
        X = torch.from_numpy(rng.integers(-top, top + 1, size=(tokens, h)).astype(np.float32)).to(torch.bfloat16)
        R = torch.from_numpy(rng.standard_normal((E, h)).astype(np.float32))
        ids, _ = oracle.route(H.f64(X), H.f64(R), 1, True)
        mid = np.concatenate([oracle.glu(H.f64(X)[t:t + 1], *(tuple(a[row:row + 1] for a in w[:3]) + w[3:]
                                                              for w in experts[e][:2]), h, 4, "none")
                              for t, e in enumerate(ids[:, 0])])
        if np.abs(mid).max() < (2 ** 16 if out == "bf16" else 2 ** 20) and not np.array_equal(parts(mid, planes - 1), mid):
            break
    Y, _, _ = oracle.moe(H.f64(X), H.f64(R), experts, h, inter, 4, 1, "none", True)
    return experts, X, R, ids, mid, Y
