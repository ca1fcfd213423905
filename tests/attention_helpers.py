"""Inputs, references and error bounds of the 4-bit cache and of attention.

u = 2^-24 (fp32 half step), B = 2^-8 (bf16 half step).  For a row with weights
p_j (they sum to 1) over values v_j:

  logits, cache: per group two fp32 chains, Σ q·(128 + c) of exact products and
      Σ q, each addition to at most 2u of the chain's absolute sum whatever the
      matrix core's internal rounding, the second times (128 + z) in one fused step:
      |error| <= (2·dim + 8)·u·s·Σ|q|·(271 + |z|) per group, folds add (dim/32)·u of
      the absolute sum; times scale.
  logits, bf16 keys: (2·dim + 8)·u·scale·Σ|q·k|.
  weights: an error e of every logit changes y by at most (e^(2e) - 1)·Σ p|v|;
      exp2 and its argument add 8u + u·|logit|·4 relative to each weight.
  values, cache: weights times s as two bf16 parts, 2^-16 of p·s; two chains over t
      positions, (2·t + 16)·u·Σ p·s·(271 + |z|).  Where a sequence brings more than 16
      query rows for a key head, weights times s are rounded once instead: both chains
      take the rounded weight w, so that y = Σ w·(c - z) with w = p·s·(1 + d), |d| <= B,
      and that costs B·Σ p·s·|c - z| = B·Σ p|v|.
  values, bf16: a weight is rounded once, B of it: B·Σ p|v|; (2·t + 16)·u·Σ p|v|.
  result: rounded once, B·|y|.

These are worst cases.  In the root mean square a rounding to bf16 is at most
B/sqrt(3) of the value, and independent from one weight to the next:
      |Y - y|_F <= B/sqrt(3)·(|y|_F + |sqrt(Σ p² v²)|_F) (the second term: weights rounded once only),
and MARGIN = 1.1 covers the fp32 parts, which are below 2^-14 of that for the sizes here.
"""
from __future__ import annotations

import numpy as np
import torch

U, B, MARGIN = 2.0 ** -24, 2.0 ** -8, 1.1


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def kept(x, group):
    """(kept values, s, z) of x [.., dim] float64, the oracle's grid in array form (tests pin it to the oracle's)."""
    g = x.reshape(*x.shape[:-1], -1, group)
    lo, hi, a = g.min(-1, keepdims=True), g.max(-1, keepdims=True), np.abs(g).max(-1, keepdims=True)
    need = np.maximum(np.maximum((hi - lo) / 15, a / 4096), 2.0 ** -100)
    m, e = np.frexp(need)
    unit = np.ldexp(1.0, e - 8)
    s = np.ceil(m * 256) * unit
    for t in (s - unit, s + unit):      # a quotient rounded past a bf16
        ok = (15 * t >= hi - lo) & (4096 * t >= a) & (t >= 2.0 ** -100)
        bad = ~((15 * s >= hi - lo) & (4096 * s >= a))
        s = np.where((ok & (t < s)) | (bad & (t > s)), t, s)
    z = -np.rint(lo / s)
    y = (np.clip(np.rint(g / s) + z, 0, 15) - z) * s
    return y.reshape(x.shape), s[..., 0], z[..., 0]


def keys_values(tokens, heads, dim, seed, dtype=torch.bfloat16):
    """Channels with means of their own, a few large; some constant and some zero groups."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(tokens, heads, dim, generator=g) + 2 * torch.randn(heads, dim, generator=g)
    k[..., 3] *= 9
    v = torch.randn(tokens, heads, dim, generator=g)
    if tokens > 2:
        v[2] = 1.7          # constant
        v[1, :, :32] = 0.0
    return k.to(dtype), v.to(dtype)


def starts(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32)


class Pages:
    """A cache of sequences of `total` positions whose unused bytes, table entries
    and pages are garbage: NaN scales, page numbers out of range."""

    def __init__(self, pq, cfg, total, seed=0, spare=3):
        self.pq, self.cfg, self.total = pq, cfg, list(total)
        rng = np.random.default_rng(seed)
        P = cfg.page_size
        counts = [-(-n // P) for n in total]
        self.count = sum(counts) + spare
        order = rng.permutation(self.count)[:sum(counts)]
        width = max(counts + [1]) + 2
        table = rng.choice([-1, self.count, 2 ** 31 - 1, -2 ** 31], size=(len(total), width))
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.bytes = torch.full((self.count, pq.gptq_kv_page_bytes(cfg)), 0xFF, dtype=torch.uint8, device="cuda")
        self.lens = torch.tensor(total, dtype=torch.int32, device="cuda")

    def fill(self, k, v):
        """Every position, from rows packed one sequence after the other."""
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pq.gptq_kv_append(self.cfg, k.cuda(), v.cuda(), self.bytes, self.table, self.lens,
                               cu_seqlens=starts(self.total).cuda(), status=st)
        assert st.item() == 0
        return self

    def read(self, counts=None, **kw):
        counts = self.total if counts is None else counts
        return self.pq.gptq_kv_read(self.cfg, self.bytes, self.table, self.lens, sum(counts),
                                    cu_seqlens=starts(counts).cuda(), **kw)


def reference(q, k, v, scale, total, news, grid=None):
    """(y, worst-case bound, rms bound squared) of rows packed as `news` over keys packed as `total`, float64.
    grid: ((s, z) of keys, (s, z) of values, group) for a cache; k, v are then what it keeps."""
    heads, dim = q.shape[1:]
    share = heads // k.shape[1]
    ys, es, ss = [], [], []
    qa = ka = 0
    once = grid is None or max(news) * share > 16
    for t, n in zip(total, news):
        y, e, s2 = (np.zeros((n, heads, dim)) for _ in range(3))
        for h in range(heads):
            kh, vh = k[ka:ka + t, h // share], v[ka:ka + t, h // share]
            qh = q[qa:qa + n, h]
            seen = np.arange(t)[None, :] <= (t - n + np.arange(n))[:, None]
            x = np.where(seen, scale * (qh @ kh.T), -np.inf)
            top = np.max(x, axis=1, keepdims=True, initial=-1e300)
            p = np.exp(x - top)
            p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
            y[:, h] = p @ vh
            pv = p @ np.abs(vh)
            if grid is None:
                ex = (2 * dim + 8) * U * abs(scale) * (np.abs(qh) @ np.abs(kh).T)
                ev = (2 * t + 16) * U * pv
            else:
                (ks, kz), (vs, vz), group = grid
                ks, kz, vs, vz = (a[ka:ka + t, h // share] for a in (ks, kz, vs, vz))
                qg = np.abs(qh).reshape(n, dim // group, group).sum(-1)                   # [n, groups]
                ex = abs(scale) * U * ((2 * dim + 8) * (qg @ (ks * (271 + np.abs(kz))).T)
                                       + dim / 32 * (np.abs(qh) @ np.abs(kh).T))
                ps = np.repeat(p @ (vs * (271 + np.abs(vz))), group, axis=1)
                ev = (2 * t + 16) * U * ps + 2.0 ** -16 * np.repeat(p @ (vs * (16 + np.abs(vz))), group, axis=1)
            if once:
                ev = ev + B * pv
                s2[:, h] = (p ** 2) @ (vh ** 2)
            ex = np.max(np.where(seen, ex, 0), axis=1, keepdims=True, initial=0)
            xa = np.max(np.where(seen, np.abs(x), 0), axis=1, keepdims=True, initial=0)
            rel = np.expm1(2 * ex) + 16 * U + 8 * U * xa
            e[:, h] = rel * pv + ev
        ys.append(y), es.append(e + B * (np.abs(y) + e) + 1e-37), ss.append(s2)
        qa, ka = qa + n, ka + t
    return np.concatenate(ys), np.concatenate(es), np.concatenate(ss)


def check(got, ref, bound, s2, what):
    g = f64(got)
    err = np.abs(g - ref)
    assert g.shape == ref.shape
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    worst = float(np.max(err / bound)) if ref.size else 0.0
    fro = float(np.linalg.norm(err))
    most = MARGIN * B / 3 ** 0.5 * (np.linalg.norm(ref) + np.sqrt(s2.sum()))
    print(f"{what}: worst error {worst:.3f} of its bound, Frobenius {fro / max(most, 1e-300):.3f} of its", flush=True)
    assert np.all(err <= bound), f"{what}: {int(np.sum(err > bound))} outputs beyond the bound ({worst:.2f}x)"
    assert fro <= most + 1e-30, f"{what}: Frobenius error {fro:.3e}, at most {most:.3e}"
