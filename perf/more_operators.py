"""Attention beside the library's layers, its cache held in 4 bits: plain forms and cases.

Three operators of a model whose weights the quantizer made, over one paged cache:

  cache   new tokens' keys and values are quantized as they are written, and read back
  attend  attention of the last few tokens of each sequence over its cache (causal,
          grouped heads): one token a sequence in decoding, several when drafts are
          checked, hundreds for a chunk of a long prompt
  prompt  causal attention over whole prompts of different lengths, packed one after the
          other, before any cache

The grid of a group of `group` neighbouring channels x of one token and head, with
lo = min x, hi = max x, a = max |x|:

  s = the smallest bf16 with 15 s >= hi - lo, 4096 s >= a and s >= 2^-100
  z = -round(lo / s),  q = clamp(round(x / s) + z, 0, 15),  x̂ = (q - z) s

Position p of sequence b is in page page_table[b][p // page], row p % page.  The n tokens that a
call brings for sequence b (rows cu[b] .. cu[b + 1]) are the last n of its kv_lens[b].
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def _cache(name, batch, longest, news, kv_heads, dim=128, group=128, page=64, ragged=True, dtype="bf16", out="bf16"):
    """`longest`: tokens of the longest sequence after the write; `news`: at most so many of them are new."""
    return dict(name=name, op="cache", batch=batch, longest=longest, news=news, kv_heads=kv_heads, dim=dim, group=group,
                page=page, ragged=ragged, dtype=dtype, out=out)


def _attend(name, batch, longest, news, heads, kv_heads, dim=128, group=128, page=64, ragged=True):
    return dict(name=name, op="attend", batch=batch, longest=longest, news=news, heads=heads, kv_heads=kv_heads, dim=dim,
                group=group, page=page, ragged=ragged)


def _prompt(name, batch, longest, heads, kv_heads, dim=128, ragged=True, fused=False):
    return dict(name=name, op="prompt", batch=batch, longest=longest, heads=heads, kv_heads=kv_heads, dim=dim,
                ragged=ragged, fused=fused)


def listed():
    return [
        # a decode step of sixteen sequences: one token each into the cache of a 32-head layer of width 4096
        _cache("cache 16 sequences 1 token", 16, 2048, 1, 32),
        # the odd one: few heads, the smallest groups and pages, writes that begin and end inside pages, fp32
        _cache("cache 5 odd fp32", 5, 700, 90, 3, dim=64, group=32, page=16, dtype="fp32", out="fp32"),
        # prompts of 2048 tokens written and read back (a chunk that goes on from an earlier prompt reads them)
        _cache("cache 8 prompts of 2048", 8, 2048, 2048, 8, group=64, ragged=False),
        # decode, one short sequence of a 32-head layer of width 4096
        _attend("attend 1 x 512", 1, 512, 1, 32, 32, ragged=False),
        # decode, one long sequence of a layer of width 8192 with 8 shared heads
        _attend("attend 1 x 32768", 1, 32768, 1, 64, 8, group=64, ragged=False),
        # a full decode batch at every length up to 8192
        _attend("attend 64 ragged", 64, 8192, 1, 32, 8),
        # drafts of up to five tokens checked in seven short sequences, small heads and pages
        _attend("attend 7 odd drafts", 7, 1000, 5, 14, 2, dim=64, group=32, page=16),
        # a chunk of a long prompt over what is cached of it
        _attend("attend chunk of 512", 1, 8192, 512, 32, 8, ragged=False),
        # a question of a few words
        _prompt("prompt 19 tokens", 1, 19, 32, 32, ragged=False),
        # short prompts of every length, small heads in groups of seven, q, k and v slices of one projection
        _prompt("prompt 23 odd", 23, 333, 14, 2, dim=64, fused=True),
        # a calibration sequence's length through a 32-head layer of width 4096
        _prompt("prompt 2048", 1, 2048, 32, 32, ragged=False),
        # long prompts packed together, a layer of width 8192 with 8 shared heads
        _prompt("prompt 6 up to 8192", 6, 8192, 64, 8, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "prompt", "prompt"])
    dim = rng.choice([128, 128, 64])
    kv_heads = rng.choice([8, 8, 4, 2, 1, 3, 32])
    share = rng.choice([1, 4, 8, 7, 3]) if kv_heads < 32 else 1
    c = dict(op=op, kv_heads=kv_heads, dim=dim)
    if op == "prompt":
        c.update(heads=kv_heads * share, fused=rng.random() < 0.5, ragged=rng.random() < 0.7)
        longest = _log(rng, 1, 6000)
        c.update(longest=longest, batch=min(_log(rng, 1, 64), max(1, 12000 // longest)))
        return c
    c.update(group=rng.choice([g for g in (32, 64, 128) if g <= dim]), page=rng.choice([16, 32, 64, 128, 256]),
             ragged=rng.random() < 0.7)
    if op == "cache":
        longest = _log(rng, 1, 8192)
        c.update(longest=longest, batch=min(_log(rng, 1, 64), max(1, 16384 * 8 // (longest * kv_heads))),
                 news=1 if rng.random() < 0.4 else rng.randint(1, longest), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                 out=rng.choice(["bf16", "fp32"]))
        return c
    longest = _log(rng, 1, 32768)
    batch = min(_log(rng, 1, 128), max(1, (1 << 20) // (longest * kv_heads)))
    c.update(longest=longest, batch=batch, heads=kv_heads * share)
    c["news"] = 1 if rng.random() < 0.6 else min(longest, _log(rng, 2, max(2, min(512, (1 << 27) // (longest * batch * kv_heads * share)))))
    return c


def _lengths(c):
    """Each sequence's tokens, and how many of them are new: the same for every seed."""
    rng = random.Random("%(op)s %(batch)d %(longest)d %(kv_heads)d" % c)
    total = [c["longest"]] + [max(1, int(c["longest"] * rng.random())) if c["ragged"] else c["longest"] for _ in range(c["batch"] - 1)]
    if c["op"] == "prompt":
        return total, total
    most = [min(n, c["news"]) for n in total]
    return total, [rng.randint(1, m) if c["ragged"] and m > 1 and b else m for b, m in enumerate(most)]


# ---------------------------------------------------------------- inputs
def _device_ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return _device_ints(at)


def _keys_values(gen, tokens, kv_heads, dim, dtype):
    """Keys have a mean of their own in every channel and a few that are many times larger; values are nearly normal."""
    k = torch.randn(tokens, kv_heads, dim, device="cuda", generator=gen)
    size = torch.where(torch.rand(kv_heads, dim, device="cuda", generator=gen) < 0.03, 6.0, 0.8)
    k = (k + torch.randn(kv_heads, dim, device="cuda", generator=gen)) * size
    v = torch.randn(tokens, kv_heads, dim, device="cuda", generator=gen)
    v = v * torch.where(torch.rand(tokens, kv_heads, 1, device="cuda", generator=gen) < 0.02, 4.0, 0.7)
    return k.to(DT[dtype]), v.to(DT[dtype])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    total, news = _lengths(c)
    H, D = c["kv_heads"], c["dim"]
    s = {"case": c, "total": total, "news": news, "cu": _starts(news)}
    if c["op"] == "prompt":
        T, HQ = sum(total), c["heads"]
        if c["fused"]:  # slices of one projection's output
            x = torch.randn(T, HQ + 2 * H, D, device="cuda", generator=gen).to(torch.bfloat16)
            s["q"], s["k"], s["v"] = x[:, :HQ], x[:, HQ:HQ + H], x[:, HQ + H:]
        else:
            s["q"] = torch.randn(T, HQ, D, device="cuda", generator=gen).to(torch.bfloat16)
            s["k"], s["v"] = _keys_values(gen, T, H, D, "bf16")
        return s
    dtype = c.get("dtype", "bf16")
    per_page = c["page"]
    width = max(-(-n // per_page) for n in total)
    need = sum(-(-n // per_page) for n in total)
    order = torch.randperm(need, device="cuda", generator=gen).to(torch.int32)
    table = torch.zeros(c["batch"], width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(total):
        n = -(-n // per_page)
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["lens"] = table, _device_ints(total)
    k, v = _keys_values(gen, sum(total), H, D, dtype)
    if c["op"] == "attend":
        s["q"] = torch.randn(sum(news), c["heads"], D, device="cuda", generator=gen).mul_(1.5).to(torch.bfloat16)
    _keep(s, need, k, v, _starts(total))
    if c["op"] == "cache":  # what comes in the place of the last of each sequence
        s["k"], s["v"] = _keys_values(gen, sum(news), H, D, dtype)
    if own and c["op"] == "attend":
        import post_weight_quantization_14_amd as pq

        s["workspace"] = torch.empty(pq.gptq_kv_attention_workspace_bytes(s["cfg"], c["heads"], c["batch"], sum(news), max(news)),
                                     dtype=torch.uint8, device="cuda")
    return s


def _keep(s, pages, k, v, cu):
    """The cache that a program holds, with what was written to it before."""
    c = s["case"]
    H, D, P = c["kv_heads"], c["dim"], c["page"]
    if own:
        import post_weight_quantization_14_amd as pq

        s["cfg"] = pq.KvConfig(kv_heads=H, head_dim=D, group_size=c["group"], page_size=P)
        s["pages"] = torch.zeros(pages, pq.gptq_kv_page_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        pq.gptq_kv_append(s["cfg"], k, v, s["pages"], s["table"], s["lens"], cu_seqlens=cu)
        return
    slot = _slots(s, s["total"])
    for name, x in (("k", k), ("v", v)):
        s[name + "_codes"] = torch.zeros(pages * P, H, D // 2, dtype=torch.uint8, device="cuda")
        s[name + "_scale"] = torch.zeros(pages * P, H, D // c["group"], dtype=torch.bfloat16, device="cuda")
        s[name + "_zero"] = torch.zeros(pages * P, H, D // c["group"], dtype=torch.int16, device="cuda")
        for part, rows in zip(x.split(1 << 16), slot.split(1 << 16)):  # 64-bit intermediates, a piece at a time
            _write(s, name, part, rows)


# ---------------------------------------------------------------- one pass
def _slots(s, counts):
    """The rows of the cache that hold the last counts[b] tokens of each sequence, one after the other."""
    n = _device_ints(counts).long()
    b = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(int(sum(counts)), device="cuda") - first[b] + s["lens"].long()[b] - n[b]
    P = s["case"]["page"]
    return s["table"][b, pos // P].long() * P + pos % P


def _write(s, name, x, rows):
    """Quantizes x [tokens, kv heads, dim] into rows of the cache.  In 64 bits: a value half way between two codes goes
    by its last bits."""
    g = x.unflatten(-1, (-1, s["case"]["group"])).double()
    lo, hi, a = g.amin(-1), g.amax(-1), g.abs().amax(-1)
    least = torch.maximum((hi - lo) / 15, a / 4096).clamp_min(2.0 ** -100)
    m, e = torch.frexp(least)
    step = ((e.long() + 1015) << 52).view(torch.float64)  # 2^(e - 8) by its bits: ldexp goes through pow, an ulp off
    scale = torch.ceil(m * 256) * step
    scale = torch.where(scale * 15 < hi - lo, scale + step, scale)
    less = scale - step  # where the quotient was rounded up past a bf16
    scale = torch.where((less * 15 >= hi - lo) & (less * 4096 >= a) & (less >= 2.0 ** -100), less, scale)
    zero = -torch.round(lo / scale)
    q = (torch.round(g / scale.unsqueeze(-1)) + zero.unsqueeze(-1)).clamp_(0, 15).to(torch.uint8).flatten(-2)
    s[name + "_codes"][rows] = q[..., 0::2] | (q[..., 1::2] << 4)
    s[name + "_scale"][rows] = scale.to(torch.bfloat16)
    s[name + "_zero"][rows] = zero.to(torch.int16)


def _read(s, name, rows):
    """The values that rows of the cache stand for, in 32 bits (they need no more than 21)."""
    w = s[name + "_codes"][rows]
    q = torch.stack((w & 15, w >> 4), -1).flatten(-2).unflatten(-1, (-1, s["case"]["group"]))
    x = (q - s[name + "_zero"][rows].unsqueeze(-1)) * s[name + "_scale"][rows].float().unsqueeze(-1)
    return x.flatten(-2)


def _attention(q, k, v, keep):
    """q [.., heads, queries, dim], k and v [.., heads, keys, dim], keep [.., 1, queries, keys], all 32 bits."""
    a = torch.matmul(q, k.transpose(-1, -2)).mul_(q.shape[-1] ** -0.5)
    a = a.masked_fill_(~keep, float("-inf"))
    a = a.sub_(a.amax(-1, keepdim=True)).exp_()
    return torch.matmul(a, v) / a.sum(-1, keepdim=True)


def _plain_attend(s):
    c = s["case"]
    B, H, D, L, n = c["batch"], c["kv_heads"], c["dim"], c["longest"], max(s["news"])
    P, G = c["page"], c["heads"] // c["kv_heads"]
    pos = torch.arange(L, device="cuda")
    rows = s["table"].long()[:, pos // P] * P + pos % P
    k, v = (_read(s, name, rows).transpose(1, 2) for name in "kv")  # [B, H, L, D], positions past a sequence's end masked below
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), count)
    i = torch.arange(len(b), device="cuda") - s["cu"].long()[b]
    q = torch.zeros(B, n, c["heads"], D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    last = s["lens"].long().unsqueeze(1) - count.unsqueeze(1) + torch.arange(n, device="cuda")
    keep = (pos <= last.unsqueeze(-1)).repeat(1, G, 1).unsqueeze(1)
    y = _attention(q, k, v, keep).view(B, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, c["heads"], D)
    return y[b, i].to(torch.bfloat16)


def _plain_prompt(s):
    c = s["case"]
    H, D, G = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    out, at = torch.empty(sum(s["total"]), c["heads"], D, dtype=torch.bfloat16, device="cuda"), 0
    for n in s["total"]:  # one prompt after the other, as many heads at once as 4 GB of weights allow
        q, k, v = (s[name][at:at + n].float().transpose(0, 1) for name in "qkv")
        keep = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(0, H, each := max(1, (1 << 30) // (n * n * G))):
            part = slice(h, h + each)
            y = _attention(q.unflatten(0, (H, G))[part], k[part].unsqueeze(1), v[part].unsqueeze(1), keep)
            out[at:at + n, h * G:(h + each) * G] = y.flatten(0, 1).transpose(0, 1)
        at += n
    return out


def run(s):
    c = s["case"]
    if own:
        import post_weight_quantization_14_amd as pq

        if c["op"] == "prompt":
            return pq.gptq_prompt_attention(s["q"], s["k"], s["v"], s["cu"])
        if c["op"] == "attend":
            return pq.gptq_kv_attention(s["cfg"], s["q"], s["pages"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                        max_queries=max(s["news"]), workspace=s["workspace"])
        pq.gptq_kv_append(s["cfg"], s["k"], s["v"], s["pages"], s["table"], s["lens"], cu_seqlens=s["cu"])
        return list(pq.gptq_kv_read(s["cfg"], s["pages"], s["table"], s["lens"], s["k"].shape[0], cu_seqlens=s["cu"],
                                    out_dtype=DT[c["out"]]))
    if c["op"] == "prompt":
        return _plain_prompt(s)
    if c["op"] == "attend":
        return _plain_attend(s)
    rows = _slots(s, s["news"])
    for name in "kv":
        _write(s, name, s[name], rows)
    return [_read(s, name, rows).to(DT[c["out"]]) for name in "kv"]


# ---------------------------------------------------------------- 64 bits
def _exact_grid(x, group):
    """What the cache stands for after x has been written to it, [tokens, heads, dim] in 64 bits: the smallest step of
    eight bits is found by trying powers of two and their 128 fractions."""
    t, h, d = x.shape
    x = x.double().reshape(t, h, d // group, group)
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    a = torch.maximum(-lo, hi)
    fits = lambda s: (15 * s >= hi - lo) & (4096 * s >= a) & (s >= 2.0 ** -100)  # noqa: E731
    e = torch.floor(torch.log2(torch.clamp(torch.maximum((hi - lo) / 15, a / 4096), min=2.0 ** -100))) - 1
    two = lambda n: ((n.long() + 1023) * (1 << 52)).view(torch.float64)  # noqa: E731  (pow may be an ulp off)
    for _ in range(2):  # the largest power of two below
        e = torch.where(fits(two(e + 1)), e, e + 1)
    low, high = torch.zeros_like(e), torch.full_like(e, 128.0)
    for _ in range(7):
        mid = torch.floor((low + high) / 2)
        ok = fits(two(e) * (1 + mid / 128))
        low, high = torch.where(ok, low, mid), torch.where(ok, mid, high)
    s = torch.where(fits(two(e)), two(e), two(e) * (1 + high / 128))
    zero = -torch.round(lo / s)
    return ((torch.clamp(torch.round(x / s) + zero, 0.0, 15.0) - zero) * s).reshape(t, h, d)


def _exact_rows(q, k, v, first):
    """Attention of query i of one head [queries, dim] over the keys up to first + i."""
    w = q @ k.t() / math.sqrt(q.shape[1])
    ahead = torch.arange(k.shape[0], device=q.device)[None, :] > first + torch.arange(q.shape[0], device=q.device)[:, None]
    return torch.softmax(torch.where(ahead, torch.full_like(w, -math.inf), w), dim=1) @ v


def exact(case, seed):
    c = dict(case)
    total, news = _lengths(c)
    H, D = c["kv_heads"], c["dim"]
    if c["op"] == "prompt":
        s = prepare(case, seed)
        k, v = s["k"], s["v"]
    else:  # the same draws as prepare()'s: page order, keys and values, queries
        gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
        torch.randperm(sum(-(-n // c["page"]) for n in total), device="cuda", generator=gen)
        k, v = _keys_values(gen, sum(total), H, D, c.get("dtype", "bf16"))
    G = c.get("heads", H) // H
    ends = [sum(total[:b + 1]) for b in range(len(total))]
    if c["op"] == "cache":
        new = _keys_values(gen, sum(news), H, D, c["dtype"])
        return [torch.cat([_exact_grid(x, c["group"]) for x in t.split(4096)]) for t in new]
    if c["op"] == "prompt":
        q = s["q"]
    else:
        q = torch.randn(sum(news), c["heads"], D, device="cuda", generator=gen).mul_(1.5).to(torch.bfloat16)
    out, at = torch.empty(sum(news), G * H, D, dtype=torch.float64, device="cuda"), 0
    for e, t, n in zip(ends, total, news):
        kb, vb = k[e - t:e], v[e - t:e]
        if c["op"] == "attend":
            kb, vb = (torch.cat([_exact_grid(x, c["group"]) for x in u.split(4096)]) for u in (kb, vb))
        for h in range(G * H):
            kh, vh = kb[:, h // G].double(), vb[:, h // G].double()
            for i in range(0, n, 2048):
                m = min(n, i + 2048)
                seen = t - n + m
                out[at + i:at + m, h] = _exact_rows(q[at + i:at + m, h].double(), kh[:seen], vh[:seen], t - n + i)
        at += n
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, size = case, {"bf16": 2, "fp32": 4}
    total, news = _lengths(c)
    H, D = c["kv_heads"], c["dim"]
    pairs = sum(n * t - n * (n - 1) // 2 for t, n in zip(total, news))  # a query and a key that it sees
    if c["op"] == "prompt":
        return {"bytes": 4.0 * sum(total) * D * (c["heads"] + H), "flops": 4.0 * pairs * c["heads"] * D}
    row = 2 * H * (D // 2 + D // c["group"] * 4)  # a token's keys and values in the cache
    if c["op"] == "attend":
        return {"bytes": 4.0 * sum(news) * c["heads"] * D + sum(total) * row, "flops": 4.0 * pairs * c["heads"] * D}
    return {"bytes": sum(news) * (2.0 * H * D * (size[c["dtype"]] + size[c["out"]]) + 2 * row), "flops": 10.0 * sum(news) * 2 * H * D}
