"""The products a model makes with this library's 2/3/4-bit weights: plain forms and cases.

Three operators on the quantizer's output (codes, a scale and a zero point per
row and group, the group of every input column):

  linear  Y = act(X Ŵᵀ + b) + R: a projection with its bias, activation and
          residual, one token to a whole prompt
  glu     Y = act(X Ŵgᵀ + bg) ⊙ (X Ŵuᵀ + bu): the gated half of an MLP
  moe     a whole mixture-of-experts layer for a few tokens: router softmax,
          the top k experts, each expert's gated MLP, the weighted sum

Ŵ[r][c] = (q[r][c] - z[r][g(c)]) · s[r][g(c)].  `run` computes them in
elementary torch operations, or (own) through the library's entry points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def _linear(name, tokens, m, n, bits=4, group=128, order=True, act="none", bias="", residual="", out="bf16"):
    return dict(name=name, op="linear", tokens=tokens, m=m, n=n, bits=bits, group=group, order=order, act=act,
                bias=bias, residual=residual, out=out)


def _glu(name, tokens, m, n, bits=4, group=128, order=True, act="silu", bias="", out="bf16"):
    return dict(name=name, op="glu", tokens=tokens, m=m, n=n, bits=bits, group=group, order=order, act=act,
                bias=bias, out=out)


def _moe(name, tokens, experts, top_k, hidden, inter, bits=4, group=64, order=True, act="silu", renorm=True,
         residual="", out="bf16", router="bf16"):
    return dict(name=name, op="moe", tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter,
                bits=bits, group=group, order=order, act=act, renorm=renorm, residual=residual, out=out,
                router=router)


def listed():
    return [
        # decode, one sequence: the attention output projection added onto the residual stream
        _linear("linear 1 token o_proj", 1, 4096, 4096, residual="bf16"),
        # decode, sixteen sequences: the down projection of the repository's flagship layer
        _linear("linear 16 tokens down_proj", 16, 4096, 11008, residual="bf16"),
        # decode, the largest layer of the repository's workloads (symmetric grid)
        _linear("linear 1 token 8192x29568", 1, 8192, 29568, residual="bf16"),
        # a full decode batch through an MLP with bias and gelu
        _linear("linear 64 tokens bias gelu", 64, 11008, 4096, act="gelu", bias="fp32"),
        # odd and ragged everything, 3 bits, fp32 out (a logits-like head of a small model)
        _linear("linear 37 tokens odd 3-bit", 37, 1031, 1000, bits=3, group=64, act="relu", bias="bf16",
                residual="fp32", out="fp32"),
        # prefill of a prompt: the query projection with its bias
        _linear("linear 2048 tokens q_proj", 2048, 4096, 4096, bias="bf16", residual="bf16"),
        # decode, one sequence: gate and up of the flagship MLP
        _glu("glu 1 token 11008x4096", 1, 11008, 4096),
        # odd sizes, 2 bits, groups of 32, fp32 out
        _glu("glu 61 tokens odd 2-bit", 61, 1003, 517, bits=2, group=32, act="gelu_tanh", bias="fp32", out="fp32"),
        # prefill of a prompt through gate and up
        _glu("glu 2048 tokens 11008x4096", 2048, 11008, 4096),
        # decode, one sequence, few large experts
        _moe("moe 1 token 8 experts", 1, 8, 2, 4096, 11008, residual="bf16"),
        # a decode batch over many small experts
        _moe("moe 64 tokens 64 experts", 64, 64, 6, 2048, 1024, residual="bf16"),
        # odd sizes, whole-row groups, raw softmax weights, fp32 out
        _moe("moe 9 tokens odd", 9, 5, 2, 1000, 333, bits=3, group=-1, renorm=False, act="gelu", out="fp32",
             router="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over its logarithm; every second one a multiple of 128, the rest as they fall."""
    v = _log(rng, lo, hi)
    return max(128, v // 128 * 128) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["linear", "linear", "glu", "moe"])
    bits = rng.choice([4, 4, 3, 2])
    order = rng.random() < 0.7
    out = rng.choice(["bf16", "bf16", "fp32"])
    c = dict(op=op, bits=bits, order=order, out=out)
    if op == "moe":
        experts = rng.choice([4, 8, 16, 32, 64, rng.randint(3, 64)])
        hidden = _size(rng, 256, 4096)
        inter = min(_size(rng, 128, 4096), 128 * 1024 * 1024 // (experts * hidden))
        c.update(tokens=_log(rng, 1, 64), experts=experts, top_k=rng.randint(1, min(8, experts)), hidden=hidden,
                 inter=inter, group=rng.choice([32, 64, 64, 128, -1]), act=rng.choice(["silu", "silu", "gelu"]),
                 renorm=rng.random() < 0.6, residual=rng.choice(["", "bf16", "fp32"]),
                 router=rng.choice(["bf16", "fp32"]))
        return c
    c.update(tokens=_log(rng, 1, 2048), m=_size(rng, 64, 11008), n=_size(rng, 64, 4096 if op == "glu" else 11008),
             group=rng.choice([128, 128, 64, 32, -1]), bias=rng.choice(["", "bf16", "fp32"]))
    if op == "linear":
        c.update(act=rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                 residual=rng.choice(["", "bf16", "fp32"]))
    else:
        c.update(act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))
    return c


# ---------------------------------------------------------------- inputs
def _groups(n, group):
    return 1 if group == -1 else -(-n // group)


def _g_idx(gen, lead, n, group, order):
    """The group of every column: runs of `group` columns in the quantizer's processing order."""
    g = n if group == -1 else group
    if not order:
        return (torch.arange(n, device="cuda") // g).to(torch.int32).expand(*lead, n).contiguous()
    rank = torch.rand(*lead, n, device="cuda", generator=gen).argsort(-1).argsort(-1)
    return (rank // g).to(torch.int32)


def _weight(gen, lead, m, n, bits, group):
    """A quantized weight as the quantizer leaves it: nibble words, scales, zero points.
    Codes are near-normal around the zero point, as those of a trained weight."""
    G, top, W = _groups(n, group), 2 ** bits - 1, -(-n // 8)
    zeros = torch.randint((top + 1) // 2 - (bits > 2), (top + 1) // 2 + 1 + (bits > 2), (*lead, m, G), device="cuda",
                          generator=gen, dtype=torch.int32)
    q = torch.randn(*lead, m, 8 * W, device="cuda", generator=gen)
    q = q.mul_((top + 1) / 5).add_((top + 1) / 2).round_().clamp_(0, top).to(torch.uint8)
    q[..., n:] = 0
    words = (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous().view(torch.int32)
    scales = torch.rand(*lead, m, G, device="cuda", generator=gen).mul_(0.01).add_(0.01)
    return {"qweight": words, "scales": scales, "zeros": zeros}


def _activations(gen, tokens, n):
    """Heavy-tailed activations, one channel in a hundred twenty times as large."""
    x = torch.randn(tokens, n, device="cuda", generator=gen)
    x = x * torch.where(torch.rand(n, device="cuda", generator=gen) < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _vector(gen, shape, dtype):
    return torch.randn(*shape, device="cuda", generator=gen).to(DT[dtype]) if dtype else None


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    T, bits, group = c["tokens"], c["bits"], c["group"]
    s = {"case": c}
    if c["op"] == "moe":
        E, h, f = c["experts"], c["hidden"], c["inter"]
        s["gate"] = _weight(gen, (E,), f, h, bits, group)
        s["up"] = _weight(gen, (E,), f, h, bits, group)
        s["down"] = _weight(gen, (E,), h, f, bits, group)
        s["g_in"] = _g_idx(gen, (E,), h, group, c["order"])
        s["g_mid"] = _g_idx(gen, (E,), f, group, c["order"])
        s["x"] = _activations(gen, T, h)
        s["router"] = (torch.randn(E, h, device="cuda", generator=gen) / math.sqrt(h)).to(DT[c["router"]])
        s["residual"] = _vector(gen, (T, h), c["residual"])
    else:
        m, n = c["m"], c["n"]
        s["w"] = _weight(gen, (), m, n, bits, group)
        s["g_in"] = _g_idx(gen, (), n, group, c["order"])
        s["x"] = _activations(gen, T, n)
        s["bias"] = _vector(gen, (m,), c["bias"])
        if c["op"] == "glu":
            s["w2"] = _weight(gen, (), m, n, bits, group)
            s["bias2"] = _vector(gen, (m,), c["bias"])
        else:
            s["residual"] = _vector(gen, (T, m), c["residual"])
    if own:  # the handle a program keeps for its weights, and its scratch memory
        _keep(s)
    return s


def _keep(s):
    """The weights in the product's layout, packed once when a model is loaded."""
    import post_weight_quantization_14_amd as pq

    c = s["case"]
    T, bits, group = c["tokens"], c["bits"], c["group"]
    if c["op"] == "moe":
        s["cfg"] = pq.MoeConfig(hidden=c["hidden"], inter=c["inter"], experts=c["experts"], top_k=c["top_k"],
                                bits=bits, group_size=group, activation=c["act"], renormalize=c["renorm"])
        s["packed"] = torch.empty(pq.gptq_w4a16_moe_packed_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
        for e in range(c["experts"]):
            g, u, d = ([s[k][f][e] for f in ("qweight", "scales", "zeros")] for k in ("gate", "up", "down"))
            pq.gptq_w4a16_moe_pack(s["cfg"], e, *g, *u, s["g_in"][e], *d, s["g_mid"][e], s["packed"])
        nbytes = pq.gptq_w4a16_moe_workspace_bytes(s["cfg"], T)
    elif c["op"] == "glu":
        g, u = ([s[k][f] for f in ("qweight", "scales", "zeros")] for k in ("w", "w2"))
        s["packed"] = pq.gptq_w4a16_glu_pack(*g, *u, s["g_in"], c["n"], bits, group)
        nbytes = pq.gptq_w4a16_glu_workspace_bytes(T, c["m"], c["n"], group)
    else:
        w = s["w"]
        s["packed"] = pq.gptq_w4a16_pack(w["qweight"], w["scales"], w["zeros"], s["g_in"], c["n"], bits, group)
        nbytes = pq.gptq_w4a16_linear_workspace_bytes(T, c["m"], c["n"], group)
    s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass
def _activate(x, act):
    if act == "relu":
        return torch.clamp_min(x, 0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))
    return x


def _dequantized(w, g_idx, n):
    """Ŵ in 32 bits, for one weight or a stack of them."""
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    q = (w["qweight"].unsqueeze(-1) >> shifts) & 15
    q = q.flatten(-2)[..., :n]
    idx = g_idx.long().unsqueeze(-2).expand(*g_idx.shape[:-1], q.shape[-2], n)
    return (q - w["zeros"].gather(-1, idx)).float() * w["scales"].gather(-1, idx)


def _plain_moe(s):
    c = s["case"]
    T, k, E, h, f = c["tokens"], c["top_k"], c["experts"], c["hidden"], c["inter"]
    x = s["x"].float()
    # which experts are chosen hangs on the last bits of the logits: in 64 bits
    p = torch.softmax(s["x"].double() @ s["router"].double().t(), dim=-1)
    p, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]
    if c["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    wt = p.float()
    if T * k <= E:  # the chosen experts' weights, one copy a pair
        pick = ids.reshape(-1)
        sub = lambda w: {name: t[pick] for name, t in w.items()}  # noqa: E731
        gi, gm = s["g_in"][pick], s["g_mid"][pick]
        xp = x.repeat_interleave(k, 0).unsqueeze(-1)
        a = _activate(torch.bmm(_dequantized(sub(s["gate"]), gi, h), xp), c["act"])
        a = a * torch.bmm(_dequantized(sub(s["up"]), gi, h), xp)
        y = torch.bmm(_dequantized(sub(s["down"]), gm, f), a).view(T, k, h)
        y = (y * wt.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, weighted by what the router gave it
        a = _activate(torch.matmul(_dequantized(s["gate"], s["g_in"], h), x.t()), c["act"])
        a = a * torch.matmul(_dequantized(s["up"], s["g_in"], h), x.t())
        y = torch.bmm(_dequantized(s["down"], s["g_mid"], f), a)
        full = torch.zeros(T, E, device="cuda").scatter_(1, ids, wt)
        y = (y * full.t().unsqueeze(1)).sum(0).t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(DT[c["out"]]).contiguous(), ids.to(torch.int32), wt]


def run(s):
    c = s["case"]
    if own:
        import post_weight_quantization_14_amd as pq

        if c["op"] == "moe":
            return list(pq.gptq_w4a16_moe(s["x"], s["router"], s["packed"], s["cfg"], residual=s["residual"],
                                          out_dtype=DT[c["out"]], workspace=s["workspace"]))
        if c["op"] == "glu":
            return pq.gptq_w4a16_glu(s["x"], s["packed"], c["m"], c["n"], c["group"], activation=c["act"],
                                     gate_bias=s["bias"], up_bias=s["bias2"], out_dtype=DT[c["out"]],
                                     workspace=s["workspace"])
        return pq.gptq_w4a16_linear(s["x"], s["packed"], c["m"], c["n"], c["group"], bias=s["bias"],
                                    activation=c["act"], residual=s["residual"], out_dtype=DT[c["out"]],
                                    workspace=s["workspace"])
    if c["op"] == "moe":
        return _plain_moe(s)
    x = s["x"].float()
    y = x @ _dequantized(s["w"], s["g_in"], c["n"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activate(y, c["act"])
    if c["op"] == "glu":
        u = x @ _dequantized(s["w2"], s["g_in"], c["n"]).t()
        if s["bias2"] is not None:
            u = u + s["bias2"].float()
        y = y * u
    elif s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[c["out"]])


# ---------------------------------------------------------------- 64 bits
def _exact_act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * 0.5 * torch.erfc(-x / math.sqrt(2.0))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x


def _exact_weight(w, g_idx, n):
    """Ŵ in 64 bits, column after column of a word."""
    words = w["qweight"].long() & 0xFFFFFFFF
    q = torch.empty(words.shape[0], words.shape[1] * 8, dtype=torch.float64, device=words.device)
    for i in range(8):
        q[:, i::8] = ((words // 16 ** i) % 16).double()
    g = g_idx.long()
    return (q[:, :n] - w["zeros"].double()[:, g]) * w["scales"].double()[:, g]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, x = s["case"], s["x"].double()
    if c["op"] != "moe":
        y = torch.matmul(x, _exact_weight(s["w"], s["g_in"], c["n"]).t())
        y = _exact_act(y if s["bias"] is None else y + s["bias"].double(), c["act"])
        if c["op"] == "glu":
            u = torch.matmul(x, _exact_weight(s["w2"], s["g_in"], c["n"]).t())
            return y * (u if s["bias2"] is None else u + s["bias2"].double())
        return y if s["residual"] is None else y + s["residual"].double()
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    logits = torch.matmul(x, s["router"].double().t()).cpu()
    ids = torch.empty(T, k, dtype=torch.int32)
    wts = torch.empty(T, k, dtype=torch.float64)
    for t in range(T):
        row = logits[t].tolist()
        top = max(row)
        e = [math.exp(v - top) for v in row]
        chosen = sorted(range(E), key=lambda i: (-row[i], i))[:k]
        total = sum(e[i] for i in chosen) if c["renorm"] else sum(e)
        ids[t] = torch.tensor(chosen, dtype=torch.int32)
        wts[t] = torch.tensor([e[i] / total for i in chosen], dtype=torch.float64)
    y = torch.zeros(T, c["hidden"], dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (v.cuda() for v in torch.nonzero(ids == e, as_tuple=True))
        part = {name: {f: v[e] for f, v in s[name].items()} for name in ("gate", "up", "down")}
        a = _exact_act(x[t] @ _exact_weight(part["gate"], s["g_in"][e], c["hidden"]).t(), c["act"])
        a = a * (x[t] @ _exact_weight(part["up"], s["g_in"][e], c["hidden"]).t())
        a = a @ _exact_weight(part["down"], s["g_mid"][e], c["inter"]).t()
        y.index_add_(0, t, a * wts.cuda()[t, j].unsqueeze(1))
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return [y, ids, wts]


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(m, n, group):
    return m * -(-n // 8) * 4 + m * _groups(n, group) * 8


def work(case):
    c, size = case, {"": 0, "bf16": 2, "fp32": 4}
    T, o = c["tokens"], size[case["out"]]
    if c["op"] == "moe":
        E, k, h, f, g = c["experts"], c["top_k"], c["hidden"], c["inter"], c["group"]
        touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that at least one token is expected to choose
        per = 2 * _weight_bytes(f, h, g) + _weight_bytes(h, f, g) + 4 * (h + f)
        nbytes = touched * per + E * h * size[c["router"]] + T * h * (2 + o + size[c["residual"]]) + T * k * 8
        return {"bytes": nbytes, "flops": 2.0 * T * h * E + 6.0 * T * k * h * f}
    m, n = c["m"], c["n"]
    mats = 2 if c["op"] == "glu" else 1
    nbytes = mats * (_weight_bytes(m, n, c["group"]) + m * size[c["bias"]]) + 4 * n + T * (2 * n + m * o)
    nbytes += T * m * size[c.get("residual", "")]
    return {"bytes": nbytes, "flops": 2.0 * mats * T * m * n}
