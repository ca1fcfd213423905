"""Every kernel of the layers on packed weights against the oracle, by the path
that the library says a call takes: each tile of the tile kernel, whole, split
along K and mixed, for each width of group; the experts' kernels that read
their rows from memory.  Bounds as in layer_helpers."""
import numpy as np
import pytest
import torch

import layer_helpers as H
import oracle
from layer_paths import linear_path, moe_path

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_14_amd as pq
    pq.lib()
    return pq


# path, tokens, m, n; the last tiles of tokens, rows and chunks are partly empty
LINEAR = [((16, "gather"), 45, 700, 517), ((16, "copied"), 17, 45, 4003), ((32, "split"), 21, 130, 5003),
          ((32, "whole"), 33, 8990, 131), ((64, "split"), 70, 1100, 5003), ((64, "whole"), 70, 10990, 131),
          ((64, "mixed"), 260, 7990, 2003), ((128, "split"), 2990, 45, 6001), ((128, "whole"), 130, 10990, 131),
          ((128, "mixed"), 900, 8990, 1003)]
GLU = [((16, "gather"), 45, 700, 517), ((16, "copied"), 16, 45, 3347), ((32, "split"), 21, 45, 4003),
       ((32, "whole"), 17, 10990, 131), ((32, "mixed"), 18, 18882, 1570), ((64, "split"), 33, 1031, 4003),
       ((64, "whole"), 33, 8990, 131), ((64, "mixed"), 260, 3990, 2003), ((128, "split"), 900, 130, 6001),
       ((128, "whole"), 70, 8990, 131), ((128, "mixed"), 260, 10990, 1103)]


def _name(c):
    return f"{c[0][0]}-{c[0][1]}-{c[1]}x{c[2]}x{c[3]}"


def _integers(rng, shape, top):
    return rng.integers(-top, top + 1, size=shape).astype(np.float32)


def _exact_weight(m, n, g, rng, gidx):
    """Codes 0..15, zero points -60..60, scales 1, 1/2, 1/4, 1/8: with activations
    -4..4 every partial sum is a multiple of 1/8 below 4·75·n < 2^21 for n <=
    6001, held exactly by 24 bits, and so are the sums of x·(16 + q) and of x."""
    return H.weight(m, n, 4, g, rng, gidx, exact=True, zero_lo=-60, zero_hi=61)


@pytest.mark.parametrize("g", [32, 64, 128, -1])
@pytest.mark.parametrize("case", LINEAR, ids=_name)
def test_linear_paths_are_exact_on_exact_inputs(pq, case, g):
    """Bias, activation and residual (in place, in a wider buffer) too, for a
    bf16 and an fp32 result: the oracle's value, rounded once."""
    path, tokens, m, n = case
    assert linear_path(pq.lib(), tokens, m, n, g) == path
    rng = np.random.default_rng(tokens + g)
    w = _exact_weight(m, n, g, rng, H.group_index(n, g, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, g)
    X = torch.from_numpy(_integers(rng, (tokens, n), 4)).to(torch.bfloat16)
    pre = oracle.dequant_matmul(H.f64(X), *w, n, 4)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, out_dtype=torch.float32)
    assert np.array_equal(H.f64(Y), pre)
    bias, res = _integers(rng, m, 100), _integers(rng, (tokens, m), 200)
    for out, bdt in (("fp32", "bf16"), ("bf16", "fp32")):
        buf = torch.full((tokens + 1, m + 5), -7.0, dtype=H.TDT[out], device="cuda")
        y = buf[:tokens, 3:3 + m]
        y.copy_(torch.from_numpy(res))
        pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, bias=torch.from_numpy(bias).to(H.TDT[bdt]).cuda(),
                             activation="relu", residual=y, Y=y)
        want = np.maximum(pre + bias, 0.0) + res
        assert np.array_equal(want, want.astype(np.float32))        # so fp32 holds it, and bf16 is rounded once
        assert torch.equal(y.cpu(), torch.from_numpy(want).to(torch.float32).to(H.TDT[out]))
        y.fill_(-7.0)
        assert torch.all(buf == -7.0)


@pytest.mark.parametrize("g", [32, 64, 128, -1])
@pytest.mark.parametrize("case", GLU, ids=_name)
def test_glu_paths_are_exact_on_exact_inputs(pq, case, g):
    """Both factors are exact, so the fp32 result is their product, rounded once."""
    path, tokens, m, n = case
    assert linear_path(pq.lib(), tokens, m, n, g, gated=True) == path
    rng = np.random.default_rng(tokens + g)
    gidx = H.group_index(n, g, rng, True)
    gate, up = (_exact_weight(m, n, g, rng, gidx) for _ in range(2))
    packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, 4, g)
    X = torch.from_numpy(_integers(rng, (tokens, n), 4)).to(torch.bfloat16)
    bg, bu = _integers(rng, m, 100), _integers(rng, m, 100)
    G, U = (oracle.dequant_matmul(H.f64(X), *w, n, 4) for w in (gate, up))
    buf = torch.full((tokens + 1, m + 5), -7.0, device="cuda")
    y = buf[:tokens, 3:3 + m]
    for act, biased in (("none", False), ("relu", True)):
        b = [torch.from_numpy(v).to(torch.bfloat16).cuda() if biased else None for v in (bg, bu)]
        pq.gptq_w4a16_glu(X.cuda(), packed, m, n, g, activation=act, gate_bias=b[0], up_bias=b[1], Y=y)
        want = oracle.activate(G + bg, act) * (U + bu) if biased else G * U      # exact: 2 x 24 bits in 53
        assert torch.equal(y.cpu(), torch.from_numpy(want.astype(np.float32)))
        y.fill_(-7.0)
        assert torch.all(buf == -7.0)


@pytest.mark.parametrize("case", LINEAR, ids=_name)
def test_linear_paths_match_the_oracle(pq, case):
    path, tokens, m, n = case
    rng = np.random.default_rng(m)
    for bits, g, act, bias, residual, out in ((4, 128, "none", "fp32", "bf16", "fp32"), (3, 32, "gelu", "bf16", "fp32", "bf16")):
        assert linear_path(pq.lib(), tokens, m, n, g) == path
        w = H.weight(m, n, bits, g, rng, H.group_index(n, g, rng, True))
        packed = pq.gptq_w4a16_pack(*H.gpu(w), n, bits, g)
        X, b, r = H.activations(tokens, n, seed=n), H.vector((m,), bias, 5), H.vector((tokens, m), residual, 6)
        Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, bias=b.cuda(), activation=act, residual=r.cuda(),
                                 out_dtype=H.TDT[out])
        ref, bound = H.linear_ref(H.f64(X), w, n, bits, H.f64(b), act, H.f64(r), out)
        H.check(Y, ref, bound, f"linear {_name(case)} {act}", out, H.REL if act == "none" else None)


@pytest.mark.parametrize("case", GLU, ids=_name)
def test_glu_paths_match_the_oracle(pq, case):
    path, tokens, m, n = case
    rng = np.random.default_rng(m)
    for bits, g, act, bias, out in ((4, 128, "silu", "fp32", "fp32"), (2, 32, "gelu_tanh", "bf16", "bf16")):
        assert linear_path(pq.lib(), tokens, m, n, g, gated=True) == path
        gidx = H.group_index(n, g, rng, True)
        gate, up = (H.weight(m, n, bits, g, rng, gidx) for _ in range(2))
        packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, bits, g)
        X, bg, bu = H.activations(tokens, n, seed=n, scale=0.25), H.vector((m,), bias, 5), H.vector((m,), bias, 6)
        Y = pq.gptq_w4a16_glu(X.cuda(), packed, m, n, g, activation=act, gate_bias=bg.cuda(), up_bias=bu.cuda(),
                              out_dtype=H.TDT[out])
        ref, e = H.glu_ref(H.f64(X), gate, up, n, bits, act, H.f64(bg), H.f64(bu))
        H.check(Y, ref, H.rounded(ref, e, out), f"glu {_name(case)} {act}", out)


@pytest.mark.parametrize("gated,case", [(False, c) for c in LINEAR] + [(True, c) for c in GLU],
                         ids=lambda v: _name(v) if isinstance(v, tuple) else "glu" if v else "linear")
def test_tokens_keep_to_their_rows_on_every_path(pq, gated, case):
    """A token of NaN and one of Inf spoil their own rows, the others keep their bits."""
    path, tokens, m, n = case
    g = 64
    assert linear_path(pq.lib(), tokens, m, n, g, gated) == path
    rng = np.random.default_rng(tokens)
    gidx = H.group_index(n, g, rng, True)
    w, v = (H.weight(m, n, 4, g, rng, gidx) for _ in range(2))
    if gated:
        packed = pq.gptq_w4a16_glu_pack(*H.gpu(w[:3]), *H.gpu(v), n, 4, g)
        call = lambda x: pq.gptq_w4a16_glu(x, packed, m, n, g)          # noqa: E731
    else:
        packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, g)
        call = lambda x: pq.gptq_w4a16_linear(x, packed, m, n, g)       # noqa: E731
    X = H.activations(tokens, n, seed=7).cuda()
    B = X.clone()
    bad = sorted({0, tokens // 2, tokens - 1})
    for i, t in enumerate(bad):
        B[t, (7 * i) % n] = float("inf") if i == 1 else float("nan")
    Y, Z = call(X), call(B)
    keep = [t for t in range(tokens) if t not in bad]
    assert torch.isfinite(Y).all() and torch.equal(Y[keep], Z[keep])
    assert not torch.isfinite(Z[bad]).any()


# ---------------------------------------------------------------- experts
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("g", [32, 64, 128, -1])
@pytest.mark.parametrize("tokens,top_k", [(7, 1), (40, 2)])
def test_moe_gate_up_reads_wide_rows_from_memory(pq, tokens, top_k, g, out):
    """Rows of 16392 columns: six tokens of an expert do not fit in LDS."""
    E, hidden, inter = 3, 16392, 70
    rng = np.random.default_rng(tokens + g)
    cfg = pq.MoeConfig(hidden, inter, E, top_k, 4, g, "silu", True)
    path = moe_path(pq.lib(), cfg, tokens, out)
    assert not path["small"] and not path["gate_up_lds"] and path["down_lds"]
    experts = []
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    for e in range(E):
        gi, gm = H.group_index(hidden, g, rng, True), H.group_index(inter, g, rng, True)
        experts.append((H.weight(inter, hidden, 4, g, rng, gi), H.weight(inter, hidden, 4, g, rng, gi),
                        H.weight(hidden, inter, 4, g, rng, gm)))
        gate, up, down = experts[-1]
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(gate[:3]), *H.gpu(up), *H.gpu(down), packed)
    X = H.activations(tokens, hidden, seed=2, scale=0.125)
    R = (H.vector((E, hidden), "fp32", 3) / hidden ** 0.5).to(torch.bfloat16)
    Y, ids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    ref, bound, rids, rwts = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, top_k, "silu", True, out=out)
    assert np.array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(wts.cpu().numpy(), rwts, rtol=2 * H.U)
    H.check(Y, ref, bound, f"wide rows, {tokens} tokens", out, 5 * H.REL)


def _gpu_weight(gen, m, n, g):
    """A random 4-bit weight on the GPU: (qweight, scales, zeros, g_idx)."""
    G = 1 if g == -1 else -(-n // g)
    q = torch.randint(-2 ** 31, 2 ** 31, (m, -(-n // 8)), dtype=torch.int64, device="cuda", generator=gen).to(torch.int32)
    scales = torch.rand(m, G, device="cuda", generator=gen) * 0.048 + 0.002
    zeros = torch.randint(0, 16, (m, G), dtype=torch.int32, device="cuda", generator=gen)
    rank = torch.randperm(n, device="cuda", generator=gen)
    return q, scales, zeros, (rank // (n if g == -1 else g)).to(torch.int32)


def _gpu_dequantized(w, n):
    """In 64 bits, column after column of a word."""
    q, scales, zeros, gidx = w
    out = torch.empty(q.shape[0], 8 * q.shape[1], dtype=torch.float64, device="cuda")
    for i in range(8):
        out[:, i::8] = ((q >> (4 * i)) & 15).double()
    g = gidx.long()
    return (out[:, :n] - zeros.double()[:, g]) * scales.double()[:, g]


@pytest.mark.parametrize("g,hidden,inter,out", [(32, 8200, 23000, "fp32"), (64, 8200, 23000, "fp32"),
                                                (128, 8200, 23000, "fp32"), (-1, 8200, 23000, "fp32"),
                                                (32, 11008, 23990, "bf16"), (64, 11008, 23990, "bf16"),
                                                (-1, 11008, 23990, "bf16")])
def test_moe_down_reads_its_rows_from_memory(pq, g, hidden, inter, out):
    """64 tokens on all of 8 experts so wide that the K slices' results would
    pass 256 MB: the down kernel reads the hidden activation from memory.
    Against 64 bits on the GPU (two experts' weights, in turn).  Relative error
    of a token's row: H.REL for the down product and, with an activation of
    slope up to 1.13 and a gated product between, at most four times that for
    the hidden activation; two bf16 parts of it add 2^-17: 2.8e-5 in all.  A bf16
    result differs from the rounded reference only where a rounding border lies
    between the two.  Borders are 2^-8 of a value apart or more, so at 2.8e-5 of
    the row's mean size that is 2^8·2.8e-5 = 0.7 % of the values of that size,
    and with the smaller ones of a normal distribution up to 4 %."""
    tokens, E = 64, 8
    cfg = pq.MoeConfig(hidden, inter, E, E, 4, g, "silu", True)
    path = moe_path(pq.lib(), cfg, tokens, out)
    assert not path["small"] and not path["down_lds"] and path["slices"] == 1
    gen = torch.Generator(device="cuda").manual_seed(inter + g)
    pairs = []
    for _ in range(2):
        gate, up, down = (_gpu_weight(gen, *s, g) for s in ((inter, hidden), (inter, hidden), (hidden, inter)))
        pairs.append((gate, up[:3] + gate[3:], down))
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    for e in range(E):
        gate, up, down = pairs[e % 2]
        pq.gptq_w4a16_moe_pack(cfg, e, *gate[:3], *up, *down, packed)
    X = H.activations(tokens, hidden, seed=2, scale=0.125).cuda()
    R = (H.vector((E, hidden), "fp32", 3) / hidden ** 0.5).cuda()
    Y, ids, wts = pq.gptq_w4a16_moe(X, R, packed, cfg, out_dtype=H.TDT[out])
    x = X.double()
    p = torch.softmax(x @ R.double().t(), dim=1)
    order = torch.argsort(p, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order)
    assert torch.allclose(wts.double(), p.gather(1, order), rtol=2 * H.U, atol=0)
    ref = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for i, (gate, up, down) in enumerate(pairs):
        a = x @ _gpu_dequantized(gate, hidden).t()
        a = a * torch.sigmoid(a) * (x @ _gpu_dequantized(up, hidden).t())
        ref += p[:, i::2].sum(1, keepdim=True) * (a @ _gpu_dequantized(down, inter).t())
    rel = ((Y.double() - ref).norm(dim=1) / ref.norm(dim=1)).max().item()
    off = (Y != ref.to(Y.dtype)).double().mean().item()
    print(f"down from memory, {out}, groups {g}: row error {rel:.2e}, {off:.2%} off the rounded reference", flush=True)
    if out == "fp32":
        assert rel <= 5 * H.REL
    else:
        assert rel <= 5 * H.REL + 2.0 ** -8 + 2.0 ** -17 and off <= 0.05


@pytest.mark.parametrize("gated,case", [(False, c) for c in LINEAR] + [(True, GLU[4]), (True, GLU[7])],
                         ids=lambda v: _name(v) if isinstance(v, tuple) else "glu" if v else "linear")
def test_graph_replays_on_every_path(pq, gated, case):
    """Captured once, replayed with new inputs, eager calls on another workspace between."""
    path, tokens, m, n = case
    assert linear_path(pq.lib(), tokens, m, n, 64, gated) == path
    rng = np.random.default_rng(m)
    gidx = H.group_index(n, 64, rng, True)
    w, v = (H.weight(m, n, 4, 64, rng, gidx) for _ in range(2))
    if gated:
        packed = pq.gptq_w4a16_glu_pack(*H.gpu(w[:3]), *H.gpu(v), n, 4, 64)
        size, fn = pq.gptq_w4a16_glu_workspace_bytes, pq.gptq_w4a16_glu
    else:
        packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
        size, fn = pq.gptq_w4a16_linear_workspace_bytes, pq.gptq_w4a16_linear
    ws = [torch.full((size(tokens, m, n, 64),), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x, y = torch.zeros(tokens, n, dtype=torch.bfloat16, device="cuda"), torch.empty(tokens, m, device="cuda")
    fn(x, packed, m, n, 64, Y=y, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(x, packed, m, n, 64, Y=y, workspace=ws[0])
    for k in range(4):
        X = H.activations(tokens, n, seed=k).cuda()
        x.copy_(X)
        y.fill_(float("nan"))
        graph.replay()
        want = fn(X, packed, m, n, 64, out_dtype=torch.float32, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.isfinite(want).all() and torch.equal(y, want), f"replay {k}"
