"""GPU parity of the layers on packed weights (gptq_w4a16_linear,
gptq_w4a16_glu, gptq_w4a16_moe) against the float64 oracle.  The bounds are
derived in layer_helpers."""
import numpy as np
import pytest
import torch

import layer_helpers as H
import oracle
import workloads
from gpu_helpers import spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_14_amd as pq
    pq.lib()
    return pq


def _cu(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------- linear
LINEAR = [
    # tokens, m, n, bits, group, act-order, activation, bias, residual, out
    (1, 16, 128, 4, 128, True, "none", "", "", "fp32"),
    (1, 1, 1, 4, 32, False, "none", "", "", "fp32"),
    (1, 17, 33, 3, -1, True, "none", "bf16", "bf16", "bf16"),
    (1, 256, 4096, 4, 128, True, "none", "", "bf16", "bf16"),
    (1, 300, 2050, 4, 64, True, "silu", "fp32", "", "fp32"),
    (2, 129, 515, 2, 32, True, "relu", "bf16", "", "fp32"),
    (3, 200, 1100, 4, -1, True, "gelu", "", "fp32", "fp32"),
    (4, 64, 9000, 4, 128, True, "none", "bf16", "fp32", "bf16"),
    (5, 37, 777, 4, 128, False, "gelu_tanh", "fp32", "bf16", "fp32"),
    (8, 400, 640, 3, 64, True, "none", "", "", "fp32"),
    (15, 40, 1300, 4, 32, True, "none", "", "", "fp32"),
    (16, 512, 4096, 4, 128, True, "none", "bf16", "bf16", "bf16"),
    (17, 100, 260, 4, 64, True, "silu", "", "", "bf16"),
    (31, 1031, 1000, 3, 64, True, "relu", "bf16", "fp32", "fp32"),
    (33, 70, 300, 4, -1, False, "none", "", "", "fp32"),
    (48, 130, 384, 2, 128, True, "none", "", "", "fp32"),
    (64, 1000, 1024, 4, 128, True, "gelu", "fp32", "", "bf16"),
    (65, 256, 512, 4, 128, True, "none", "bf16", "bf16", "bf16"),
    (100, 33, 1537, 4, 32, True, "gelu_tanh", "", "", "fp32"),
    (128, 128, 128, 4, 128, False, "none", "", "", "fp32"),
    (129, 300, 700, 3, 64, True, "none", "fp32", "", "fp32"),
    (200, 77, 1000, 4, -1, True, "none", "", "fp32", "fp32"),
    (257, 640, 900, 4, 128, True, "silu", "bf16", "bf16", "bf16"),
    (300, 17, 64, 2, 32, True, "none", "", "", "fp32"),
    (513, 513, 257, 4, 64, False, "relu", "", "bf16", "bf16"),
    (1024, 256, 1024, 4, 128, True, "none", "", "", "fp32"),
    (4103, 20, 96, 4, 32, True, "none", "bf16", "", "fp32"),     # more than one launch sequence
    (1, 17, 90001, 4, 128, True, "none", "", "bf16", "fp32"),    # one token's row beyond LDS
    (3, 40, 33000, 4, 64, True, "none", "", "", "fp32"),
    (7, 64, 11008, 4, 128, True, "silu", "", "", "fp32"),
    (14, 33, 4096, 4, 32, True, "none", "bf16", "", "bf16"),
    (100, 16, 40000, 4, -1, True, "none", "", "", "fp32"),
]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(v) for v in c))
def test_linear_matches_oracle(pq, case):
    tokens, m, n, bits, g, order, act, bias, residual, out = case
    rng = np.random.default_rng(m * 31 + n + tokens)
    w = H.weight(m, n, bits, g, rng, H.group_index(n, g, rng, order))
    X = H.activations(tokens, n, seed=n + tokens, scale=2.0)
    b = H.vector((m,), bias, 5) if bias else None
    r = H.vector((tokens, m), residual, 6) if residual else None
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, bits, g)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, bias=_cu(b), activation=act, residual=_cu(r),
                             out_dtype=H.TDT[out])
    assert Y.dtype == H.TDT[out]
    ref, bound = H.linear_ref(H.f64(X), w, n, bits, H.f64(b), act, H.f64(r), out)
    H.check(Y, ref, bound, f"linear {case}", out, H.REL if act == "none" and tokens * m > 64 else None)


@pytest.mark.parametrize("tokens", [1, 3, 7, 20, 70, 150, 300])
@pytest.mark.parametrize("g", [32, 64, 128, -1])
def test_linear_exact_inputs_match_bit_for_bit(pq, g, tokens):
    """Small-integer activations and power-of-two scales make every sum exact:
    every kernel has to return the oracle's value itself."""
    m, n, bits = 150, 1000, 4
    rng = np.random.default_rng(11 + g)
    w = H.weight(m, n, bits, g, rng, H.group_index(n, g, rng, True), exact=True)
    X = torch.from_numpy(rng.integers(-8, 9, size=(tokens, n)).astype(np.float32)).to(torch.bfloat16)
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, bits, g)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, out_dtype=torch.float32)
    assert np.array_equal(H.f64(Y), oracle.dequant_matmul(H.f64(X), *w, n, bits))


def test_linear_zero_points_outside_the_code_range(pq):
    """The linear quantizer's asymmetric zero points may lie outside [0, 15]."""
    m, n = 40, 300
    rng = np.random.default_rng(3)
    for tokens in (1, 20, 200):
        w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, False), zero_lo=-200, zero_hi=200)
        X = H.activations(tokens, n, seed=4)
        packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
        Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, 64, out_dtype=torch.float32)
        ref, bound = H.linear_ref(H.f64(X), w, n, 4)
        H.check(Y, ref, bound, f"zero points -200..200, {tokens} tokens")


@pytest.mark.parametrize("tokens", [1, 5, 40, 140])
def test_linear_strided_rows_leave_the_padding_alone(pq, tokens):
    m, n = 45, 203
    rng = np.random.default_rng(tokens)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    big = torch.full((tokens + 2, n + 7), float("nan"), dtype=torch.bfloat16, device="cuda")
    X = H.activations(tokens, n, seed=8)
    big[1:1 + tokens, 3:3 + n] = X.cuda()                       # odd row stride, 2-byte aligned rows
    rbuf = torch.full((tokens, m + 5), float("nan"), device="cuda")
    R = H.vector((tokens, m), "fp32", 9)
    rbuf[:, 2:2 + m] = R.cuda()
    ybuf = torch.full((tokens + 2, m + 3), -7.0, dtype=torch.bfloat16, device="cuda")
    pq.gptq_w4a16_linear(big[1:1 + tokens, 3:3 + n], packed, m, n, 64, residual=rbuf[:, 2:2 + m],
                         Y=ybuf[1:1 + tokens, 1:1 + m])
    ref, bound = H.linear_ref(H.f64(X), w, n, 4, residual=H.f64(R), out="bf16")
    H.check(ybuf[1:1 + tokens, 1:1 + m], ref, bound, f"strided, {tokens} tokens", "bf16")
    assert torch.all(ybuf[0] == -7) and torch.all(ybuf[-1] == -7)
    assert torch.all(ybuf[:, 0] == -7) and torch.all(ybuf[:, 1 + m:] == -7)


@pytest.mark.parametrize("tokens", [1, 6, 40, 200])
def test_linear_adds_onto_its_own_residual(pq, tokens):
    m, n = 100, 256
    rng = np.random.default_rng(21)
    w = H.weight(m, n, 4, 128, rng, H.group_index(n, 128, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 128)
    X = H.activations(tokens, n, seed=22)
    R = H.vector((tokens, m), "bf16", 23)
    Y = R.cuda()
    pq.gptq_w4a16_linear(X.cuda(), packed, m, n, 128, residual=Y, Y=Y)
    ref, bound = H.linear_ref(H.f64(X), w, n, 4, residual=H.f64(R), out="bf16")
    H.check(Y, ref, bound, f"in place, {tokens} tokens", "bf16")


@pytest.mark.parametrize("tokens", [1, 4, 16, 64, 300])
def test_a_token_does_not_reach_its_neighbours(pq, tokens):
    """A token of NaN and one of Inf spoil their own rows only, and a token's
    result does not depend on which others are in the batch."""
    m, n = 64, 500
    rng = np.random.default_rng(31)
    w = H.weight(m, n, 4, 128, rng, H.group_index(n, 128, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 128)
    X = H.activations(tokens, n, seed=32).cuda()
    Y = pq.gptq_w4a16_linear(X, packed, m, n, 128)
    B = X.clone()
    B[0, 7] = float("nan")
    if tokens > 1:
        B[tokens // 2, 9] = float("inf")
    Z = pq.gptq_w4a16_linear(B, packed, m, n, 128)
    bad = {0, tokens // 2} if tokens > 1 else {0}
    for t in range(tokens):
        if t in bad:
            assert not torch.isfinite(Z[t]).any()
        else:
            assert torch.equal(Y[t], Z[t])


# ---------------------------------------------------------------- glu
GLU = [
    (1, 16, 128, 4, 128, True, "silu", "", "fp32"),
    (1, 1, 5, 4, 32, False, "none", "fp32", "fp32"),
    (1, 333, 4096, 4, 128, True, "silu", "", "bf16"),
    (2, 50, 700, 3, 64, True, "gelu", "bf16", "fp32"),
    (4, 100, 300, 2, 32, True, "relu", "", "bf16"),
    (7, 48, 515, 4, -1, True, "gelu_tanh", "fp32", "fp32"),
    (16, 520, 1024, 4, 128, True, "silu", "", "bf16"),
    (23, 33, 260, 4, 64, False, "silu", "", "fp32"),
    (61, 1003, 517, 2, 32, True, "gelu_tanh", "fp32", "fp32"),
    (64, 640, 512, 4, 128, True, "silu", "bf16", "bf16"),
    (65, 129, 300, 3, 128, True, "gelu", "", "fp32"),
    (130, 200, 640, 4, -1, True, "silu", "", "fp32"),
    (300, 77, 1000, 4, 64, True, "silu", "fp32", "bf16"),
    (700, 256, 256, 4, 128, False, "relu", "", "fp32"),
]


@pytest.mark.parametrize("case", GLU, ids=lambda c: "-".join(str(v) for v in c))
def test_glu_matches_oracle(pq, case):
    tokens, m, n, bits, g, order, act, bias, out = case
    rng = np.random.default_rng(m * 17 + n + tokens)
    gidx = H.group_index(n, g, rng, order)
    gate, up = (H.weight(m, n, bits, g, rng, gidx) for _ in range(2))
    X = H.activations(tokens, n, seed=n + tokens, scale=0.5)
    bg, bu = ((H.vector((m,), bias, s) for s in (1, 2)) if bias else (None, None))
    packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, bits, g)
    Y = pq.gptq_w4a16_glu(X.cuda(), packed, m, n, g, activation=act, gate_bias=_cu(bg), up_bias=_cu(bu),
                          out_dtype=H.TDT[out])
    ref, e = H.glu_ref(H.f64(X), gate, up, n, bits, act, H.f64(bg), H.f64(bu))
    H.check(Y, ref, H.rounded(ref, e, out), f"glu {case}", out)


def test_glu_takes_one_bias(pq):
    m, n = 40, 200
    rng = np.random.default_rng(2)
    gidx = H.group_index(n, 64, rng, True)
    gate, up = (H.weight(m, n, 4, 64, rng, gidx) for _ in range(2))
    packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, 4, 64)
    X = H.activations(9, n, seed=3)
    b = H.vector((m,), "bf16", 4)
    for kw in ({"gate_bias": b}, {"up_bias": b}):
        Y = pq.gptq_w4a16_glu(X.cuda(), packed, m, n, 64, out_dtype=torch.float32,
                              **{k: v.cuda() for k, v in kw.items()})
        ref, e = H.glu_ref(H.f64(X), gate, up, n, 4, "silu", **{k: H.f64(v) for k, v in kw.items()})
        H.check(Y, ref, H.rounded(ref, e, "fp32"), f"glu with {list(kw)[0]}")


# ---------------------------------------------------------------- moe
def _experts(E, hidden, inter, bits, g, rng, order):
    out = []
    for _ in range(E):
        gi, gm = H.group_index(hidden, g, rng, order), H.group_index(inter, g, rng, order)
        out.append((H.weight(inter, hidden, bits, g, rng, gi), H.weight(inter, hidden, bits, g, rng, gi),
                    H.weight(hidden, inter, bits, g, rng, gm)))
    return out


def _pack(pq, cfg, experts):
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    for e, (gate, up, down) in enumerate(experts):
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(gate[:3]), *H.gpu(up), *H.gpu(down), packed)
    return packed


MOE = [
    # tokens, experts, top_k, hidden, inter, bits, group, act-order, act, renorm, residual, out, router
    (1, 8, 2, 256, 384, 4, 64, True, "silu", True, "bf16", "bf16", "bf16"),
    (1, 1, 1, 1, 1, 4, 32, False, "none", True, "", "fp32", "fp32"),
    (1, 4, 4, 130, 67, 4, 32, True, "gelu", False, "", "fp32", "bf16"),
    (2, 16, 3, 1000, 333, 3, -1, True, "silu", True, "fp32", "fp32", "fp32"),
    (5, 6, 2, 2050, 100, 4, 128, True, "gelu_tanh", True, "", "fp32", "bf16"),
    (9, 5, 2, 300, 1100, 4, 64, True, "silu", False, "bf16", "bf16", "bf16"),
    (16, 64, 6, 128, 128, 4, 64, True, "silu", True, "", "fp32", "bf16"),
    (33, 3, 2, 200, 136, 2, 128, False, "relu", True, "", "fp32", "fp32"),       # more than 16 tokens an expert
    (64, 2, 1, 515, 200, 4, 64, True, "silu", True, "bf16", "bf16", "bf16"),
    (70, 12, 4, 256, 140, 4, 32, True, "silu", True, "", "fp32", "bf16"),        # more than one launch sequence
    (7, 200, 3, 64, 32, 4, 32, True, "silu", True, "", "fp32", "bf16"),          # several words of expert bits
    (2, 1024, 64, 40, 16, 4, 32, False, "relu", False, "", "fp32", "bf16"),      # the largest counts
    (3, 4, 1, 8200, 48, 4, 128, True, "silu", True, "", "fp32", "bf16"),
    (1, 3, 2, 515, 2000, 2, 128, True, "silu", False, "fp32", "fp32", "fp32"),
    (16, 4, 4, 256, 128, 4, 64, True, "silu", True, "bf16", "bf16", "bf16"),     # the most pairs of two launches
    (1, 16, 8, 4096, 256, 4, 64, True, "silu", True, "", "bf16", "bf16"),
    (1, 20, 8, 4096, 256, 4, 64, True, "silu", True, "", "bf16", "bf16"),
    (50, 40, 3, 1024, 64, 4, 64, True, "silu", True, "", "fp32", "fp32"),        # logits in a launch of their own
    (66, 33, 2, 999, 64, 4, 128, True, "silu", False, "", "bf16", "bf16"),
    (20, 3, 2, 4104, 1500, 4, 64, True, "silu", True, "bf16", "bf16", "bf16"),   # a pass that LDS does not hold
]


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(str(v) for v in c))
def test_moe_matches_oracle(pq, case):
    tokens, E, k, hidden, inter, bits, g, order, act, renorm, residual, out, rdt = case
    rng = np.random.default_rng(hidden + 7 * inter + tokens)
    experts = _experts(E, hidden, inter, bits, g, rng, order)
    cfg = pq.MoeConfig(hidden, inter, E, k, bits, g, act, renorm)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=hidden + tokens, scale=0.5)
    R = (H.vector((E, hidden), "fp32", 3) / hidden ** 0.5).to(H.TDT[rdt])
    res = H.vector((tokens, hidden), residual, 4) if residual else None
    Y, ids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, residual=_cu(res), out_dtype=H.TDT[out])
    ref, bound, rids, rwts = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, bits, k, act, renorm, H.f64(res), out)
    assert np.array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(wts.cpu().numpy(), rwts, rtol=2 * H.U)
    H.check(Y, ref, bound, f"moe {case}", out)


@pytest.mark.parametrize("tokens", [5, 40])
def test_moe_ties_go_to_the_lower_expert(pq, tokens):
    E, k, hidden, inter = 9, 4, 64, 32
    rng = np.random.default_rng(1)
    experts = _experts(E, hidden, inter, 4, 32, rng, True)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 32, "silu", True)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=2)
    R = H.vector((E, hidden), "bf16", 3)
    R[4] = R[7]
    R[2] = R[7]
    R[8] = R[1]
    Y, ids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=torch.float32)
    ref, bound, rids, _ = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", True)
    assert np.array_equal(ids.cpu().numpy(), rids)
    H.check(Y, ref, bound, "tied logits")
    same = torch.zeros_like(R)
    _, ids, wts = pq.gptq_w4a16_moe(X.cuda(), same.cuda(), packed, cfg)
    assert torch.equal(ids.cpu(), torch.arange(k, dtype=torch.int32).expand(tokens, k))
    assert torch.all(wts == 0.25)


@pytest.mark.parametrize("tokens,E", [(3, 8), (5, 24), (40, 24)])
def test_moe_router_rows_of_the_types_lowest_value(pq, tokens, E):
    # products of 1e38 and more, of both signs: their sums are finite in 64 bits
    k, hidden, inter = 3, 128, 64
    rng = np.random.default_rng(11)
    experts = _experts(E, hidden, inter, 4, 32, rng, True)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 32, "silu", False)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=12)
    R = H.vector((E, hidden), "bf16", 13)
    R[2] = torch.finfo(torch.bfloat16).min
    R[5] = torch.finfo(torch.bfloat16).min
    Y, ids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=torch.float32)
    ref, bound, rids, rw = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", False)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.max(np.abs(wts.cpu().numpy() - rw)) <= 1e-6
    H.check(Y, ref, bound, "lowest rows")


@pytest.mark.parametrize("tokens,out", [(4, "fp32"), (6, "fp32"), (12, "fp32"), (12, "bf16"), (70, "bf16")])
def test_moe_wide_inner_layer(pq, tokens, out):
    # three tokens' hidden activation fills LDS: the down product's K is sliced;
    # nearly all tokens choose one expert
    E, k, hidden, inter = 2, 1, 64, 8192
    rng = np.random.default_rng(21)
    experts = _experts(E, hidden, inter, 4, 64, rng, True)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 64, "silu", True)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=22).abs()
    X[-1] = -X[-1]
    R = torch.zeros(E, hidden, dtype=torch.bfloat16)
    R[1] = 1.0
    Y, ids, _ = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    assert ids.flatten().tolist() == [1] * (tokens - 1) + [0]
    ref, bound, _, _ = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", True, out=out)
    H.check(Y, ref, bound, "wide inner layer", out=out)


@pytest.mark.parametrize("tokens", [6, 20])
def test_moe_token_of_nan_spoils_its_own_row(pq, tokens):
    E, k, hidden, inter = 8, 2, 128, 96
    rng = np.random.default_rng(5)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 32, "silu", True)
    packed = _pack(pq, cfg, _experts(E, hidden, inter, 4, 32, rng, True))
    X = H.activations(tokens, hidden, seed=6).cuda()
    R = H.vector((E, hidden), "bf16", 7).cuda()
    Y, ids, _ = pq.gptq_w4a16_moe(X, R, packed, cfg)
    B = X.clone()
    B[3, 5] = float("nan")
    Z, zids, _ = pq.gptq_w4a16_moe(B, R, packed, cfg)
    assert torch.equal(zids[3].cpu(), torch.arange(k, dtype=torch.int32))   # all logits NaN: the lowest experts
    assert not torch.isfinite(Z[3]).any()
    keep = [t for t in range(tokens) if t != 3]
    assert torch.equal(Y[keep], Z[keep]) and torch.equal(ids[keep], zids[keep])


@pytest.mark.parametrize("tokens", [4, 11, 90])
def test_moe_strided_rows_and_in_place_residual(pq, tokens):
    E, k, hidden, inter = 6, 2, 203, 77
    rng = np.random.default_rng(8)
    experts = _experts(E, hidden, inter, 4, 64, rng, True)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 64, "silu", True)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=9)
    big = torch.full((tokens, hidden + 6), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 3:3 + hidden] = X.cuda()
    R = H.vector((E, hidden), "bf16", 10)
    res = H.vector((tokens, hidden), "bf16", 11)
    ybuf = torch.full((tokens, hidden + 9), -7.0, dtype=torch.bfloat16, device="cuda")
    y = ybuf[:, 4:4 + hidden]
    y.copy_(res)
    pq.gptq_w4a16_moe(big[:, 3:3 + hidden], R.cuda(), packed, cfg, residual=y, Y=y)
    ref, bound, _, _ = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", True, H.f64(res), "bf16")
    H.check(y, ref, bound, "moe in place, strided", "bf16")
    assert torch.all(ybuf[:, :4] == -7) and torch.all(ybuf[:, 4 + hidden:] == -7)


# ---------------------------------------------------------------- together, as a model runs them
def _quantize(pq, m, n, X, seed, bits=4, g=128):
    W = workloads.gen_weight(spec(m=m, n=n, tokens=1, w_seed=seed), "cuda")
    return W, pq.quantize_layer(W, [X], pq.QuantConfig(bits=bits, group_size=g, desc_act=True))


def _np(o):
    return tuple(o[k].cpu().numpy() for k in ("qweight", "scales", "zeros", "g_idx"))


@pytest.mark.parametrize("tokens", [1, 19, 150])
def test_mlp_block_on_the_quantizers_output(pq, tokens):
    """x + down(silu(gate x) * up x) with weights the quantizer made from
    calibration activations (gate and up share an input), act-order on."""
    hidden, inter = 256, 640
    Xc = workloads.gen_x(spec(m=inter, n=hidden, tokens=2000), "cuda")
    cfg = pq.QuantConfig(bits=4, group_size=128, desc_act=True)
    Wg, Wu = (workloads.gen_weight(spec(m=inter, n=hidden, tokens=1, w_seed=s), "cuda") for s in (1, 2))
    (gate,), (up,) = pq.quantize_shared_input([Wg, Wu], [Xc], [cfg])
    _, down = _quantize(pq, hidden, inter, workloads.gen_x(spec(m=hidden, n=inter, tokens=2000), "cuda"), 3)
    pg = pq.gptq_w4a16_glu_pack(gate["qweight"], gate["scales"], gate["zeros"], up["qweight"], up["scales"],
                                up["zeros"], gate["g_idx"], hidden, 4, 128)
    pd = pq.gptq_w4a16_pack(down["qweight"], down["scales"], down["zeros"], down["g_idx"], inter, 4, 128)
    x = workloads.gen_x(spec(m=1, n=hidden, tokens=tokens, x_seed=77), "cuda")
    mid = pq.gptq_w4a16_glu(x, pg, inter, hidden, 128)
    y = pq.gptq_w4a16_linear(mid, pd, hidden, inter, 128, residual=x)
    ref, e = H.glu_ref(H.f64(x), _np(gate), _np(up), hidden, 4, "silu")
    H.check(mid, ref, H.rounded(ref, e, "bf16"), "gate/up", "bf16")
    ref, bound = H.linear_ref(H.f64(mid), _np(down), inter, 4, residual=H.f64(x), out="bf16")
    H.check(y, ref, bound, "down + residual", "bf16")


def test_moe_layer_on_the_quantizers_output(pq):
    """Experts quantized by GPTQ (gate and up on one input, act-order) and by
    the linear quantizer, packed together."""
    hidden, inter, E, k = 256, 256, 4, 2
    cfg = pq.QuantConfig(bits=4, group_size=64, desc_act=True)
    made = []
    for e in range(E):
        Ws = [workloads.gen_weight(spec(m=m, n=n, tokens=1, w_seed=10 * e + i), "cuda")
              for i, (m, n) in enumerate(((inter, hidden), (inter, hidden), (hidden, inter)))]
        if e % 2 == 0:
            Xc = workloads.gen_x(spec(m=1, n=hidden, tokens=1500, x_seed=e), "cuda")
            (g,), (u,) = pq.quantize_shared_input(Ws[:2], [Xc], [cfg])
            d = pq.quantize_layer(Ws[2], [workloads.gen_x(spec(m=1, n=inter, tokens=1500, x_seed=50 + e), "cuda")], cfg)
        else:
            g, u, d = (pq.rtn_quantize(W, pq.RtnConfig(bits=4, group_size=64, sym=False, clip_ratio=1.0)) for W in Ws)
            for o, n in ((g, hidden), (u, hidden), (d, inter)):
                o["g_idx"] = (torch.arange(n, device="cuda") // 64).to(torch.int32)
        made.append((g, u, d))
    mcfg = pq.MoeConfig(hidden, inter, E, k, 4, 64)
    bare = [tuple({f: v for f, v in o.items() if f != "g_idx" or e % 2 == 0} for o in ex) for e, ex in enumerate(made)]
    packed = pq.moe_pack_experts(mcfg, bare)
    x = workloads.gen_x(spec(m=1, n=hidden, tokens=12, x_seed=99), "cuda")
    R = H.vector((E, hidden), "bf16", 3)
    Y, ids, _ = pq.gptq_w4a16_moe(x, R.cuda(), packed, mcfg, residual=x)
    ref, bound, rids, _ = H.moe_ref(H.f64(x), H.f64(R), [tuple(_np(o) for o in ex) for ex in made], hidden, inter, 4,
                                    k, "silu", True, H.f64(x), "bf16")
    assert np.array_equal(ids.cpu().numpy(), rids)
    H.check(Y, ref, bound, "moe of quantized experts", "bf16")


# ---------------------------------------------------------------- streams, graphs, workspaces
def _three(pq, tokens):
    """The three layers on one set of inputs: a function that runs them, with
    its own workspaces and outputs."""
    hidden, inter, E = 256, 384, 4
    rng = np.random.default_rng(41)
    gidx = H.group_index(hidden, 64, rng, True)
    gate, up = (H.weight(inter, hidden, 4, 64, rng, gidx) for _ in range(2))
    down = H.weight(hidden, inter, 4, 64, rng, H.group_index(inter, 64, rng, True))
    pg = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), hidden, 4, 64)
    pd = pq.gptq_w4a16_pack(*H.gpu(down), inter, 4, 64)
    cfg = pq.MoeConfig(hidden, 128, E, 2, 4, 64)
    pm = _pack(pq, cfg, _experts(E, hidden, 128, 4, 64, rng, True))
    R = H.vector((E, hidden), "bf16", 3).cuda()

    class Run:
        def __init__(self):
            self.x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
            self.mid = torch.empty(tokens, inter, dtype=torch.bfloat16, device="cuda")
            self.h = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
            self.y = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
            self.ids = torch.empty(tokens, 2, dtype=torch.int32, device="cuda")
            self.w = torch.empty(tokens, 2, device="cuda")
            self.ws = torch.empty(max(pq.gptq_w4a16_glu_workspace_bytes(tokens, inter, hidden, 64),
                                      pq.gptq_w4a16_linear_workspace_bytes(tokens, hidden, inter, 64),
                                      pq.gptq_w4a16_moe_workspace_bytes(cfg, tokens)), dtype=torch.uint8, device="cuda")

        def __call__(self, stream=None):
            pq.gptq_w4a16_glu(self.x, pg, inter, hidden, 64, Y=self.mid, workspace=self.ws, stream=stream)
            pq.gptq_w4a16_linear(self.mid, pd, hidden, inter, 64, residual=self.x, Y=self.h, workspace=self.ws,
                                 stream=stream)
            pq.gptq_w4a16_moe(self.h, R, pm, cfg, residual=self.h, Y=self.y, topk_ids=self.ids, topk_weights=self.w,
                              workspace=self.ws, stream=stream)
            return self.y

    return Run


@pytest.mark.parametrize("tokens", [1, 24, 130])
def test_graph_replays_match_eager(pq, tokens):
    """Two graphs that share the packed weights (each its own workspace),
    replayed with new inputs, eager calls and synchronizations between."""
    Run = _three(pq, tokens)
    eager, runs = Run(), [Run(), Run()]
    graphs = []
    for r in runs:
        r.x.copy_(H.activations(tokens, 256, seed=1).cuda())
        r()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r()
        graphs.append(g)
    for k in range(4):
        for i, (r, g) in enumerate(zip(runs, graphs)):
            r.x.copy_(H.activations(tokens, 256, seed=10 * k + i).cuda())
            r.y.fill_(float("nan"))
            g.replay()
        for i, r in enumerate(runs):
            eager.x.copy_(H.activations(tokens, 256, seed=10 * k + i).cuda())
            want = eager().clone()
            torch.cuda.synchronize()
            assert torch.isfinite(want).all()
            assert torch.equal(r.y, want), f"replay {k} of graph {i}"
            assert torch.equal(r.ids, eager.ids) and torch.equal(r.w, eager.w)


@pytest.mark.parametrize("tokens", [1, 24, 130])
def test_two_streams_at_once(pq, tokens):
    """Calls on two streams, each with its own workspace, share the weights."""
    Run = _three(pq, tokens)
    want = []
    for seed in (1, 2):
        r = Run()
        r.x.copy_(H.activations(tokens, 256, seed=seed).cuda())
        want.append(r().clone())
    torch.cuda.synchronize()
    streams, runs = [torch.cuda.Stream() for _ in range(2)], [Run(), Run()]
    for r, seed in zip(runs, (1, 2)):
        r.x.copy_(H.activations(tokens, 256, seed=seed).cuda())
    torch.cuda.synchronize()
    for _ in range(5):
        for r, s in zip(runs, streams):
            r(stream=s)
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(r.y, w)


def test_calls_on_another_stream_allocate_for_it(pq):
    """With stream= given and neither output nor workspace, both come from
    memory that is that stream's: results hold while the current stream reuses
    what it freed."""
    Run = _three(pq, 24)
    r = Run()
    r.x.copy_(H.activations(24, 256, seed=5).cuda())
    want = r().clone()
    m, n = 256, 512
    rng = np.random.default_rng(3)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X = H.activations(40, n, seed=6).cuda()
    ref = pq.gptq_w4a16_linear(X, packed, m, n, 64)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        outs = []
        for _ in range(8):
            outs.append(pq.gptq_w4a16_linear(X, packed, m, n, 64, stream=handle))
            torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
    assert torch.equal(r(), want)


def test_empty_batches_and_small_workspaces(pq):
    m, n = 32, 64
    rng = np.random.default_rng(1)
    w = H.weight(m, n, 4, 32, rng, H.group_index(n, 32, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 32)
    X = H.activations(3, n, seed=1).cuda()
    assert pq.gptq_w4a16_linear(X[:0], packed, m, n, 32).shape == (0, m)
    tiny = torch.empty(16, dtype=torch.uint8, device="cuda")    # too small: the call takes its own
    a = pq.gptq_w4a16_linear(X, packed, m, n, 32, workspace=tiny)
    b = pq.gptq_w4a16_linear(X, packed, m, n, 32)
    assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [1, 16, 64])
def test_full_size_down_projection_agrees_with_the_plain_product(pq, tokens):
    """4096 x 11008: every output against gptq_w4a16_matmul's fp32 result
    (both within their bounds of the oracle; sampled rows against it)."""
    m, n = 4096, 11008
    rng = np.random.default_rng(9)
    gidx = H.group_index(n, 128, rng, True)
    w = H.weight(m, n, 4, 128, rng, gidx)
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 128)
    X = H.activations(tokens, n, seed=5)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, 128, out_dtype=torch.float32)
    P = pq.gptq_w4a16_matmul(X.cuda(), packed, m, n, 128)
    # the plain product's own relative error is held to 1e-4 by its tests
    assert float((Y - P).norm() / P.norm()) <= 1e-4
    rows = np.sort(rng.choice(m, 48, replace=False))
    ws = (w[0][rows], w[1][rows], w[2][rows], gidx)
    ref, bound = H.linear_ref(H.f64(X), ws, n, 4)
    H.check(Y[:, torch.from_numpy(rows).cuda()], ref, bound, f"down projection, {tokens} tokens", rel=H.REL)


@pytest.mark.parametrize("op", ["linear", "glu"])
def test_full_size_prefill(pq, op):
    """300 and 2048 tokens through 4096-wide weights: sampled rows and tokens
    against the oracle, the whole result twice bit for bit."""
    m, n = 4096, 4096
    rng = np.random.default_rng(19)
    gidx = H.group_index(n, 128, rng, True)
    w = [H.weight(m, n, 4, 128, rng, gidx) for _ in range(2 if op == "glu" else 1)]
    if op == "glu":
        packed = pq.gptq_w4a16_glu_pack(*H.gpu(w[0][:3]), *H.gpu(w[1]), n, 4, 128)
    else:
        packed = pq.gptq_w4a16_pack(*H.gpu(w[0]), n, 4, 128)
    rows = np.sort(rng.choice(m, 40, replace=False))
    sub = [(a[0][rows], a[1][rows], a[2][rows], gidx) for a in w]
    for tokens in (300, 2048):
        X = H.activations(tokens, n, seed=tokens, scale=0.25)
        call = (lambda: pq.gptq_w4a16_glu(X.cuda(), packed, m, n, 128, out_dtype=torch.float32)) if op == "glu" else (
            lambda: pq.gptq_w4a16_linear(X.cuda(), packed, m, n, 128, out_dtype=torch.float32))
        Y, Z = call(), call()
        assert torch.equal(Y, Z)
        at = np.sort(rng.choice(tokens, 64, replace=False))
        got = Y[torch.from_numpy(at).cuda()][:, torch.from_numpy(rows).cuda()]
        Xf = H.f64(X)[at]
        if op == "glu":
            ref, e = H.glu_ref(Xf, *sub, n, 4, "silu")
            H.check(got, ref, H.rounded(ref, e, "fp32"), f"glu, {tokens} tokens")
        else:
            ref, bound = H.linear_ref(Xf, sub[0], n, 4)
            H.check(got, ref, bound, f"linear, {tokens} tokens", rel=H.REL)
