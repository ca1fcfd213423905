"""The precision that the layers on packed weights promise, beyond the worst-case
bounds: limits of layer_precision, and results that are exact."""
import numpy as np
import pytest
import torch

import layer_helpers as H
import layer_precision as P
from layer_paths import moe_path
from test_gpu_w4a16_layers import GLU, LINEAR, MOE, _cu, _experts, _pack

pytestmark = pytest.mark.gpu

EXACT = [(1, 128), (3, 300), (20, 300), (40, 1000), (40, 8200), (70, 300)]


@pytest.fixture(scope="module")
def pq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_14_amd as pq
    pq.lib()
    return pq


def _check(what, Y, ref, out, rel):
    fro, off = P.errors(Y, ref, out)
    print(f"{what}: rel frob {fro:.2e}, {off:.2%} off the rounded reference", flush=True)
    assert P.within(fro, off, ref.size, out, rel)


@pytest.mark.parametrize("case", [c for c in LINEAR if c[0] * c[1] >= 1000], ids=lambda c: "-".join(map(str, c)))
def test_linear_precision(pq, case):
    tokens, m, n, bits, g, order, act, bias, residual, out = case
    rng = np.random.default_rng(m + n + tokens)
    w = H.weight(m, n, bits, g, rng, H.group_index(n, g, rng, order))
    X = H.activations(tokens, n, seed=n, scale=2.0)
    b = H.vector((m,), bias, 5) if bias else None
    r = H.vector((tokens, m), residual, 6) if residual else None
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, bits, g)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, bias=_cu(b), activation=act, residual=_cu(r),
                             out_dtype=H.TDT[out])
    ref, _ = H.linear_ref(H.f64(X), w, n, bits, H.f64(b), act, H.f64(r), out)
    _check("linear", Y, ref, out, P.GLU)


@pytest.mark.parametrize("case", [c for c in GLU if c[0] * c[1] >= 300], ids=lambda c: "-".join(map(str, c)))
def test_glu_precision(pq, case):
    tokens, m, n, bits, g, order, act, bias, out = case
    rng = np.random.default_rng(m + n + tokens)
    gidx = H.group_index(n, g, rng, order)
    gate, up = (H.weight(m, n, bits, g, rng, gidx) for _ in range(2))
    X = H.activations(tokens, n, seed=n, scale=0.5)
    bg, bu = ((H.vector((m,), bias, s) for s in (1, 2)) if bias else (None, None))
    packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, bits, g)
    Y = pq.gptq_w4a16_glu(X.cuda(), packed, m, n, g, activation=act, gate_bias=_cu(bg), up_bias=_cu(bu),
                          out_dtype=H.TDT[out])
    ref, _ = H.glu_ref(H.f64(X), gate, up, n, bits, act, H.f64(bg), H.f64(bu))
    _check("glu", Y, ref, out, P.GLU)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("case", [c for c in MOE if c[0] * c[3] >= 250], ids=lambda c: "-".join(map(str, c)))
def test_moe_precision(pq, case, out):
    tokens, E, k, hidden, inter, bits, g, order, act, renorm, residual, _, rdt = case
    rng = np.random.default_rng(hidden + inter + tokens)
    experts = _experts(E, hidden, inter, bits, g, rng, order)
    cfg = pq.MoeConfig(hidden, inter, E, k, bits, g, act, renorm)
    packed = _pack(pq, cfg, experts)
    X = H.activations(tokens, hidden, seed=hidden, scale=0.5)
    R = (H.vector((E, hidden), "fp32", 3) / hidden ** 0.5).to(H.TDT[rdt])
    Y, ids, _ = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    ref, _, rids, _ = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, bits, k, act, renorm, None, out)
    assert np.array_equal(ids.cpu().numpy(), rids)
    _check("moe", Y, ref, out, P.MOE)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("g", [32, 64, 128, -1])
@pytest.mark.parametrize("tokens,inter", EXACT)
def test_moe_hidden_activation_keeps_its_bits(pq, tokens, inter, g, out):
    experts, X, R, ids, mid, Y = P.exact_moe(tokens, inter, g, out, seed=tokens + inter)
    cfg = pq.MoeConfig(256, inter, 3, 1, 4, g, "none", True)
    path = moe_path(pq.lib(), cfg, tokens, out)
    assert path["small"] == (tokens == 1 or tokens == 3) and (path["slices"] > 1) == (inter == 8200)
    packed = _pack(pq, cfg, experts)
    got, gids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    assert np.array_equal(gids.cpu().numpy(), ids) and torch.all(wts == 1.0)
    assert torch.equal(got.cpu(), torch.from_numpy(Y).to(torch.float32).to(H.TDT[out]))
