"""The limits of layer_precision notice a hidden activation held in too few
bits: the mistake is planted in the oracle."""
import numpy as np
import pytest
import torch

import layer_helpers as H
import layer_precision as P
import oracle


def _case(tokens, E, k, hidden, inter, bits, g):
    rng = np.random.default_rng(hidden + inter + tokens)
    experts = []
    for _ in range(E):
        gi, gm = H.group_index(hidden, g, rng, True), H.group_index(inter, g, rng, True)
        experts.append((H.weight(inter, hidden, bits, g, rng, gi), H.weight(inter, hidden, bits, g, rng, gi),
                        H.weight(hidden, inter, bits, g, rng, gm)))
    X = H.f64(H.activations(tokens, hidden, seed=hidden, scale=0.5))
    R = H.f64(H.vector((E, hidden), "fp32", 3)) / hidden ** 0.5
    return X, R, experts, hidden, inter, bits, k, "silu", True, None


@pytest.mark.parametrize("case", [(1, 8, 2, 256, 384, 4, 64), (16, 20, 6, 128, 128, 4, 64), (33, 3, 2, 200, 136, 2, 128),
                                  (2, 16, 3, 1000, 333, 3, -1), (20, 3, 2, 1024, 1500, 4, 64)])
def test_one_part_of_the_hidden_activation_is_noticed(case):
    args = _case(*case)
    ref, ids, _ = oracle.moe(*args)
    for out in ("fp32", "bf16"):
        for planes, good in ((1, False), (2, True), (3, True)):
            y = P.moe_with_parts(*args, planes)
            fro, off = P.errors(torch.from_numpy(y).to(H.TDT[out]), ref, out)
            assert P.within(fro, off, ref.size, out, P.MOE) == good, (out, planes, fro, off)


@pytest.mark.parametrize("tokens,inter", [(1, 128), (3, 300), (20, 300), (40, 1000), (40, 8200), (70, 300)])
@pytest.mark.parametrize("out,planes", [("fp32", 3), ("bf16", 2)])
def test_exact_case_needs_all_parts(tokens, inter, out, planes):
    for g in (32, -1):
        experts, X, R, ids, mid, Y = P.exact_moe(tokens, inter, g, out, seed=tokens + inter)
        assert np.array_equal(P.parts(mid, planes), mid) and not np.array_equal(P.parts(mid, planes - 1), mid)
        want = torch.from_numpy(Y).to(torch.float32).to(H.TDT[out])
        assert out == "bf16" or np.array_equal(H.f64(want), Y)
        fewer = P.moe_with_parts(H.f64(X), H.f64(R), experts, 256, inter, 4, 1, "none", True, None, planes - 1)
        assert not torch.equal(torch.from_numpy(fewer).to(torch.float32).to(H.TDT[out]), want)
