"""The layers on packed weights at the ends of their ranges, against the
float64 oracle: activations near the largest finite value, infinities, calls
on the null stream.  Bounds as in layer_helpers."""
import numpy as np
import pytest
import torch

import layer_helpers as H

pytestmark = pytest.mark.gpu

BIG = torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module")
def pq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_14_amd as pq
    pq.lib()
    return pq


def _largest(tokens, n, seed):
    """Activations within a factor of four of the largest bf16 value, the first
    token all at the lowest one."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.rand(tokens, n, generator=g) * 0.75 + 0.25) * BIG * 0.99
    x = (x * torch.where(torch.rand(tokens, n, generator=g) < 0.5, -1.0, 1.0)).to(torch.bfloat16)
    x[0] = -BIG
    return x


def _scaled(w, factor):
    return w[0], (w[1] * np.float32(factor)).astype(np.float32), w[2], w[3]


# The group sums x·(16 + q) and their difference pass fp32's range where the
# results, with scales of 2^-10 of the usual, do not.  One token, tiles of 16 in
# the few-token kernel, inputs too wide for it, a prompt's tiles.
LARGEST = [(1, 130, 600, 4, 128), (20, 130, 600, 3, 32), (40, 130, 5000, 4, 64), (4000, 1100, 600, 4, -1),
           (70, 1100, 5000, 2, 32)]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("case", LARGEST, ids=lambda c: "-".join(map(str, c)))
def test_linear_of_the_largest_activations(pq, case, out):
    tokens, m, n, bits, g = case
    rng = np.random.default_rng(tokens + n)
    w = _scaled(H.weight(m, n, bits, g, rng, H.group_index(n, g, rng, True)), 2.0 ** -10)
    X = _largest(tokens, n, seed=tokens)
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, bits, g)
    Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, out_dtype=H.TDT[out])
    ref, bound = H.linear_ref(H.f64(X), w, n, bits, out=out)
    assert np.abs(ref).max() < 0.5 * BIG
    H.check(Y, ref, bound, f"largest activations {case}", out)


@pytest.mark.parametrize("tokens", [1, 30, 500])
def test_glu_of_the_largest_activations(pq, tokens):
    m, n = 600, 640
    rng = np.random.default_rng(tokens)
    gidx = H.group_index(n, 64, rng, True)
    gate, up = (_scaled(H.weight(m, n, 4, 64, rng, gidx), 2.0 ** -72) for _ in range(2))
    X = _largest(tokens, n, seed=3)
    packed = pq.gptq_w4a16_glu_pack(*H.gpu(gate[:3]), *H.gpu(up), n, 4, 64)
    Y = pq.gptq_w4a16_glu(X.cuda(), packed, m, n, 64, out_dtype=torch.float32)
    ref, e = H.glu_ref(H.f64(X), gate, up, n, 4, "silu")
    assert np.abs(ref).max() < 0.5 * BIG
    H.check(Y, ref, H.rounded(ref, e, "fp32"), "largest activations, glu")


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_moe_of_the_largest_activations(pq, tokens, out):
    """The hidden activation is large too: 1e35 and more."""
    E, k, hidden, inter = 5, 2, 600, 400
    rng = np.random.default_rng(tokens)
    experts = []
    for _ in range(E):
        gi, gm = H.group_index(hidden, 64, rng, True), H.group_index(inter, 64, rng, True)
        experts.append((_scaled(H.weight(inter, hidden, 4, 64, rng, gi), 2.0 ** -72),
                        _scaled(H.weight(inter, hidden, 4, 64, rng, gi), 2.0 ** -72),
                        H.weight(hidden, inter, 4, 64, rng, gm)))
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 64, "silu", True)
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    for e, (gate, up, down) in enumerate(experts):
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(gate[:3]), *H.gpu(up), *H.gpu(down), packed)
    X = _largest(tokens, hidden, seed=5)
    R = H.vector((E, hidden), "fp32", 6) * 1e-39
    Y, ids, wts = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    ref, bound, rids, rwts = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", True, out=out)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert 1e35 < np.abs(ref).max() < 0.5 * BIG
    H.check(Y, ref, bound, "largest activations, moe", out)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_moe_hidden_value_above_the_largest_bf16(pq, tokens, out):
    """A hidden activation between the largest bf16 and the largest fp32 value
    stays finite in its bf16 parts.  One column, codes one above the zero
    points: gate 2^64, up v·2^-64, down v·2^-10, every step exact (three parts
    hold 24 bits; two hold the 16 of the second value)."""
    values = np.array([0x7F7FFFFF if out == "fp32" else 0x7F7FFF00, 0xFF7FF100], dtype=np.uint32).view(np.float32)
    E, k = 2, 1
    one = lambda s: (H.pack_words(np.array([[5]])), np.array([[s]], dtype=np.float32),  # noqa: E731
                     np.array([[4]], dtype=np.int32), np.zeros(1, dtype=np.int32))
    cfg = pq.MoeConfig(1, 1, E, k, 4, 32, "none", True)
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    for e in range(E):
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(one(2.0 ** 64)[:3]), *H.gpu(one(values[e] * np.float32(2.0 ** -64))),
                               *H.gpu(one(2.0 ** -10)), packed)
    X = torch.ones(tokens, 1, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        R = torch.zeros(E, 1, dtype=torch.bfloat16, device="cuda")
        R[e] = 1.0
        Y, ids, _ = pq.gptq_w4a16_moe(X, R, packed, cfg, out_dtype=H.TDT[out])
        assert torch.all(ids == e)
        want = torch.full((tokens, 1), float(values[e]) * 2.0 ** -10, dtype=torch.float32).to(H.TDT[out])
        assert torch.equal(Y.cpu(), want)


# two launches; a router workgroup per token that reads bf16 rows, fp32 rows or
# unaligned ones; logits in a launch of their own
@pytest.mark.parametrize("tokens,E,hidden,rdt", [(1, 8, 96, "bf16"), (3, 8, 96, "fp32"), (70, 9, 136, "bf16"),
                                                 (70, 9, 136, "fp32"), (70, 9, 131, "bf16"), (70, 40, 1000, "bf16"),
                                                 (70, 40, 1000, "fp32")])
def test_moe_routes_a_token_with_an_infinity_by_its_logits(pq, tokens, E, hidden, rdt):
    """x·router with one Inf in x, in any column: the logits are Inf of the
    router's signs, so the experts are chosen by those (ties: the lower one)."""
    k, inter = 3, 32
    rng = np.random.default_rng(7)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, 32, "silu", True)
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    gi, gm = H.group_index(hidden, 32, rng, False), H.group_index(inter, 32, rng, False)
    gate, down = H.weight(inter, hidden, 4, 32, rng, gi), H.weight(hidden, inter, 4, 32, rng, gm)
    for e in range(E):
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(gate[:3]), *H.gpu(gate), *H.gpu(down), packed)
    X = H.activations(tokens, hidden, seed=8)
    R = H.vector((E, hidden), rdt, 9)
    want = np.argsort(-(H.f64(X) @ H.f64(R).T), axis=1, kind="stable")[:, :k]
    for col in (0, 1, 7, 8, hidden // 2, hidden - 1):
        B = X.clone()
        B[tokens // 2, col] = float("inf")
        Y, ids, _ = pq.gptq_w4a16_moe(B.cuda(), R.cuda(), packed, cfg)
        rows = want.copy()
        rows[tokens // 2] = np.argsort(-np.sign(H.f64(R)[:, col]), kind="stable")[:k]
        assert np.array_equal(ids.cpu().numpy(), rows), col
        keep = torch.arange(tokens) != tokens // 2
        assert torch.isfinite(Y.cpu()[keep]).all() and torch.isnan(Y.cpu()[tokens // 2]).all()


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_output_between_the_rows_of_its_input(pq, tokens):
    """X, the residual and Y are column slices of one buffer: none overlaps
    another.  Shifted onto X by one column, the call is refused."""
    m, n = 40, 200
    rng = np.random.default_rng(tokens)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X, R = H.activations(tokens, n, seed=1), H.vector((tokens, m), "bf16", 2)
    for order in (("r", "x", "y"), ("y", "r", "x"), ("x", "y", "r")):
        at, col = {}, 0
        for name in order:
            at[name] = col
            col += n if name == "x" else m
        buf = torch.zeros(tokens, col, dtype=torch.bfloat16, device="cuda")
        x, r, y = (buf[:, at[v]:at[v] + (n if v == "x" else m)] for v in "xry")
        x.copy_(X)
        r.copy_(R)
        pq.gptq_w4a16_linear(x, packed, m, n, 64, residual=r, Y=y)
        ref, bound = H.linear_ref(H.f64(X), w, n, 4, residual=H.f64(R), out="bf16")
        H.check(y, ref, bound, f"slices {order}", "bf16")
        over = buf[:, at["x"]:at["x"] + m]
        with pytest.raises(pq.GptqError, match="overlaps X"):
            pq.gptq_w4a16_linear(x, packed, m, n, 64, Y=over)


def test_memory_of_a_call_belongs_to_the_stream_it_is_given(pq):
    """Output and workspace come from the memory of the stream of the call, of
    the default stream too where it is given as its handle, 0."""
    m, n = 40, 200
    rng = np.random.default_rng(4)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X = H.activations(9, n, seed=5).cuda()
    want = pq.gptq_w4a16_linear(X, packed, m, n, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda.empty_cache()

    def owner(t):
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]

    for stream, handle in ((0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                           (side.cuda_stream, side.cuda_stream)):
        before = {s["address"] for s in torch.cuda.memory_snapshot()}
        Y = pq.gptq_w4a16_linear(X, packed, m, n, 64, stream=stream)
        torch.cuda.synchronize()
        assert owner(Y) == [handle]
        assert {s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] not in before} <= {handle}
        assert torch.equal(Y, want)


@pytest.mark.parametrize("pair", [False, True])
def test_pack_on_another_stream_waits_for_the_memory_it_is_given(pq, pair):
    """The packed weight's memory was freed on the current stream while work on
    it was still to come there."""
    m, n, g = 512, 1024, 64
    rng = np.random.default_rng(6)
    gidx = H.group_index(n, g, rng, True)
    w = H.gpu(H.weight(m, n, 4, g, rng, gidx))
    call = lambda s: (pq.gptq_w4a16_glu_pack(*w[:3], *w, n, 4, g, stream=s) if pair else       # noqa: E731
                      pq.gptq_w4a16_pack(*w, n, 4, g, stream=s))
    want = call(None)
    head, body = want[:256].clone(), want[256:].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for handle in (side, side.cuda_stream):
        was = torch.empty_like(want)
        torch.cuda._sleep(50_000_000)
        was.fill_(255)
        at = was.data_ptr()
        del was
        got = call(handle)
        assert got.data_ptr() == at
        torch.cuda.synchronize()
        assert torch.equal(got[256:], body) and torch.equal(got[:4], head[:4])
        del got


@pytest.mark.parametrize("tokens", [1, 40])
def test_linear_of_the_most_columns(pq, tokens):
    """2^20 columns, the most a call takes: groups of 32 and whole rows."""
    m, n = 17, 1 << 20
    rng = np.random.default_rng(1)
    for g in (32, -1):
        w = H.weight(m, n, 4, g, rng, H.group_index(n, g, rng, True))
        packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, g)
        X = H.activations(tokens, n, seed=2)
        Y = pq.gptq_w4a16_linear(X.cuda(), packed, m, n, g, out_dtype=torch.float32)
        ref, bound = H.linear_ref(H.f64(X), w, n, 4)
        H.check(Y, ref, bound, f"2^20 columns, {tokens} tokens, groups of {g}")
    with pytest.raises(pq.GptqError, match="too large"):
        pq.gptq_w4a16_linear(torch.empty(1, n + 1, dtype=torch.bfloat16, device="cuda"), packed, m, n + 1, 32)


@pytest.mark.parametrize("m,n", [(40, 300), (40, 5003)])
def test_linear_rows_beyond_32_bit_offsets(pq, m, n):
    """Rows 2^27 elements apart: the last of 20 tokens is 2.4e9 in."""
    tokens, ld = 20, 1 << 27
    rng = np.random.default_rng(3)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X, R = H.activations(tokens, n, seed=4), H.vector((tokens, m), "bf16", 5)
    buf = torch.empty((tokens - 1) * ld + n + m, dtype=torch.bfloat16, device="cuda")
    x, y = buf.as_strided((tokens, n), (ld, 1)), buf.as_strided((tokens, m), (ld, 1), n)
    x.copy_(X)
    y.copy_(R)
    pq.gptq_w4a16_linear(x, packed, m, n, 64, residual=y, Y=y)
    ref, bound = H.linear_ref(H.f64(X), w, n, 4, residual=H.f64(R), out="bf16")
    H.check(y, ref, bound, f"rows 2^27 apart, {n} columns", "bf16")


@pytest.mark.parametrize("hidden,inter,E,k,tokens", [(32768, 40, 3, 2, 1), (32768, 40, 3, 2, 9), (32768, 40, 20, 3, 9),
                                                     (40, 32768, 3, 2, 1), (40, 32768, 3, 2, 9), (40, 32768, 2, 1, 30)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_moe_of_the_most_columns(pq, hidden, inter, E, k, tokens, out):
    g = 128
    rng = np.random.default_rng(tokens)
    cfg = pq.MoeConfig(hidden, inter, E, k, 4, g, "silu", True)
    packed = torch.empty(pq.gptq_w4a16_moe_packed_bytes(cfg), dtype=torch.uint8, device="cuda")
    experts = []
    for e in range(E):
        gi, gm = H.group_index(hidden, g, rng, True), H.group_index(inter, g, rng, True)
        experts.append((H.weight(inter, hidden, 4, g, rng, gi), H.weight(inter, hidden, 4, g, rng, gi),
                        H.weight(hidden, inter, 4, g, rng, gm)))
        gate, up, down = experts[-1]
        pq.gptq_w4a16_moe_pack(cfg, e, *H.gpu(gate[:3]), *H.gpu(up), *H.gpu(down), packed)
    X = H.activations(tokens, hidden, seed=5, scale=0.125)
    R = (H.vector((E, hidden), "fp32", 6) / hidden ** 0.5).to(torch.bfloat16)
    Y, ids, _ = pq.gptq_w4a16_moe(X.cuda(), R.cuda(), packed, cfg, out_dtype=H.TDT[out])
    ref, bound, rids, _ = H.moe_ref(H.f64(X), H.f64(R), experts, hidden, inter, 4, k, "silu", True, out=out)
    assert np.array_equal(ids.cpu().numpy(), rids)
    H.check(Y, ref, bound, f"experts of {hidden} x {inter}, {tokens} tokens", out)


@pytest.mark.parametrize("tokens,m,n", [(1, 130, 600), (40, 130, 600), (40, 130, 5003)])
@pytest.mark.parametrize("power", [-100, 80])
def test_linear_scales_exactly_with_its_activations(pq, tokens, m, n, power):
    """Activations times a power of two give results times it, bit for bit: at
    2^-100 the smallest step of a group's sum, held times 2^-12, is 2^-112."""
    rng = np.random.default_rng(tokens)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X = torch.from_numpy(rng.integers(-200, 201, size=(tokens, n)).astype(np.float32)).to(torch.bfloat16).cuda()
    Y = pq.gptq_w4a16_linear(X, packed, m, n, 64, out_dtype=torch.float32)
    Z = pq.gptq_w4a16_linear(X * 2.0 ** power, packed, m, n, 64, out_dtype=torch.float32)
    assert torch.equal(Z, Y * 2.0 ** power)


@pytest.mark.parametrize("tokens,m,n", [(1, 130, 600), (40, 130, 600), (40, 130, 5003)])
def test_linear_of_the_smallest_activations(pq, tokens, m, n):
    """Integers up to 200 times 2^-124: products held times 2^-12 end at fp32's
    smallest step, 2^-149, that is 2^-13 of the activations' own step, each off by
    half of one: n of them are sqrt(n)·2^-14 steps, where the results are about
    sqrt(n)·115·6 steps: 9e-8 of them, and held to ten times that.  Sums of x in
    bf16 parts, which end at 2^-133, must still hold the step itself."""
    rng = np.random.default_rng(tokens)
    w = H.weight(m, n, 4, 64, rng, H.group_index(n, 64, rng, True))
    packed = pq.gptq_w4a16_pack(*H.gpu(w), n, 4, 64)
    X = torch.from_numpy(rng.integers(-200, 201, size=(tokens, n)).astype(np.float32)).to(torch.bfloat16).cuda()
    Y = pq.gptq_w4a16_linear(X, packed, m, n, 64, out_dtype=torch.float32).double()
    Z = pq.gptq_w4a16_linear(X * 2.0 ** -124, packed, m, n, 64, out_dtype=torch.float32).double()
    assert float((Z * 2.0 ** 124 - Y).norm() / Y.norm()) <= 9e-7
