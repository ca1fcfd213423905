"""The cache and the attention operators as a decoder layer uses them: after one
another, captured, on other streams, with shared pages and caches beyond 4 GB."""
import numpy as np
import pytest
import torch

import oracle
from attention_helpers import Pages, check, f64, kept, keys_values, reference, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_weight_quantization_14_amd as pq
    pq.lib()
    return pq


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def against_cache(y, q, k, v, cfg, total, news, what):
    """y against the reference over what the cache keeps of k, v (packed as `total`)."""
    g = cfg.head_dim if cfg.group_size == -1 else cfg.group_size
    (kk, ks, kz), (vk, vs, vz) = kept(f64(k), g), kept(f64(v), g)
    check(y, *reference(f64(q), kk, vk, cfg.head_dim ** -0.5, total, news, ((ks, kz), (vs, vz), g)), what)


class Layer:
    """A 4-bit projection to q, k and v of 4, 2 and 2 heads of 64, and one back."""
    heads, kv_heads, dim, width = 4, 2, 64, 256

    def __init__(self, pq, seed):
        self.pq = pq
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = {n: self.packed(torch.randn(m, k, device="cuda", generator=g) * k ** -0.5)
                  for n, m, k in (("qkv", 8 * 64, self.width), ("out", self.width, 4 * 64))}

    def packed(self, W):
        m, n = W.shape
        out = self.pq.rtn_quantize(W, self.pq.RtnConfig(bits=4, group_size=128, sym=False, clip_ratio=1.0))
        gidx = (torch.arange(n, device="cuda", dtype=torch.int32) // 128).to(torch.int32)
        return self.pq.gptq_w4a16_pack(out["qweight"], out["scales"], out["zeros"], gidx, n, 4, 128)

    def project(self, x):
        qkv = self.pq.gptq_w4a16_linear(x, self.w["qkv"], 8 * 64, self.width, 128).view(-1, 8, 64)
        return qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]

    def back(self, y, x):
        return self.pq.gptq_w4a16_linear(y.reshape(-1, 256), self.w["out"], self.width, 256, 128, residual=x)


@pytest.mark.parametrize("side", [False, True])
def test_a_layer_prompts_then_tokens(pq, side):
    """Three prompts through projections, attention and the cache, then six decode steps and one of three drafts."""
    layer, cfg = Layer(pq, 1), pq.KvConfig(2, 64, 32, 16)
    lengths = [37, 5, 128]
    with torch.cuda.stream(torch.cuda.Stream() if side else torch.cuda.current_stream()):
        pages = Pages(pq, cfg, [n + 9 for n in lengths], seed=5)
        g = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn(sum(lengths), 256, device="cuda", generator=g).to(torch.bfloat16)
        cu = starts(lengths).cuda()
        q, k, v = layer.project(x)
        y = pq.gptq_prompt_attention(q, k, v, cu)
        lens = ints(lengths)
        pq.gptq_kv_append(cfg, k, v, pages.bytes, pages.table, lens, cu_seqlens=cu)
        check(y, *reference(f64(q), f64(k), f64(v), 0.125, lengths, lengths), "prompts")
        hidden = layer.back(y, x)
        assert torch.isfinite(hidden).all()
        past = [[t[a:a + n] for a, n in zip((0, 37, 42), lengths)] for t in (k, v)]
        x = hidden[[36, 41, 169]]
        for step, n in enumerate([1] * 6 + [3]):
            x = x.repeat_interleave(n, 0)
            q, k, v = layer.project(x)
            lens += n
            news = [n] * 3
            cu = starts(news).cuda()
            pq.gptq_kv_append(cfg, k, v, pages.bytes, pages.table, lens, cu_seqlens=None if n == 1 else cu)
            y = pq.gptq_kv_attention(cfg, q, pages.bytes, pages.table, lens, cu_seqlens=None if n == 1 else cu, max_queries=n)
            past = [[torch.cat((old, t[b * n:b * n + n])) for b, old in enumerate(p)] for p, t in zip(past, (k, v))]
            against_cache(y, q, torch.cat(past[0]), torch.cat(past[1]), cfg, [len(t) for t in past[0]], news, f"step {step}")
            x = layer.back(y, x)
        torch.cuda.synchronize()


@pytest.mark.parametrize("width", [8, 100])      # one launch, or pieces of a long table that are joined
def test_captured_decode(pq, width):
    """A captured append and attention over lengths that grow on the device, replayed with eager work between."""
    cfg = pq.KvConfig(2, 128, 64, 16)
    total, steps = [20, 50, 90], 6
    seen = [n + steps for n in total]
    k, v = keys_values(sum(seen), 2, 128, seed=3)
    k, v = k.cuda(), v.cuda()
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(steps, 3, 4, 128, device="cuda", generator=g).to(torch.bfloat16)
    at = np.cumsum([0] + seen)
    old = torch.cat([torch.arange(a, a + n) for a, n in zip(at, total)]).cuda()

    def cache():
        pages = Pages(pq, cfg, seen, seed=2)
        table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
        table[:, :min(width, pages.table.shape[1])] = pages.table[:, :width]
        pq.gptq_kv_append(cfg, k[old], v[old], pages.bytes, table, ints(total), cu_seqlens=starts(total).cuda())
        return pages.bytes, table

    want = []
    bytes_, table = cache()
    for i in range(steps):
        rows = torch.tensor([a + n + i for a, n in zip(at, total)], device="cuda")
        lens = ints([n + i + 1 for n in total])
        pq.gptq_kv_append(cfg, k[rows], v[rows], bytes_, table, lens)
        want.append(pq.gptq_kv_attention(cfg, q[i], bytes_, table, lens))
    bytes_, table = cache()
    lens, qs, ks, vs = ints(total), torch.zeros_like(q[0]), torch.zeros_like(k[:3]), torch.zeros_like(v[:3])
    ys = torch.empty_like(qs)
    ws = [torch.empty(pq.gptq_kv_attention_workspace_bytes(cfg, 4, 3, 3), dtype=torch.uint8, device="cuda") for _ in range(2)]
    spare = torch.empty_like(ys)

    def step(w, y):
        pq.gptq_kv_append(cfg, ks, vs, bytes_, table, lens)
        pq.gptq_kv_attention(cfg, qs, bytes_, table, lens, Y=y, workspace=w)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        step(ws[0], ys)
    for i in range(steps):
        rows = torch.tensor([a + n + i for a, n in zip(at, total)], device="cuda")
        qs.copy_(q[i]), ks.copy_(k[rows]), vs.copy_(v[rows])
        ws[0].fill_(0xFF)                       # nothing is kept in it
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys, want[i]), f"replay {i}"
        step(ws[1], spare)                      # eager: the same again
        assert torch.equal(spare, want[i]), f"eager {i}"


def test_captured_prompt_and_read(pq):
    cfg = pq.KvConfig(2, 64, 64, 16)
    k, v = (t.cuda() for t in keys_values(100, 2, 64, seed=8))
    pages = Pages(pq, cfg, [60, 40]).fill(k, v)
    q = torch.zeros(100, 4, 64, dtype=torch.bfloat16, device="cuda")
    cu = starts([60, 40]).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kr, vr = pq.gptq_kv_read(cfg, pages.bytes, pages.table, pages.lens, 100, cu_seqlens=cu)
        y = pq.gptq_prompt_attention(q, kr, vr, cu)
    for seed in range(4):
        q.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        torch.cuda.synchronize()
        want = pq.gptq_prompt_attention(q, *pages.read(), cu)
        assert torch.equal(y, want) and torch.equal(kr, pages.read()[0])


def test_two_streams_at_once(pq):
    """Calls on two streams with workspaces of their own, over one cache."""
    cfg = pq.KvConfig(4, 128, 128, 64)
    total = [4000, 900, 2500]
    k, v = keys_values(sum(total), 4, 128, seed=12)
    pages = Pages(pq, cfg, total).fill(k, v)
    q = [torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(2)]
    want = [pq.gptq_kv_attention(cfg, x, pages.bytes, pages.table, pages.lens) for x in q]
    nbytes = pq.gptq_kv_attention_workspace_bytes(cfg, 8, 3, 3)
    ws = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for j, s in enumerate(streams):
            pq.gptq_kv_attention(cfg, q[j], pages.bytes, pages.table, pages.lens, Y=got[j][i], workspace=ws[j], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for w, ys in zip(want, got) for y in ys)


def test_small_workspace_is_replaced(pq):
    cfg = pq.KvConfig(2, 64, 64, 16)
    k, v = keys_values(1500, 2, 64, seed=14)
    pages = Pages(pq, cfg, [1500]).fill(k, v)
    q = torch.randn(1, 4, 64).to(torch.bfloat16).cuda()
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    a = pq.gptq_kv_attention(cfg, q, pages.bytes, pages.table, pages.lens, workspace=small)
    assert torch.equal(a, pq.gptq_kv_attention(cfg, q, pages.bytes, pages.table, pages.lens)) and not small.any()


# units of a call are at most kv heads x (rows / tile + sequences): 8, 4, 2 and 1 waves each
@pytest.mark.parametrize("batch", [5, 30, 70, 150, 300])
@pytest.mark.parametrize("heads,kv_heads,dim,group,news", [(24, 8, 128, 128, 1), (48, 4, 64, 32, 1), (16, 8, 128, 32, 9),
                                                         (8, 8, 64, 64, 2)])
def test_many_short_sequences(pq, batch, heads, kv_heads, dim, group, news):
    rng = np.random.default_rng(batch + heads)
    total = [int(n) for n in rng.integers(0, 70, batch)]
    total[0] = 130
    new = [min(n, int(rng.integers(1, news + 1))) if news > 1 else 1 for n in total]
    if news == 1:
        total = [max(n, 1) for n in total]
    cfg = pq.KvConfig(kv_heads, dim, group, 16)
    k, v = keys_values(sum(total), kv_heads, dim, seed=batch)
    pages = Pages(pq, cfg, total, batch).fill(k, v)
    q = torch.randn(sum(new), heads, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for width in (pages.table.shape[1], 80):        # positions that the table can hold: up to 1024, and more
        table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        table[:, :pages.table.shape[1]] = pages.table
        y = pq.gptq_kv_attention(cfg, q.cuda(), pages.bytes, table, pages.lens, cu_seqlens=starts(new).cuda(),
                                 max_queries=max(new))
        against_cache(y, q, k, v, cfg, total, new, f"{batch} sequences, table {width}")


@pytest.mark.parametrize("width", [64, 65])
@pytest.mark.parametrize("heads,kv_heads,dim,group,news", [(8, 1, 64, 64, 1), (12, 1, 128, 32, 1), (4, 1, 128, 64, 9)])
def test_either_side_of_the_one_launch_limit(pq, width, heads, kv_heads, dim, group, news):
    total, new = [1024, 3, 500, 993], [news, min(news, 3), news, 1]
    cfg = pq.KvConfig(kv_heads, dim, group, 16)
    k, v = keys_values(sum(total), kv_heads, dim, seed=width)
    pages = Pages(pq, cfg, total).fill(k, v)
    table = torch.full((4, width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[:, :64] = pages.table[:, :64]
    q = torch.randn(sum(new), heads, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    y = pq.gptq_kv_attention(cfg, q.cuda(), pages.bytes, table, pages.lens, cu_seqlens=starts(new).cuda(), max_queries=news)
    against_cache(y, q, k, v, cfg, total, new, f"width {width}")


# up to 256 workgroups of 128 queries (heads of 64: 512) two waves share 32 queries, beyond that each has its own:
# three sequences of 512 tokens are 6 of them a head
@pytest.mark.parametrize("heads,dim", [(1, 128), (42, 128), (43, 128), (1, 64), (85, 64), (86, 64)])
@pytest.mark.parametrize("total", [[512], [300, 212], [65, 383, 64]])
def test_either_form_of_prompts(pq, heads, dim, total):
    """Results, and a NaN value and an infinite key that only the last tokens see."""
    T = sum(total)
    q, k, v = (torch.randn(T, h, dim, generator=torch.Generator().manual_seed(h + dim)).to(torch.bfloat16)
               for h in (heads, 1, 1))
    some = sorted({0, heads // 2, heads - 1})
    ref = reference(f64(q[:, some]), f64(k), f64(v), dim ** -0.5, total, total)
    cu = starts(total).cuda()
    y = pq.gptq_prompt_attention(q.cuda(), k.cuda(), v.cuda(), cu)
    check(y[:, some], *ref, f"{heads} heads of {dim}, {total}")
    last = total[0] - 1
    v[last] = float("nan")
    k[T - 1, 0, 0] = float("inf")
    z = pq.gptq_prompt_attention(q.cuda(), k.cuda(), v.cuda(), cu)
    rest = [i for i in range(T) if i not in (last, T - 1)]
    check(z[rest][:, some], *(r[rest] for r in ref), "but the last")
    assert torch.isnan(z[last]).all()
    again = pq.gptq_prompt_attention(q.cuda(), k.cuda(), v.cuda(), cu)
    assert torch.equal(z.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("heads,kv_heads,dim,group,news", [(8, 2, 128, 64, 1), (24, 2, 64, 32, 1), (8, 2, 128, 128, 9),
                                                         (12, 3, 64, 64, 3)])
@pytest.mark.parametrize("total", [[6000, 40, 1], [700], [33, 2000]])
def test_few_units_of_long_tables(pq, heads, kv_heads, dim, group, news, total):
    """Tables for 65536 positions of the units together and more: pieces are taken by eight waves."""
    new = [min(news, n) for n in total]
    cfg = pq.KvConfig(kv_heads, dim, group, 64)
    k, v = keys_values(sum(total), kv_heads, dim, seed=len(total))
    pages = Pages(pq, cfg, total).fill(k, v)
    table = torch.full((len(total), 600), -1, dtype=torch.int32, device="cuda")
    table[:, :pages.table.shape[1]] = pages.table
    q = torch.randn(sum(new), heads, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    run = lambda: pq.gptq_kv_attention(cfg, q.cuda(), pages.bytes, table, pages.lens,  # noqa: E731
                                       cu_seqlens=starts(new).cuda(), max_queries=news)
    y = run()
    against_cache(y, q, k, v, cfg, total, new, f"{heads} heads, {total}")
    assert torch.equal(y, run())


@pytest.mark.parametrize("most", [1, 2])
def test_the_most_heads(pq, most):
    """4096 query heads of one key head."""
    cfg = pq.KvConfig(1, 64, 64, 16)
    total, new = [40, 7], [most, 1]
    k, v = keys_values(47, 1, 64, seed=20)
    pages = Pages(pq, cfg, total).fill(k, v)
    q = torch.randn(sum(new), 4096, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    y = pq.gptq_kv_attention(cfg, q.cuda(), pages.bytes, pages.table, pages.lens, cu_seqlens=starts(new).cuda(),
                             max_queries=most)
    against_cache(y, q, k, v, cfg, total, new, "4096 heads")
    kd, vd = k.cuda(), v.cuda()
    q = torch.randn(47, 4096, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    y = pq.gptq_prompt_attention(q.cuda(), kd, vd, starts(total).cuda())
    some = [0, 1, 2047, 4095]
    check(y[:, some], *reference(f64(q[:, some]), f64(k), f64(v), 0.125, total, total), "prompt of 4096 heads")


@pytest.mark.parametrize("total,news", [([300, 20], 1), ([300, 20], 9), ([1500], 2)])
def test_queries_of_any_size(pq, total, news):
    """Queries 2^100 times as large with a scale 2^-100 times as large: the same bits."""
    cfg = pq.KvConfig(2, 128, 64, 16)
    k, v = keys_values(sum(total), 2, 128, seed=41)
    pages = Pages(pq, cfg, total).fill(k, v)
    new = [news] * len(total)
    q = torch.randn(sum(new), 8, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    args = (pages.bytes, pages.table, pages.lens, starts(new).cuda(), news)
    y = pq.gptq_kv_attention(cfg, q, *args, scale=0.125)
    for e in (100, -60):
        assert torch.equal(y, pq.gptq_kv_attention(cfg, q * 2.0 ** e, *args, scale=0.125 * 2.0 ** -e))
    cu, kd, vd = starts(total).cuda(), k.cuda(), v.cuda()
    q = torch.randn(sum(total), 8, 128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    y = pq.gptq_prompt_attention(q, kd, vd, cu, scale=0.125)
    for e in (100, -60):
        assert torch.equal(y, pq.gptq_prompt_attention(q * 2.0 ** e, kd, vd, cu, scale=0.125 * 2.0 ** -e))


def test_shared_pages_and_a_sequence_twice(pq):
    """Two sequences over the pages of one prefix, and one sequence listed twice."""
    cfg = pq.KvConfig(2, 128, -1, 16)
    k, v = keys_values(60, 2, 128, seed=22)
    pages = Pages(pq, cfg, [60]).fill(k, v)
    table = pages.table.repeat(3, 1)
    lens = ints([60, 35, 60])
    q = torch.randn(1, 4, 128).to(torch.bfloat16).cuda().repeat(3, 1, 1)
    y = pq.gptq_kv_attention(cfg, q, pages.bytes, table, lens)
    assert torch.equal(y[0], y[2])
    for b, n in ((0, 60), (1, 35)):
        against_cache(y[b:b + 1], q[:1], k[:n], v[:n], cfg, [n], [1], f"prefix of {n}")


def test_a_cache_past_4_gb(pq):
    cfg = pq.KvConfig(32, 128, 128, 256)
    each = pq.gptq_kv_page_bytes(cfg)
    count = (9 << 29) // each + 1
    pages = torch.empty(count, each, dtype=torch.uint8, device="cuda")
    total = [300, 700]
    table = ints([[count - 1, 0, -1], [count // 2, count - 2, count - 3]])
    k, v = keys_values(1000, 32, 128, seed=25)
    cu = starts(total).cuda()
    st = ints([0])
    pq.gptq_kv_append(cfg, k.cuda(), v.cuda(), pages, table, ints(total), cu_seqlens=cu, status=st)
    kr, vr = pq.gptq_kv_read(cfg, pages, table, ints(total), 1000, cu_seqlens=cu, out_dtype=torch.float32, status=st)
    kk, vk = kept(f64(k), 128)[0], kept(f64(v), 128)[0]
    assert st.item() == 0 and np.array_equal(f64(kr), kk) and np.array_equal(f64(vr), vk)
    q = torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    y = pq.gptq_kv_attention(cfg, q.cuda(), pages, table, ints(total))
    some = [0, 31]
    against_cache(y[:, some], q[:, some], k[:, some], v[:, some], cfg, total, [1, 1], "past 4 GB")


@pytest.mark.parametrize("ld", [1 << 22, (1 << 23) + 8])
def test_rows_far_apart(pq, ld):
    """Tokens whose rows lie 8 and 16 MB apart: offsets beyond 32 bits."""
    T = (5 << 29) // ld
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    x = big.view(T, ld)[:, :8 * 64].view(T, 8, 64)
    near = torch.randn(T, 8, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    x.copy_(near)
    cu = starts([T - 9, 9]).cuda()
    parts = lambda t: (t[:, :4], t[:, 4:6], t[:, 6:])  # noqa: E731
    want = pq.gptq_prompt_attention(*parts(near), cu)
    check(want, *reference(*(f64(t) for t in parts(near)), 0.125, [T - 9, 9], [T - 9, 9]), "near")
    assert torch.equal(pq.gptq_prompt_attention(*parts(x), cu), want)
    cfg = pq.KvConfig(2, 64, 64, 16)
    pages = Pages(pq, cfg, [T - 9, 9])
    out = []
    for t in (near, x):
        q, k, v = parts(t)
        pages.fill(k, v)
        y = torch.empty_like(near[:, :4])
        out.append((pages.read()[0], pq.gptq_kv_attention(cfg, q, pages.bytes, pages.table, pages.lens, cu_seqlens=cu, Y=y)))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_an_oracle_of_the_whole_path(pq):
    """One prompt appended and one token decoded against the oracle in words."""
    cfg = pq.KvConfig(1, 64, 32, 16)
    k, v = keys_values(21, 1, 64, seed=31)
    pages = Pages(pq, cfg, [21]).fill(k, v)
    q = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    y = pq.gptq_kv_attention(cfg, q.cuda(), pages.bytes, pages.table, pages.lens)
    kk, vk = (np.stack([oracle.kv_kept(f64(t)[i, 0], 32) for i in range(21)])[:, None] for t in (k, v))
    ref = oracle.attention(f64(q), kk, vk, 0.125, [20])
    # the result is rounded once: half a step, 2^-8, and the fp32 chains are far below another 2^-12 of the largest
    assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * np.abs(ref).max())


def test_refusals_in_words(pq):
    """What the calls say of tensors that do not fit, before anything is launched."""
    cfg = pq.KvConfig(2, 64, 32, 16)
    k, v = (t.cuda() for t in keys_values(20, 2, 64, seed=50))
    pages = Pages(pq, cfg, [20]).fill(k, v)
    q = torch.randn(1, 4, 64).to(torch.bfloat16).cuda()
    fits = dict(pages=pages.bytes, page_table=pages.table, kv_lens=pages.lens)
    bad = [("page_table", pages.table.long(), "page_table"), ("page_table", pages.table[0], "page_table"),
           ("page_table", pages.table.repeat(1, 2)[:, ::2], "contiguous rows"), ("page_table", pages.table.cpu(), "page_table is on"),
           ("kv_lens", ints([20, 20]), "kv_lens"), ("kv_lens", pages.lens.long(), "kv_lens"), ("kv_lens", pages.lens[0], "kv_lens"),
           ("pages", pages.bytes[:, ::2], "pages must be contiguous"), ("pages", pages.bytes.cpu(), "pages is on")]
    before = pages.bytes.clone()
    for name, t, match in bad:
        kw = {**fits, name: t}
        for call in (lambda: pq.gptq_kv_attention(cfg, q, **kw), lambda: pq.gptq_kv_append(cfg, k[:1], v[:1], **kw),
                     lambda: pq.gptq_kv_read(cfg, tokens=1, **kw)):
            with pytest.raises(ValueError, match=match if name != "pages" or "on" not in match else "on"):
                call()
    for cu in (ints([0, 1, 2]), ints([0, 1]).long(), ints([0, 1]).cpu()):
        with pytest.raises(ValueError):
            pq.gptq_kv_attention(cfg, q, **fits, cu_seqlens=cu)
    for kw, error in ((dict(status=ints([0, 0])), ValueError), (dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)), ValueError),
                      (dict(Y=torch.empty(1, 4, 64, device="cuda")), TypeError), (dict(Y=q), pq.GptqError),
                      (dict(scale=float("nan")), pq.GptqError), (dict(max_queries=-1), pq.GptqError)):
        with pytest.raises(error):
            pq.gptq_kv_attention(cfg, q, **fits, **kw)
    odd = torch.zeros(pages.bytes.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view_as(pages.bytes)
    with pytest.raises(pq.GptqError, match="16-byte"):
        pq.gptq_kv_attention(cfg, q, **{**fits, "pages": odd})
    with pytest.raises(pq.GptqError, match="table 0 wide"):
        pq.gptq_kv_attention(cfg, q, **{**fits, "page_table": pages.table[:, :0]})
    with pytest.raises(pq.GptqError, match="one token a sequence"):
        pq.gptq_kv_append(cfg, k[:3], v[:3], **fits)
    torch.cuda.synchronize()
    assert torch.equal(before, pages.bytes)
