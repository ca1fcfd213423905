// extern "C" entry points of the 4-bit key/value cache and of the attention
// operators: every argument is checked on the host before any HIP call.
#include <cmath>

#include "attention.hpp"

using namespace gptq;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 27;   // rows of a call
constexpr int64_t kMaxBatch = int64_t(1) << 16;   // workgroups look for their sequence 64 at a time
constexpr int kMaxHeads = 4096;

template <class... A>
gptq_status fail(gptq_status st, const char* fmt, A... a) {
  set_error(fmt, a...);
  return st;
}

bool bad_ptr(const void* p, size_t align) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % align != 0; }

gptq_status check_kv_config(const gptq_kv_config* c) {
  if (c == nullptr) return fail(GPTQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->kv_heads <= 0) return fail(GPTQ_ERR_INVALID_ARG, "kv_heads=%d", c->kv_heads);
  if (c->kv_heads > kMaxHeads) return fail(GPTQ_ERR_UNSUPPORTED, "kv_heads=%d above %d", c->kv_heads, kMaxHeads);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(GPTQ_ERR_UNSUPPORTED, "head_dim=%d (built: 64, 128)", c->head_dim);
  const int g = c->group_size;
  if (!(g == -1 || g == 32 || g == 64 || g == 128) || g > c->head_dim)
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 up to head_dim, or -1)", g);
  const int p = c->page_size;
  if (p < 16 || p > 65536 || (p & (p - 1)) != 0)
    return fail(GPTQ_ERR_UNSUPPORTED, "page_size=%d (a power of two, 16 to 65536)", p);
  return GPTQ_OK;
}

// a [tokens][heads][dim] tensor
gptq_status check_rows(const char* name, const void* p, int32_t dtype, int64_t tokens, int64_t heads, int dim,
                       int64_t ld, int64_t hs, HeadRows* out) {
  const int size = dtype == GPTQ_FP32 ? 4 : 2;
  if (bad_ptr(p, size)) return fail(GPTQ_ERR_INVALID_ARG, "%s is NULL or misaligned", name);
  if (tokens == 1) ld = 0;
  if (heads == 1) hs = 0;
  // strides may be in either order (heads before tokens too) but rows may not overlap, nor bytes pass 62 bits
  const int64_t most = INT64_MAX / 16;
  if (ld < 0 || hs < 0 || (tokens > 1 && ld > most / tokens) || (heads > 1 && hs > most / heads))
    return fail(GPTQ_ERR_INVALID_ARG, "%s: strides %lld, %lld", name, (long long)ld, (long long)hs);
  if ((tokens > 1 && ld < dim) || (heads > 1 && hs < dim) ||
      (tokens > 1 && heads > 1 && ld < (heads - 1) * hs + dim && hs < (tokens - 1) * ld + dim))
    return fail(GPTQ_ERR_INVALID_ARG, "%s: rows of %d overlap with strides %lld, %lld", name, dim, (long long)ld,
                (long long)hs);
  const int64_t step = 16 / size;
  *out = HeadRows{p, ld, hs, reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % step == 0 && hs % step == 0};
  return GPTQ_OK;
}

// times log2(e), as the kernels take it
gptq_status check_scale(float scale) {
  if (!std::isfinite(scale * 1.44269504088896340736f))
    return fail(GPTQ_ERR_INVALID_ARG, "scale=%g: it or log2(e) times it is not finite", (double)scale);
  return GPTQ_OK;
}

struct Span {
  const void* p;
  int64_t bytes;   // from the first to past the last
};
Span span_of(const HeadRows& r, int64_t tokens, int64_t heads, int dim, int size) {
  return Span{r.p, ((tokens - 1) * r.ld + (heads - 1) * r.hs + dim) * size};
}
bool meet(const Span& a, const Span& b) {
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  return d < a.bytes && -d < b.bytes;
}
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a ^ b) < 0); }
// Whether |d + o·S + i·s| < w for some o in o0 .. o1, i in i0 .. i1 (S >= s > 0, or 0 where its range is only 0).
// Rows of a tensor do not overlap, so S is at least the inner rows' span and few o come into question.
bool near_zero(int64_t d, int64_t S, int64_t o0, int64_t o1, int64_t s, int64_t i0, int64_t i1, int64_t w) {
  if (S > 0) {
    o0 = std::max(o0, floor_div(-w - i1 * s - d, S));
    o1 = std::min(o1, floor_div(w - i0 * s - d, S) + 1);
  }
  for (int64_t o = o0; o <= o1; ++o) {
    const int64_t r = d + o * S, i = s > 0 ? floor_div(-r, s) : 0;
    for (int64_t j = i; j <= i + 1; ++j) {
      const int64_t x = r + std::min(std::max(j, i0), i1) * s;
      if (x < w && -x < w) return true;
    }
  }
  return false;
}
// Rows of two tensors of the same tokens that share a byte.  Exact where strides of tokens and heads are the
// same, as of slices of one buffer in any order of its dimensions, or where each token's heads lie within the same
// pitch; otherwise spans that meet count.
bool overlap(const HeadRows& a, int64_t ha, const HeadRows& b, int64_t hb, int64_t tokens, int dim, int size) {
  if (!meet(span_of(a, tokens, ha, dim, size), span_of(b, tokens, hb, dim, size))) return false;
  if (tokens > 1 && a.ld != b.ld) return true;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)), w = (int64_t)dim * size;
  const int64_t ld = a.ld * size, hs = (ha > 1 ? a.hs : b.hs) * size, t = tokens - 1;
  if (ha == 1 || hb == 1 || a.hs == b.hs)
    return ld >= hs ? near_zero(d, ld, -t, t, hs, 1 - ha, hb - 1, w) : near_zero(d, hs, 1 - ha, hb - 1, ld, -t, t, w);
  const int64_t wa = (ha - 1) * a.hs * size + w, wb = (hb - 1) * b.hs * size + w;
  if (tokens == 1 || wa > ld || wb > ld) return true;
  const int64_t at = d - floor_div(d, ld) * ld;   // b's first byte within a's pitch
  return at < wa || at + wb > ld;
}

gptq_status check_seqs(const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t batch, int64_t tokens,
                       int64_t width, int64_t stride, int64_t pages, const int32_t* status, const void* mem,
                       KvSeqs* out) {
  if (cu == nullptr && tokens != batch)
    return fail(GPTQ_ERR_INVALID_ARG, "cu_seqlens is NULL (one token a sequence) with %lld tokens and %lld sequences",
                (long long)tokens, (long long)batch);
  if (width <= 0 || pages <= 0 || (batch > 1 && stride < width) || stride > INT64_MAX / 16 / std::max<int64_t>(batch, 1))
    return fail(GPTQ_ERR_INVALID_ARG, "page table %lld wide with stride %lld, %lld pages", (long long)width,
                (long long)stride, (long long)pages);
  if (width > INT32_MAX || pages > INT32_MAX)
    return fail(GPTQ_ERR_UNSUPPORTED, "page table %lld wide, %lld pages", (long long)width, (long long)pages);
  if ((cu && bad_ptr(cu, 4)) || bad_ptr(lens, 4) || bad_ptr(table, 4) || (status && bad_ptr(status, 4)))
    return fail(GPTQ_ERR_INVALID_ARG, "cu_seqlens, kv_lens, page_table or status is NULL or misaligned");
  if (bad_ptr(mem, 16)) return fail(GPTQ_ERR_INVALID_ARG, "pages is NULL or not 16-byte aligned");
  *out = KvSeqs{cu, lens, table, batch, tokens, width, batch > 1 ? stride : width, pages, const_cast<int32_t*>(status)};
  return GPTQ_OK;
}

gptq_status check_counts(int64_t tokens, int64_t batch) {
  if (tokens < 0 || batch < 0)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld batch=%lld", (long long)tokens, (long long)batch);
  if (tokens > kMaxTokens || batch > kMaxBatch)
    return fail(GPTQ_ERR_UNSUPPORTED, "tokens=%lld batch=%lld too large", (long long)tokens, (long long)batch);
  return GPTQ_OK;
}

gptq_status check_page_bytes(const KvLayout& L, int64_t pages) {
  if (pages > 0 && L.page_bytes > INT64_MAX / 2 / pages)
    return fail(GPTQ_ERR_INVALID_ARG, "%lld pages of %lld bytes", (long long)pages, (long long)L.page_bytes);
  return GPTQ_OK;
}

gptq_status check_beside_pages(const HeadRows& k, const HeadRows& v, const KvLayout& L, int64_t tokens, int size,
                               const void* pages, int64_t count) {
  const Span cache{pages, L.page_bytes * count};
  if (meet(span_of(k, tokens, L.heads, L.dim, size), cache) || meet(span_of(v, tokens, L.heads, L.dim, size), cache))
    return fail(GPTQ_ERR_INVALID_ARG, "K or V overlaps the pages");
  return GPTQ_OK;
}

}  // namespace

extern "C" {

size_t gptq_kv_page_bytes(const gptq_kv_config* cfg) {
  if (check_kv_config(cfg) != GPTQ_OK) {
    clear_error();
    return 0;
  }
  return (size_t)plan_kv(*cfg).page_bytes;
}

gptq_status gptq_kv_append(const gptq_kv_config* cfg, const void* K, const void* V, int32_t dtype, int64_t tokens,
                           int64_t ldk, int64_t k_head_stride, int64_t ldv, int64_t v_head_stride,
                           const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* page_table, int64_t batch,
                           int64_t table_width, int64_t table_stride, void* pages, int64_t num_pages, int32_t* status,
                           void* stream) {
  clear_error();
  GPTQ_TRY(check_kv_config(cfg));
  GPTQ_TRY(check_counts(tokens, batch));
  if (dtype != GPTQ_BF16 && dtype != GPTQ_FP32) return fail(GPTQ_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (tokens == 0 || batch == 0) return GPTQ_OK;
  const KvLayout L = plan_kv(*cfg);
  GPTQ_TRY(check_page_bytes(L, num_pages));
  HeadRows k, v;
  KvSeqs q;
  GPTQ_TRY(check_rows("K", K, dtype, tokens, L.heads, L.dim, ldk, k_head_stride, &k));
  GPTQ_TRY(check_rows("V", V, dtype, tokens, L.heads, L.dim, ldv, v_head_stride, &v));
  GPTQ_TRY(check_seqs(cu_seqlens, kv_lens, page_table, batch, tokens, table_width, table_stride, num_pages, status, pages, &q));
  GPTQ_TRY(check_beside_pages(k, v, L, tokens, dtype == GPTQ_FP32 ? 4 : 2, pages, num_pages));
  return run_kv_append(L, k, v, dtype, q, pages, static_cast<hipStream_t>(stream));
}

gptq_status gptq_kv_read(const gptq_kv_config* cfg, void* K, void* V, int32_t dtype, int64_t tokens, int64_t ldk,
                         int64_t k_head_stride, int64_t ldv, int64_t v_head_stride, const int32_t* cu_seqlens,
                         const int32_t* kv_lens, const int32_t* page_table, int64_t batch, int64_t table_width,
                         int64_t table_stride, const void* pages, int64_t num_pages, int32_t* status, void* stream) {
  clear_error();
  GPTQ_TRY(check_kv_config(cfg));
  GPTQ_TRY(check_counts(tokens, batch));
  if (dtype != GPTQ_BF16 && dtype != GPTQ_FP32) return fail(GPTQ_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (tokens == 0 || batch == 0) return GPTQ_OK;
  const KvLayout L = plan_kv(*cfg);
  GPTQ_TRY(check_page_bytes(L, num_pages));
  HeadRows k, v;
  KvSeqs q;
  GPTQ_TRY(check_rows("K", K, dtype, tokens, L.heads, L.dim, ldk, k_head_stride, &k));
  GPTQ_TRY(check_rows("V", V, dtype, tokens, L.heads, L.dim, ldv, v_head_stride, &v));
  GPTQ_TRY(check_seqs(cu_seqlens, kv_lens, page_table, batch, tokens, table_width, table_stride, num_pages, status, pages, &q));
  const int size = dtype == GPTQ_FP32 ? 4 : 2;
  if (overlap(k, L.heads, v, L.heads, tokens, L.dim, size)) return fail(GPTQ_ERR_INVALID_ARG, "K overlaps V");
  GPTQ_TRY(check_beside_pages(k, v, L, tokens, size, pages, num_pages));
  return run_kv_read(L, k, v, dtype, q, pages, static_cast<hipStream_t>(stream));
}

size_t gptq_kv_attention_workspace_bytes(const gptq_kv_config* cfg, int32_t heads, int64_t batch, int64_t tokens,
                                         int64_t max_queries) {
  if (check_kv_config(cfg) != GPTQ_OK || check_counts(tokens, batch) != GPTQ_OK || heads <= 0 || max_queries < 0 ||
      heads % cfg->kv_heads != 0 || heads > kMaxHeads) {
    clear_error();
    return 0;
  }
  return plan_kv_attention(plan_kv(*cfg), heads, batch, tokens, max_queries, false, 0).total;
}

gptq_status gptq_kv_attention(const gptq_kv_config* cfg, const void* Q, int64_t tokens, int32_t heads, int64_t ldq,
                              int64_t q_head_stride, const int32_t* cu_seqlens, int64_t max_queries,
                              const int32_t* kv_lens, const int32_t* page_table, int64_t batch, int64_t table_width,
                              int64_t table_stride, const void* pages, int64_t num_pages, float scale, void* Y,
                              int64_t ldy, int64_t y_head_stride, int32_t* status, void* workspace, size_t ws_bytes,
                              void* stream) {
  clear_error();
  GPTQ_TRY(check_kv_config(cfg));
  GPTQ_TRY(check_counts(tokens, batch));
  if (heads <= 0 || heads % cfg->kv_heads != 0 || max_queries < 0)
    return fail(GPTQ_ERR_INVALID_ARG, "heads=%d (kv_heads=%d) max_queries=%lld", heads, cfg->kv_heads, (long long)max_queries);
  if (heads > kMaxHeads) return fail(GPTQ_ERR_UNSUPPORTED, "heads=%d above %d", heads, kMaxHeads);
  GPTQ_TRY(check_scale(scale));
  if (tokens == 0 || batch == 0) return GPTQ_OK;
  const KvLayout L = plan_kv(*cfg);
  GPTQ_TRY(check_page_bytes(L, num_pages));
  HeadRows q, y;
  KvSeqs s;
  GPTQ_TRY(check_rows("Q", Q, GPTQ_BF16, tokens, heads, L.dim, ldq, q_head_stride, &q));
  GPTQ_TRY(check_rows("Y", Y, GPTQ_BF16, tokens, heads, L.dim, ldy, y_head_stride, &y));
  GPTQ_TRY(check_seqs(cu_seqlens, kv_lens, page_table, batch, tokens, table_width, table_stride, num_pages, status, pages, &s));
  if (overlap(q, heads, y, heads, tokens, L.dim, 2)) return fail(GPTQ_ERR_INVALID_ARG, "Y overlaps Q");
  if (meet(span_of(y, tokens, heads, L.dim, 2), Span{pages, L.page_bytes * num_pages}))
    return fail(GPTQ_ERR_INVALID_ARG, "Y overlaps the pages");
  const KvAttentionPlan p = plan_kv_attention(L, heads, batch, tokens, max_queries, cu_seqlens == nullptr,
                                              table_width * cfg->page_size);
  if (workspace == nullptr || ws_bytes < p.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, p.total);
  return run_kv_attention(L, heads, q, y, scale, s, pages, workspace, p, static_cast<hipStream_t>(stream));
}

gptq_status gptq_prompt_attention(const void* Q, const void* K, const void* V, int64_t tokens, int32_t heads,
                                  int32_t kv_heads, int32_t head_dim, int64_t ldq, int64_t q_head_stride, int64_t ldk,
                                  int64_t k_head_stride, int64_t ldv, int64_t v_head_stride, const int32_t* cu_seqlens,
                                  int64_t batch, float scale, void* Y, int64_t ldy, int64_t y_head_stride,
                                  void* stream) {
  clear_error();
  GPTQ_TRY(check_counts(tokens, batch));
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0)
    return fail(GPTQ_ERR_INVALID_ARG, "heads=%d kv_heads=%d", heads, kv_heads);
  if (heads > kMaxHeads) return fail(GPTQ_ERR_UNSUPPORTED, "heads=%d above %d", heads, kMaxHeads);
  if (head_dim != 64 && head_dim != 128)
    return fail(GPTQ_ERR_UNSUPPORTED, "head_dim=%d (built: 64, 128)", head_dim);
  GPTQ_TRY(check_scale(scale));
  if (tokens == 0 || batch == 0) return GPTQ_OK;
  PromptCall c;
  GPTQ_TRY(check_rows("Q", Q, GPTQ_BF16, tokens, heads, head_dim, ldq, q_head_stride, &c.Q));
  GPTQ_TRY(check_rows("K", K, GPTQ_BF16, tokens, kv_heads, head_dim, ldk, k_head_stride, &c.K));
  GPTQ_TRY(check_rows("V", V, GPTQ_BF16, tokens, kv_heads, head_dim, ldv, v_head_stride, &c.V));
  GPTQ_TRY(check_rows("Y", Y, GPTQ_BF16, tokens, heads, head_dim, ldy, y_head_stride, &c.Y));
  if (bad_ptr(cu_seqlens, 4)) return fail(GPTQ_ERR_INVALID_ARG, "cu_seqlens is NULL or misaligned");
  // workgroups of 256 threads, of which a grid holds fewer than 2^32
  if ((tokens / 128 + std::min(batch, tokens) + 1 + 8) * heads >= int64_t(1) << 24)
    return fail(GPTQ_ERR_UNSUPPORTED, "%lld tokens of %lld sequences of %d heads in one call", (long long)tokens,
                (long long)batch, heads);
  if (overlap(c.Q, heads, c.Y, heads, tokens, head_dim, 2) || overlap(c.K, kv_heads, c.Y, heads, tokens, head_dim, 2) ||
      overlap(c.V, kv_heads, c.Y, heads, tokens, head_dim, 2))
    return fail(GPTQ_ERR_INVALID_ARG, "Y overlaps Q, K or V");
  c.cu = cu_seqlens;
  c.batch = batch;
  c.tokens = tokens;
  c.heads = heads;
  c.kv_heads = kv_heads;
  c.dim = head_dim;
  c.scale = scale;
  return run_prompt_attention(c, static_cast<hipStream_t>(stream));
}

// What tests ask the checks and choices of the calls above; host only.
int gptq_internal_kv_attention_plan(const gptq_kv_config* cfg, int32_t heads, int64_t batch, int64_t tokens,
                                    int64_t max_queries, int32_t each, int64_t capacity, int32_t out[6]) {
  if (check_kv_config(cfg) != GPTQ_OK || check_counts(tokens, batch) != GPTQ_OK || heads <= 0 || heads > kMaxHeads ||
      heads % cfg->kv_heads != 0 || max_queries < 0 || tokens == 0 || batch == 0) {
    clear_error();
    return 0;
  }
  const KvAttentionPlan p = plan_kv_attention(plan_kv(*cfg), heads, batch, tokens, max_queries, each != 0, capacity);
  const int32_t v[6] = {p.tile, p.parts, p.whole, p.wgs, p.waves, p.rows};
  std::copy(v, v + 6, out);
  return 1;
}

int gptq_internal_heads_overlap(const void* a, int64_t lda, int64_t hsa, int64_t ha, const void* b, int64_t ldb,
                                int64_t hsb, int64_t hb, int64_t tokens, int32_t dim, int32_t dtype) {
  HeadRows ra, rb;
  if (check_rows("a", a, dtype, tokens, ha, dim, lda, hsa, &ra) != GPTQ_OK ||
      check_rows("b", b, dtype, tokens, hb, dim, ldb, hsb, &rb) != GPTQ_OK) {
    clear_error();
    return -1;
  }
  return overlap(ra, ha, rb, hb, tokens, dim, dtype == GPTQ_FP32 ? 4 : 2);
}

}  // extern "C"
