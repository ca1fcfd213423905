// extern "C" entry points of libgptq_mi355x: argument validation on the host,
// workspace layout, then the stage launchers (hessian.hip, prepare.hip,
// quantize.hip).  Every check here runs before any HIP call, so a rejected
// call touches no GPU state.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <vector>

#include "gptq_internal.hpp"

namespace gptq {
namespace {
thread_local char g_err[512] = {0};
}

void set_error(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
}

void clear_error() { g_err[0] = 0; }

namespace {
constexpr int64_t kMaxN = 131072;

gptq_status fail(gptq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

bool bad_ptr(const void* p, size_t align) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % align) != 0;
}

gptq_status check_config(const gptq_config* cfg) {
  if (!cfg) return fail(GPTQ_ERR_INVALID_ARG, "cfg is NULL");
  if (!(cfg->bits == 2 || cfg->bits == 3 || cfg->bits == 4 || cfg->bits == 8))
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d (built: 2, 3, 4, 8)", cfg->bits);
  if (cfg->block_size != kQBlock)
    return fail(GPTQ_ERR_UNSUPPORTED, "block_size=%d (built: 128)", cfg->block_size);
  const int g = cfg->group_size;
  if (!(g == -1 || g == 8 || g == 16 || g == 32 || g == 64 || g == 128))
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (built: -1, 8, 16, 32, 64, 128)", g);
  if (cfg->sym != 0 && cfg->sym != 1) return fail(GPTQ_ERR_INVALID_ARG, "sym=%d", cfg->sym);
  if (cfg->desc_act != 0 && cfg->desc_act != 1)
    return fail(GPTQ_ERR_INVALID_ARG, "desc_act=%d", cfg->desc_act);
  return GPTQ_OK;
}
}  // namespace
}  // namespace gptq

using namespace gptq;

namespace gptq {

gptq_status get_side_stream(SideStream& out, int which) {
  thread_local std::vector<SideStream> per_device;   // [device][which]
  if (which < 0 || which >= kSideStreams) {
    set_error("side stream %d out of range", which);
    return GPTQ_ERR_INVALID_ARG;
  }
  int dev = 0;
  GPTQ_HIP_CHECK(hipGetDevice(&dev));
  if ((int)per_device.size() < kSideStreams * (dev + 1)) per_device.resize(kSideStreams * (dev + 1));
  SideStream& s = per_device[kSideStreams * dev + which];
  if (s.stream == nullptr) {
    GPTQ_HIP_CHECK(hipStreamCreateWithFlags(&s.stream, hipStreamNonBlocking));
    // only streams of this device wait on them: a device-scope release suffices
    GPTQ_HIP_CHECK(hipEventCreateWithFlags(&s.ready, hipEventDisableTiming | hipEventReleaseToDevice));
    GPTQ_HIP_CHECK(hipEventCreateWithFlags(&s.done, hipEventDisableTiming | hipEventReleaseToDevice));
    for (hipEvent_t& e : s.aux)
      GPTQ_HIP_CHECK(hipEventCreateWithFlags(&e, hipEventDisableTiming | hipEventReleaseToDevice));
  }
  out = s;
  return GPTQ_OK;
}

}  // namespace gptq

extern "C" {

const char* gptq_last_error(void) { return g_err; }

int64_t gptq_qweight_words(int64_t n, int32_t bits) {
  if (n < 0) return -1;
  if (bits == 2 || bits == 3 || bits == 4) return ceil_div(n, 8);
  if (bits == 8) return ceil_div(n, 4);
  return -1;
}

int64_t gptq_num_groups(int64_t n, int32_t group_size) {
  if (n < 0) return -1;
  if (group_size == -1) return n > 0 ? 1 : 0;
  if (group_size <= 0) return -1;
  return ceil_div(n, group_size);
}

size_t gptq_hessian_workspace_bytes(int64_t n, int64_t tokens, int32_t x_dtype) {
  if (n <= 0 || n > kMaxN || tokens < 0) return 0;
  if (x_dtype != GPTQ_BF16) return 0;
  return plan_syrk_bf16(n, tokens).total_bytes;
}

gptq_status gptq_hessian_accumulate(float* H, double* diag_key, int64_t n, const void* X,
                                    int32_t x_dtype, int64_t tokens, int64_t ldx, float alpha,
                                    void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  if (n <= 0) return fail(GPTQ_ERR_INVALID_ARG, "n=%lld must be positive", (long long)n);
  if (n > kMaxN) return fail(GPTQ_ERR_UNSUPPORTED, "n=%lld above %lld", (long long)n, (long long)kMaxN);
  if (tokens < 0) return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld", (long long)tokens);
  if (x_dtype != GPTQ_BF16 && x_dtype != GPTQ_FP32)
    return fail(GPTQ_ERR_UNSUPPORTED, "x_dtype=%d", x_dtype);
  if (bad_ptr(H, 4)) return fail(GPTQ_ERR_INVALID_ARG, "H is NULL or misaligned");
  if (diag_key && bad_ptr(diag_key, 8)) return fail(GPTQ_ERR_INVALID_ARG, "diag_key misaligned");
  if (!std::isfinite(alpha)) return fail(GPTQ_ERR_INVALID_ARG, "alpha not finite");
  if (tokens == 0) return GPTQ_OK;
  if (ldx < n) return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld < n=%lld", (long long)ldx, (long long)n);
  if (bad_ptr(X, x_dtype == GPTQ_BF16 ? 2 : 4)) return fail(GPTQ_ERR_INVALID_ARG, "X is NULL or misaligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (x_dtype == GPTQ_FP32)
    return launch_hessian_f32(H, diag_key, n, static_cast<const float*>(X), tokens, ldx, alpha, s);
  const SyrkPlan plan = plan_syrk_bf16(n, tokens);
  if (plan.total_bytes > 0 && (workspace == nullptr || ws_bytes < plan.total_bytes || bad_ptr(workspace, 256)))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes,
                plan.total_bytes);
  return launch_hessian_bf16(H, diag_key, n, static_cast<const uint16_t*>(X), tokens, ldx, alpha,
                             workspace, plan, s);
}

size_t gptq_prepare_workspace_bytes(int64_t n) {
  if (n <= 0 || n > kPrepareMaxN) return 0;
  return plan_prepare(n).total;
}

gptq_status gptq_prepare_hinv(float* H_inout, const double* diag_key, int64_t n,
                              double damp_percent, int32_t desc_act, int32_t* perm_out,
                              void* workspace, size_t ws_bytes, double* damp_out, void* stream) {
  clear_error();
  if (n < 0) return fail(GPTQ_ERR_INVALID_ARG, "n=%lld", (long long)n);
  if (n == 0) return GPTQ_OK;
  if (n > kPrepareMaxN)
    return fail(GPTQ_ERR_UNSUPPORTED, "n=%lld above %lld", (long long)n, (long long)kPrepareMaxN);
  if (bad_ptr(H_inout, 4)) return fail(GPTQ_ERR_INVALID_ARG, "H_inout is NULL or misaligned");
  if (diag_key && bad_ptr(diag_key, 8)) return fail(GPTQ_ERR_INVALID_ARG, "diag_key misaligned");
  if (bad_ptr(perm_out, 4)) return fail(GPTQ_ERR_INVALID_ARG, "perm_out is NULL or misaligned");
  if (desc_act != 0 && desc_act != 1) return fail(GPTQ_ERR_INVALID_ARG, "desc_act=%d", desc_act);
  if (!std::isfinite(damp_percent) || damp_percent < 0.0)
    return fail(GPTQ_ERR_INVALID_ARG, "damp_percent=%g", (double)damp_percent);
  const PreparePlan plan = plan_prepare(n);
  if (workspace == nullptr || ws_bytes < plan.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes,
                plan.total);
  return run_prepare(H_inout, diag_key, n, damp_percent, desc_act, perm_out, workspace, plan,
                     damp_out, static_cast<hipStream_t>(stream));
}

size_t gptq_quantize_workspace_bytes(int64_t m, int64_t n, const gptq_config* cfg) {
  if (m <= 0 || n <= 0 || n > kPrepareMaxN || check_config(cfg) != GPTQ_OK) {
    clear_error();
    return 0;
  }
  return plan_quantize(m, n, *cfg).total;
}

gptq_status gptq_quantize_layer(const void* W, int32_t w_dtype, int64_t m, int64_t n,
                                const float* U, const int32_t* perm, const gptq_config* cfg,
                                uint32_t* qweight, float* scales, int32_t* zeros, int32_t* g_idx,
                                double* loss, int32_t* status_out, void* workspace, size_t ws_bytes,
                                void* stream) {
  clear_error();
  if (m < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  gptq_status st = check_config(cfg);
  if (st != GPTQ_OK) return st;
  if (w_dtype != GPTQ_BF16 && w_dtype != GPTQ_FP32)
    return fail(GPTQ_ERR_UNSUPPORTED, "w_dtype=%d", w_dtype);
  if (m == 0 || n == 0) return GPTQ_OK;
  if (n > kPrepareMaxN)
    return fail(GPTQ_ERR_UNSUPPORTED, "n=%lld above %lld", (long long)n, (long long)kPrepareMaxN);
  if (m > (int64_t)1 << 24) return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld too large", (long long)m);
  if (bad_ptr(W, w_dtype == GPTQ_BF16 ? 2 : 4)) return fail(GPTQ_ERR_INVALID_ARG, "W is NULL or misaligned");
  if (bad_ptr(U, 4)) return fail(GPTQ_ERR_INVALID_ARG, "U is NULL or misaligned");
  if (bad_ptr(perm, 4)) return fail(GPTQ_ERR_INVALID_ARG, "perm is NULL or misaligned");
  if (bad_ptr(qweight, 4) || bad_ptr(scales, 4) || bad_ptr(zeros, 4) || bad_ptr(g_idx, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "an output pointer is NULL or misaligned");
  if (bad_ptr(loss, 8)) return fail(GPTQ_ERR_INVALID_ARG, "loss is NULL or misaligned");
  if (status_out && bad_ptr(status_out, 4)) return fail(GPTQ_ERR_INVALID_ARG, "status_out misaligned");
  const QuantPlan plan = plan_quantize(m, n, *cfg);
  if (workspace == nullptr || ws_bytes < plan.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes,
                plan.total);
  return run_quantize(W, w_dtype, m, n, U, perm, *cfg, qweight, scales, zeros, g_idx, loss,
                      status_out, workspace, plan, static_cast<hipStream_t>(stream));
}

static gptq_status check_rtn_config(const gptq_rtn_config* cfg) {
  if (cfg == nullptr) return fail(GPTQ_ERR_INVALID_ARG, "cfg is NULL");
  if (cfg->bits != 2 && cfg->bits != 3 && cfg->bits != 4 && cfg->bits != 8)
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d", cfg->bits);
  if (cfg->group_size != -1 && cfg->group_size < 1)
    return fail(GPTQ_ERR_INVALID_ARG, "group_size=%d", cfg->group_size);
  if (cfg->sym != 0 && cfg->sym != 1) return fail(GPTQ_ERR_INVALID_ARG, "sym=%d", cfg->sym);
  if (!(cfg->clip_ratio > 0.f && cfg->clip_ratio <= 1.f))
    return fail(GPTQ_ERR_INVALID_ARG, "clip_ratio=%g outside (0, 1]", (double)cfg->clip_ratio);
  return GPTQ_OK;
}

size_t gptq_rtn_workspace_bytes(int64_t m, int64_t n, const gptq_rtn_config* cfg) {
  if (m < 0 || n < 0 || cfg == nullptr) return 0;
  return plan_rtn(m, n, cfg->group_size).total;
}

gptq_status gptq_rtn_quantize(const void* W, int32_t w_dtype, int64_t m, int64_t n,
                              const gptq_rtn_config* cfg, uint32_t* qweight, float* scales,
                              int32_t* zeros, double* err, int32_t* status_out, void* workspace,
                              size_t ws_bytes, void* stream) {
  clear_error();
  if (m < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  gptq_status st = check_rtn_config(cfg);
  if (st != GPTQ_OK) return st;
  if (w_dtype != GPTQ_BF16 && w_dtype != GPTQ_FP32)
    return fail(GPTQ_ERR_UNSUPPORTED, "w_dtype=%d", w_dtype);
  if (m == 0 || n == 0) return GPTQ_OK;
  if (m > ((int64_t)1 << 31) - 1) return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld too large", (long long)m);
  const RtnPlan plan = plan_rtn(m, n, cfg->group_size);
  if (plan.lds_bytes > kRtnMaxLds)
    return fail(GPTQ_ERR_UNSUPPORTED, "n=%lld with group_size %d needs %zu bytes of LDS per row (max %zu)",
                (long long)n, cfg->group_size, plan.lds_bytes, kRtnMaxLds);
  if (bad_ptr(W, w_dtype == GPTQ_BF16 ? 2 : 4)) return fail(GPTQ_ERR_INVALID_ARG, "W is NULL or misaligned");
  if (bad_ptr(qweight, 4) || bad_ptr(scales, 4) || bad_ptr(zeros, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "an output pointer is NULL or misaligned");
  if (bad_ptr(err, 8)) return fail(GPTQ_ERR_INVALID_ARG, "err is NULL or misaligned");
  if (status_out && bad_ptr(status_out, 4)) return fail(GPTQ_ERR_INVALID_ARG, "status_out misaligned");
  if (workspace == nullptr || ws_bytes < plan.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes,
                plan.total);
  return run_rtn(W, w_dtype, m, n, cfg->bits, cfg->sym, cfg->clip_ratio, qweight, scales, zeros, err,
                 status_out, workspace, plan, static_cast<hipStream_t>(stream));
}

size_t gptq_awq_stats_workspace_bytes(int64_t n, int64_t tokens) {
  if (n < 0 || tokens < 0) return 0;
  return plan_awq_stats(n, tokens).total;
}

gptq_status gptq_awq_channel_stats(const void* X, int32_t x_dtype, int64_t tokens, int64_t ldx,
                                   int64_t n, double* abs_sum, void* workspace, size_t ws_bytes,
                                   void* stream) {
  clear_error();
  if (tokens < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld n=%lld", (long long)tokens, (long long)n);
  if (x_dtype != GPTQ_BF16 && x_dtype != GPTQ_FP32) return fail(GPTQ_ERR_UNSUPPORTED, "x_dtype=%d", x_dtype);
  if (tokens == 0 || n == 0) return GPTQ_OK;
  if (ldx < n) return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld < n=%lld", (long long)ldx, (long long)n);
  if (bad_ptr(X, x_dtype == GPTQ_BF16 ? 2 : 4)) return fail(GPTQ_ERR_INVALID_ARG, "X is NULL or misaligned");
  if (bad_ptr(abs_sum, 8)) return fail(GPTQ_ERR_INVALID_ARG, "abs_sum is NULL or misaligned");
  const AwqStatsPlan p = plan_awq_stats(n, tokens);
  if (workspace == nullptr || ws_bytes < p.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, p.total);
  return run_awq_stats(X, x_dtype, tokens, ldx, n, abs_sum, workspace, p, static_cast<hipStream_t>(stream));
}

size_t gptq_awq_workspace_bytes(int64_t m, int64_t n, const gptq_rtn_config* cfg) {
  if (m < 0 || n < 0 || cfg == nullptr) return 0;
  return awq_extra_bytes() + plan_rtn(m, n, cfg->group_size).total;
}

gptq_status gptq_awq_quantize(const void* W, int32_t w_dtype, int64_t m, int64_t n,
                              const double* abs_sum, int64_t tokens, float protect,
                              const gptq_rtn_config* cfg, uint32_t* qweight, float* scales,
                              int32_t* zeros, float* channel_scale, double* err, int32_t* status_out,
                              void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  if (m < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  gptq_status st = check_rtn_config(cfg);
  if (st != GPTQ_OK) return st;
  if (w_dtype != GPTQ_BF16 && w_dtype != GPTQ_FP32) return fail(GPTQ_ERR_UNSUPPORTED, "w_dtype=%d", w_dtype);
  if (tokens <= 0) return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld: importance is a mean over tokens", (long long)tokens);
  if (!(protect > 0.f) || !std::isfinite(protect))
    return fail(GPTQ_ERR_INVALID_ARG, "protect=%g must be positive and finite", (double)protect);
  if (m == 0 || n == 0) return GPTQ_OK;
  if (m > ((int64_t)1 << 31) - 1) return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld too large", (long long)m);
  const RtnPlan plan = plan_rtn(m, n, cfg->group_size);
  if (plan.lds_bytes > kRtnMaxLds)
    return fail(GPTQ_ERR_UNSUPPORTED, "n=%lld with group_size %d needs %zu bytes of LDS per row (max %zu)",
                (long long)n, cfg->group_size, plan.lds_bytes, kRtnMaxLds);
  if (bad_ptr(W, w_dtype == GPTQ_BF16 ? 2 : 4)) return fail(GPTQ_ERR_INVALID_ARG, "W is NULL or misaligned");
  if (bad_ptr(abs_sum, 8)) return fail(GPTQ_ERR_INVALID_ARG, "abs_sum is NULL or misaligned");
  if (bad_ptr(qweight, 4) || bad_ptr(scales, 4) || bad_ptr(zeros, 4) || bad_ptr(channel_scale, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "an output pointer is NULL or misaligned");
  if (bad_ptr(err, 8)) return fail(GPTQ_ERR_INVALID_ARG, "err is NULL or misaligned");
  if (status_out && bad_ptr(status_out, 4)) return fail(GPTQ_ERR_INVALID_ARG, "status_out misaligned");
  const size_t need = awq_extra_bytes() + plan.total;
  if (workspace == nullptr || ws_bytes < need || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, need);
  return run_awq_quantize(W, w_dtype, m, n, abs_sum, tokens, protect, cfg->bits, cfg->sym, cfg->clip_ratio,
                          qweight, scales, zeros, channel_scale, err, status_out, workspace, plan,
                          static_cast<hipStream_t>(stream));
}

static bool w4_group_ok(int32_t g) { return g == -1 || g == 32 || g == 64 || g == 128; }

size_t gptq_w4a16_packed_bytes(int64_t m, int64_t n, int32_t group_size) {
  if (m < 0 || n < 0 || !w4_group_ok(group_size)) return 0;
  return plan_w4a16(m, n, group_size).total;
}

gptq_status gptq_w4a16_pack(const uint32_t* qweight, const float* scales, const int32_t* zeros,
                            const int32_t* g_idx, int64_t m, int64_t n, int32_t bits,
                            int32_t group_size, void* packed, size_t packed_bytes, void* stream) {
  clear_error();
  if (m < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  if (bits != 2 && bits != 3 && bits != 4)
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d (the W4A16 product takes 2-, 3- and 4-bit codes)", bits);
  if (!w4_group_ok(group_size))
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", group_size);
  if (m == 0 || n == 0) return GPTQ_OK;
  if (m > ((int64_t)1 << 30) || n > ((int64_t)1 << 30))
    return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld n=%lld too large", (long long)m, (long long)n);
  if (bad_ptr(qweight, 4) || bad_ptr(scales, 4) || bad_ptr(zeros, 4) || bad_ptr(g_idx, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "an input pointer is NULL or misaligned");
  const W4Layout L = plan_w4a16(m, n, group_size);
  if (packed == nullptr || packed_bytes < L.total || bad_ptr(packed, 256))
    return fail(GPTQ_ERR_WORKSPACE, "packed buffer %zu bytes, need %zu (256-byte aligned)",
                packed_bytes, L.total);
  return run_w4a16_pack(qweight, scales, zeros, g_idx, bits, L, packed,
                        static_cast<hipStream_t>(stream));
}

int64_t gptq_checkpoint_qweight_rows(int64_t n, int32_t bits) {
  if (n < 0 || !(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return -1;
  return ceil_div(n * bits, 32);
}

int64_t gptq_checkpoint_qzeros_words(int64_t m, int32_t bits) {
  if (m < 0 || !(bits == 2 || bits == 3 || bits == 4 || bits == 8)) return -1;
  return ceil_div(m * bits, 32);
}

gptq_status gptq_export_checkpoint(const uint32_t* qweight, const float* scales, const int32_t* zeros,
                                   int64_t m, int64_t n, int32_t bits, int32_t group_size, int32_t zero_offset,
                                   int32_t* ck_qweight, int32_t* ck_qzeros, uint16_t* ck_scales, void* stream) {
  clear_error();
  if (m < 0 || n < 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  if (!(bits == 2 || bits == 3 || bits == 4 || bits == 8))
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d (2, 3, 4 or 8)", bits);
  if (zero_offset != 0 && zero_offset != 1) return fail(GPTQ_ERR_INVALID_ARG, "zero_offset=%d (0 or 1)", zero_offset);
  const int64_t G = gptq_num_groups(n, group_size);
  if (G < 0) return fail(GPTQ_ERR_INVALID_ARG, "group_size=%d", group_size);
  if (m == 0 || n == 0) return GPTQ_OK;
  if (m > 65535LL * 64 || G > 65535 || n > ((int64_t)1 << 40))
    return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld n=%lld (%lld groups) too large", (long long)m, (long long)n,
                (long long)G);
  if (bad_ptr(qweight, 4) || bad_ptr(scales, 4) || bad_ptr(zeros, 4))
    return fail(GPTQ_ERR_INVALID_ARG, "an input pointer is NULL or misaligned");
  if (bad_ptr(ck_qweight, 4) || bad_ptr(ck_qzeros, 4) || bad_ptr(ck_scales, 2))
    return fail(GPTQ_ERR_INVALID_ARG, "an output pointer is NULL or misaligned");
  return run_checkpoint_export(qweight, scales, zeros, m, n, bits, G, zero_offset, ck_qweight, ck_qzeros,
                               ck_scales, static_cast<hipStream_t>(stream));
}

size_t gptq_w4a16_workspace_bytes(int64_t tokens, int64_t m, int64_t n) {
  if (tokens < 0 || m < 0 || n < 0) return 0;
  return plan_w4a16_gemm(tokens, m, n).total;
}

gptq_status gptq_w4a16_matmul(const void* X, int64_t tokens, int64_t ldx, const void* packed,
                              int64_t m, int64_t n, int32_t group_size, float* Y, int64_t ldy,
                              void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  if (tokens < 0 || m < 0 || n < 0)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld m=%lld n=%lld", (long long)tokens, (long long)m,
                (long long)n);
  if (!w4_group_ok(group_size))
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", group_size);
  if (tokens == 0 || m == 0 || n == 0) return GPTQ_OK;
  if (m > ((int64_t)1 << 30) || n > ((int64_t)1 << 30))
    return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld n=%lld too large", (long long)m, (long long)n);
  if (ldx < n || ldy < m)
    return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld < n or ldy=%lld < m", (long long)ldx, (long long)ldy);
  if (bad_ptr(X, 2) || bad_ptr(Y, 4)) return fail(GPTQ_ERR_INVALID_ARG, "X or Y is NULL or misaligned");
  if (bad_ptr(packed, 256)) return fail(GPTQ_ERR_INVALID_ARG, "packed is NULL or not 256-byte aligned");
  const W4GemmPlan p = plan_w4a16_gemm(tokens, m, n);
  if (workspace == nullptr || ws_bytes < p.total || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, p.total);
  return run_w4a16_matmul(static_cast<const uint16_t*>(X), tokens, ldx, packed,
                          plan_w4a16(m, n, group_size), Y, ldy, workspace, p,
                          static_cast<hipStream_t>(stream));
}

size_t gptq_w4a16_noalloc_scratch_bytes(void) { return w4a16_noalloc_scratch_bytes(); }

gptq_status gptq_w4a16_matmul_noalloc(const void* X, int64_t tokens, int64_t ldx, const void* packed,
                                      int64_t m, int64_t n, int32_t group_size, float* Y, int64_t ldy,
                                      void* stream) {
  clear_error();
  if (tokens < 0 || m < 0 || n < 0)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld m=%lld n=%lld", (long long)tokens, (long long)m,
                (long long)n);
  if (!w4_group_ok(group_size))
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", group_size);
  if (tokens == 0 || m == 0 || n == 0) return GPTQ_OK;
  if (m > ((int64_t)1 << 30) || n > ((int64_t)1 << 30))
    return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld n=%lld too large", (long long)m, (long long)n);
  if (ldx < n || ldy < m)
    return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld < n or ldy=%lld < m", (long long)ldx, (long long)ldy);
  if (bad_ptr(X, 2) || bad_ptr(Y, 4)) return fail(GPTQ_ERR_INVALID_ARG, "X or Y is NULL or misaligned");
  if (bad_ptr(packed, 256)) return fail(GPTQ_ERR_INVALID_ARG, "packed is NULL or not 256-byte aligned");
  return run_w4a16_matmul_noalloc(static_cast<const uint16_t*>(X), tokens, ldx, packed,
                                  plan_w4a16(m, n, group_size), Y, ldy, static_cast<hipStream_t>(stream));
}

// ---------------------------------------------------------------- layers on packed weights
static bool float_dtype(int32_t d) { return d == GPTQ_BF16 || d == GPTQ_FP32; }
static size_t dtype_bytes(int32_t d) { return d == GPTQ_FP32 ? 4 : 2; }
constexpr int64_t kL4MaxRows = (int64_t)1 << 23;
constexpr int64_t kL4MaxCols = (int64_t)1 << 20;   // 256 rows of X' stay within 32-bit offsets
constexpr int64_t kL4MaxTokens = (int64_t)1 << 30;

// the checks that the linear and the glu share; *done: nothing to compute
static gptq_status check_l4(const void* X, int64_t tokens, int64_t ldx, const void* packed, int64_t m, int64_t n,
                            int32_t group_size, int32_t activation, const void* Y, int32_t y_dtype, int64_t ldy,
                            bool* done) {
  *done = false;
  if (tokens < 0 || m < 0 || n <= 0)
    return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld m=%lld n=%lld", (long long)tokens, (long long)m, (long long)n);
  if (!w4_group_ok(group_size)) return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", group_size);
  if (activation < GPTQ_ACT_NONE || activation > GPTQ_ACT_GELU_TANH)
    return fail(GPTQ_ERR_UNSUPPORTED, "activation=%d", activation);
  if (!float_dtype(y_dtype)) return fail(GPTQ_ERR_UNSUPPORTED, "y_dtype=%d", y_dtype);
  if (m > kL4MaxRows || n > kL4MaxCols || tokens > kL4MaxTokens)
    return fail(GPTQ_ERR_UNSUPPORTED, "tokens=%lld m=%lld n=%lld too large", (long long)tokens, (long long)m,
                (long long)n);
  if (tokens == 0 || m == 0) {
    *done = true;
    return GPTQ_OK;
  }
  if (ldx < n || ldy < m)
    return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld < n or ldy=%lld < m", (long long)ldx, (long long)ldy);
  if (bad_ptr(X, 2) || bad_ptr(Y, dtype_bytes(y_dtype)))
    return fail(GPTQ_ERR_INVALID_ARG, "X or Y is NULL or misaligned");
  if (bad_ptr(packed, 256)) return fail(GPTQ_ERR_INVALID_ARG, "packed is NULL or not 256-byte aligned");
  return GPTQ_OK;
}

static gptq_status check_l4_buffers(size_t packed_bytes, size_t need_packed, const void* workspace, size_t ws_bytes,
                                    size_t need) {
  if (packed_bytes < need_packed)
    return fail(GPTQ_ERR_INVALID_ARG, "packed buffer %zu bytes, this weight takes %zu", packed_bytes, need_packed);
  if (workspace == nullptr || ws_bytes < need || bad_ptr(workspace, 256))
    return fail(GPTQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu (256-byte aligned)", ws_bytes, need);
  return GPTQ_OK;
}

static gptq_status check_l4_tensor(const char* name, const void* p, int32_t dtype) {
  if (p == nullptr) return GPTQ_OK;
  if (!float_dtype(dtype)) return fail(GPTQ_ERR_UNSUPPORTED, "%s dtype=%d", name, dtype);
  if (bad_ptr(p, dtype_bytes(dtype))) return fail(GPTQ_ERR_INVALID_ARG, "%s is misaligned", name);
  return GPTQ_OK;
}

struct RowSpan {
  const void* p;
  int64_t rows, pitch, width;   // of a row, in bytes; width <= pitch
};

// Whether a row of `a` shares a byte with a row of `b`.  Column slices of one
// buffer lie between each other's rows and do not.
static bool rows_overlap(const RowSpan& a, const RowSpan& b) {
  const int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p);
  if (d >= (a.rows - 1) * a.pitch + a.width || -d >= (b.rows - 1) * b.pitch + b.width) return false;
  auto meet = [&](int64_t i, int64_t j) {   // a's row i and b's row j
    const int64_t at = d + j * b.pitch - i * a.pitch;
    return i >= 0 && i < a.rows && at < a.width && at + b.width > 0;
  };
  auto row_at = [&](int64_t x) { return x / a.pitch - (x % a.pitch < 0); };   // rounded down
  if (a.pitch == b.pitch) {   // b's row j can meet a's rows j + q and j + q + 1, for every j alike
    const int64_t q = row_at(d), j0 = std::max<int64_t>(0, -q), j1 = std::max<int64_t>(0, -q - 1);
    return (j0 < b.rows && meet(j0 + q, j0)) || (j1 < b.rows && meet(j1 + q + 1, j1));
  }
  for (int64_t j = 0; j < b.rows; ++j) {
    const int64_t i = std::max<int64_t>(0, row_at(d + j * b.pitch));
    if (meet(i, j) || meet(i + 1, j)) return true;
  }
  return false;
}

// Y overlaps X, or the residual without being it
static gptq_status check_l4_overlap(const void* X, int64_t ldx, int64_t n, const void* res, int32_t res_dtype, int64_t ldr,
                                    const void* Y, int32_t y_dtype, int64_t ldy, int64_t m, int64_t tokens) {
  if (tokens == 1) {   // no second row: any stride will do
    ldx = n;
    ldr = ldy = m;
  }
  for (int64_t ld : {ldx, ldy, res ? ldr : 0})
    if (ld > INT64_MAX / 8 / tokens) return fail(GPTQ_ERR_INVALID_ARG, "a row stride of %lld", (long long)ld);
  const int64_t ysz = (int64_t)dtype_bytes(y_dtype), rsz = (int64_t)dtype_bytes(res_dtype);
  const RowSpan y{Y, tokens, ldy * ysz, m * ysz};
  if (rows_overlap(RowSpan{X, tokens, ldx * 2, n * 2}, y)) return fail(GPTQ_ERR_INVALID_ARG, "Y overlaps X");
  if (res && res != Y && rows_overlap(RowSpan{res, tokens, ldr * rsz, m * rsz}, y))
    return fail(GPTQ_ERR_INVALID_ARG, "Y overlaps the residual");
  return GPTQ_OK;
}

size_t gptq_w4a16_linear_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int32_t group_size) {
  if (tokens < 0 || tokens > kL4MaxTokens || m < 0 || m > kL4MaxRows || n <= 0 || n > kL4MaxCols ||
      !w4_group_ok(group_size))
    return 0;
  return w4a16_linear_workspace(tokens, n, plan_w4a16(m, n, group_size).mt * 16);
}

gptq_status gptq_w4a16_linear(const void* X, int64_t tokens, int64_t ldx, const void* packed, size_t packed_bytes,
                              int64_t m, int64_t n, int32_t group_size, const gptq_epilogue* epilogue, void* Y,
                              int32_t y_dtype, int64_t ldy, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  const gptq_epilogue e = epilogue ? *epilogue : gptq_epilogue{GPTQ_ACT_NONE, 0, nullptr, 0, nullptr, 0};
  bool done = false;
  GPTQ_TRY(check_l4(X, tokens, ldx, packed, m, n, group_size, e.activation, Y, y_dtype, ldy, &done));
  if (done) return GPTQ_OK;
  GPTQ_TRY(check_l4_tensor("bias", e.bias, e.bias_dtype));
  GPTQ_TRY(check_l4_tensor("residual", e.residual, e.residual_dtype));
  if (e.residual && e.ldr < m) return fail(GPTQ_ERR_INVALID_ARG, "ldr=%lld < m", (long long)e.ldr);
  if (e.residual == Y && (e.residual_dtype != y_dtype || e.ldr != ldy))
    return fail(GPTQ_ERR_INVALID_ARG, "Y is the residual, with another type or row stride");
  const W4Layout L = plan_w4a16(m, n, group_size);
  const L4LinearPlan p = plan_w4a16_linear(tokens, n, L.mt * 16);
  GPTQ_TRY(check_l4_buffers(packed_bytes, L.total, workspace, ws_bytes, p.total));
  GPTQ_TRY(check_l4_overlap(X, ldx, n, e.residual, e.residual_dtype, e.ldr, Y, y_dtype, ldy, m, tokens));
  const L4Call c{static_cast<const uint16_t*>(X), tokens, ldx, m, packed, e.activation, e.bias_dtype,
                 e.residual_dtype, y_dtype, e.bias, nullptr, e.residual, e.ldr, Y, ldy};
  return run_w4a16_linear(c, L, false, workspace, p, static_cast<hipStream_t>(stream));
}

size_t gptq_w4a16_glu_packed_bytes(int64_t m, int64_t n, int32_t group_size) {
  if (m < 0 || n < 0 || m > kL4MaxRows || n > kL4MaxCols || !w4_group_ok(group_size)) return 0;
  return plan_w4a16_pair(m, n, group_size).total;
}

static gptq_status check_l4_pack(int64_t m, int64_t n, int32_t bits, int32_t group_size) {
  if (m <= 0 || n <= 0) return fail(GPTQ_ERR_INVALID_ARG, "m=%lld n=%lld", (long long)m, (long long)n);
  if (bits != 2 && bits != 3 && bits != 4)
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d (the W4A16 layers take 2-, 3- and 4-bit codes)", bits);
  if (!w4_group_ok(group_size)) return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", group_size);
  if (m > kL4MaxRows || n > kL4MaxCols)
    return fail(GPTQ_ERR_UNSUPPORTED, "m=%lld n=%lld too large", (long long)m, (long long)n);
  return GPTQ_OK;
}

gptq_status gptq_w4a16_glu_pack(const uint32_t* gate_qweight, const float* gate_scales, const int32_t* gate_zeros,
                                const uint32_t* up_qweight, const float* up_scales, const int32_t* up_zeros,
                                const int32_t* g_idx, int64_t m, int64_t n, int32_t bits, int32_t group_size,
                                void* packed, size_t packed_bytes, void* stream) {
  clear_error();
  GPTQ_TRY(check_l4_pack(m, n, bits, group_size));
  const void* in[] = {gate_qweight, gate_scales, gate_zeros, up_qweight, up_scales, up_zeros, g_idx};
  for (const void* p : in)
    if (bad_ptr(p, 4)) return fail(GPTQ_ERR_INVALID_ARG, "an input pointer is NULL or misaligned");
  const W4Layout L = plan_w4a16_pair(m, n, group_size);
  if (packed == nullptr || packed_bytes < L.total || bad_ptr(packed, 256))
    return fail(GPTQ_ERR_WORKSPACE, "packed buffer %zu bytes, need %zu (256-byte aligned)", packed_bytes, L.total);
  const L4PairSource src{gate_qweight, up_qweight, gate_scales, up_scales, gate_zeros, up_zeros, m, nullptr};
  return run_w4a16_glu_pack(src, g_idx, L, packed, static_cast<hipStream_t>(stream));
}

size_t gptq_w4a16_glu_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int32_t group_size) {
  if (tokens < 0 || tokens > kL4MaxTokens || m < 0 || m > kL4MaxRows || n <= 0 || n > kL4MaxCols ||
      !w4_group_ok(group_size))
    return 0;
  return w4a16_linear_workspace(tokens, n, plan_w4a16_pair(m, n, group_size).mt * 16);
}

gptq_status gptq_w4a16_glu(const void* X, int64_t tokens, int64_t ldx, const void* packed, size_t packed_bytes,
                           int64_t m, int64_t n, int32_t group_size, int32_t activation, const void* gate_bias,
                           const void* up_bias, int32_t bias_dtype, void* Y, int32_t y_dtype, int64_t ldy,
                           void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  bool done = false;
  GPTQ_TRY(check_l4(X, tokens, ldx, packed, m, n, group_size, activation, Y, y_dtype, ldy, &done));
  if (done) return GPTQ_OK;
  GPTQ_TRY(check_l4_tensor("gate_bias", gate_bias, bias_dtype));
  GPTQ_TRY(check_l4_tensor("up_bias", up_bias, bias_dtype));
  const W4Layout L = plan_w4a16_pair(m, n, group_size);
  const L4LinearPlan p = plan_w4a16_linear(tokens, n, L.mt * 16);
  GPTQ_TRY(check_l4_buffers(packed_bytes, L.total, workspace, ws_bytes, p.total));
  GPTQ_TRY(check_l4_overlap(X, ldx, n, nullptr, 0, 0, Y, y_dtype, ldy, m, tokens));
  const L4Call c{static_cast<const uint16_t*>(X), tokens, ldx, m, packed, activation, bias_dtype, 0, y_dtype,
                 gate_bias, up_bias, nullptr, 0, Y, ldy};
  return run_w4a16_linear(c, L, true, workspace, p, static_cast<hipStream_t>(stream));
}

// ---------------------------------------------------------------- mixture of experts
static gptq_status check_moe(const gptq_moe_config* c) {
  if (c == nullptr) return fail(GPTQ_ERR_INVALID_ARG, "cfg is NULL");
  if (c->hidden <= 0 || c->inter <= 0 || c->experts <= 0 || c->top_k <= 0 || c->top_k > c->experts)
    return fail(GPTQ_ERR_INVALID_ARG, "hidden=%lld inter=%lld experts=%d top_k=%d", (long long)c->hidden,
                (long long)c->inter, c->experts, c->top_k);
  if (c->renormalize != 0 && c->renormalize != 1) return fail(GPTQ_ERR_INVALID_ARG, "renormalize=%d", c->renormalize);
  if (c->hidden > 32768 || c->inter > 32768 || c->experts > 1024 || c->top_k > 64)
    return fail(GPTQ_ERR_UNSUPPORTED, "hidden=%lld inter=%lld experts=%d top_k=%d (up to 32768, 32768, 1024, 64)",
                (long long)c->hidden, (long long)c->inter, c->experts, c->top_k);
  if (c->bits != 2 && c->bits != 3 && c->bits != 4)
    return fail(GPTQ_ERR_UNSUPPORTED, "bits=%d (the W4A16 layers take 2-, 3- and 4-bit codes)", c->bits);
  if (!w4_group_ok(c->group_size))
    return fail(GPTQ_ERR_UNSUPPORTED, "group_size=%d (32, 64, 128 or -1)", c->group_size);
  if (c->activation < GPTQ_ACT_NONE || c->activation > GPTQ_ACT_GELU_TANH)
    return fail(GPTQ_ERR_UNSUPPORTED, "activation=%d", c->activation);
  return GPTQ_OK;
}

size_t gptq_w4a16_moe_packed_bytes(const gptq_moe_config* cfg) {
  if (check_moe(cfg) != GPTQ_OK) {
    clear_error();
    return 0;
  }
  return plan_moe(*cfg).stride * (size_t)cfg->experts;
}

gptq_status gptq_w4a16_moe_pack(const gptq_moe_config* cfg, int32_t expert, const uint32_t* gate_qweight,
                                const float* gate_scales, const int32_t* gate_zeros, const uint32_t* up_qweight,
                                const float* up_scales, const int32_t* up_zeros, const int32_t* g_idx,
                                const uint32_t* down_qweight, const float* down_scales, const int32_t* down_zeros,
                                const int32_t* down_g_idx, void* packed, size_t packed_bytes, void* stream) {
  clear_error();
  GPTQ_TRY(check_moe(cfg));
  if (expert < 0 || expert >= cfg->experts) return fail(GPTQ_ERR_INVALID_ARG, "expert=%d of %d", expert, cfg->experts);
  const void* in[] = {gate_qweight, gate_scales,  gate_zeros,  up_qweight, up_scales, up_zeros,
                      g_idx,        down_qweight, down_scales, down_zeros, down_g_idx};
  for (const void* p : in)
    if (bad_ptr(p, 4)) return fail(GPTQ_ERR_INVALID_ARG, "an input pointer is NULL or misaligned");
  const size_t need = plan_moe(*cfg).stride * (size_t)cfg->experts;
  if (packed == nullptr || packed_bytes < need || bad_ptr(packed, 256))
    return fail(GPTQ_ERR_WORKSPACE, "packed buffer %zu bytes, need %zu (256-byte aligned)", packed_bytes, need);
  const L4PairSource src{gate_qweight, up_qweight, gate_scales, up_scales, gate_zeros, up_zeros, cfg->inter, nullptr};
  return run_moe_pack(*cfg, expert, src, g_idx, down_qweight, down_scales, down_zeros, down_g_idx, packed,
                      static_cast<hipStream_t>(stream));
}

size_t gptq_w4a16_moe_workspace_bytes(const gptq_moe_config* cfg, int64_t tokens) {
  if (check_moe(cfg) != GPTQ_OK || tokens < 0 || tokens > kL4MaxTokens) {
    clear_error();
    return 0;
  }
  return moe_workspace(*cfg, tokens);
}

// Host only, not in the public header: the kernels that a call would run, for
// the tests, which say which of them each case is meant to reach.
int gptq_internal_w4a16_linear_path(int64_t tokens, int64_t m, int64_t n, int32_t group_size, int32_t gated,
                                    int32_t out[5]) {
  if (tokens <= 0 || m <= 0 || n <= 0 || tokens > kL4MaxTokens || m > kL4MaxRows || n > kL4MaxCols ||
      !w4_group_ok(group_size))
    return 0;
  const W4Layout L = gated ? plan_w4a16_pair(m, n, group_size) : plan_w4a16(m, n, group_size);
  const L4Path p = w4a16_linear_path(tokens, L, gated != 0);
  const int32_t v[5] = {p.tile, p.gather, p.whole, p.parted, p.splits};
  std::copy(v, v + 5, out);
  return 1;
}

int gptq_internal_w4a16_moe_path(const gptq_moe_config* cfg, int64_t tokens, int32_t y_dtype, int32_t out[7]) {
  if (check_moe(cfg) != GPTQ_OK || tokens <= 0 || tokens > kL4MaxTokens || !float_dtype(y_dtype)) {
    clear_error();
    return 0;
  }
  const MoePath p = moe_path(*cfg, tokens, y_dtype);
  const int32_t v[7] = {p.small, p.logits, p.gate_up_lds, p.gate_up_pass, p.down_lds, p.down_pass, p.slices};
  std::copy(v, v + 7, out);
  return 1;
}

gptq_status gptq_w4a16_moe(const void* X, int64_t tokens, int64_t ldx, const void* router, int32_t router_dtype,
                           const gptq_moe_config* cfg, const void* packed, size_t packed_bytes,
                           const void* residual, int32_t residual_dtype, int64_t ldr, void* Y, int32_t y_dtype,
                           int64_t ldy, int32_t* topk_ids, float* topk_weights, void* workspace, size_t ws_bytes,
                           void* stream) {
  clear_error();
  GPTQ_TRY(check_moe(cfg));
  if (tokens < 0) return fail(GPTQ_ERR_INVALID_ARG, "tokens=%lld", (long long)tokens);
  if (tokens > kL4MaxTokens) return fail(GPTQ_ERR_UNSUPPORTED, "tokens=%lld too large", (long long)tokens);
  if (!float_dtype(y_dtype)) return fail(GPTQ_ERR_UNSUPPORTED, "y_dtype=%d", y_dtype);
  if (!float_dtype(router_dtype)) return fail(GPTQ_ERR_UNSUPPORTED, "router dtype=%d", router_dtype);
  if (tokens == 0) return GPTQ_OK;
  if (ldx < cfg->hidden || ldy < cfg->hidden)
    return fail(GPTQ_ERR_INVALID_ARG, "ldx=%lld or ldy=%lld < hidden", (long long)ldx, (long long)ldy);
  if (bad_ptr(X, 2) || bad_ptr(Y, dtype_bytes(y_dtype)) || bad_ptr(router, dtype_bytes(router_dtype)))
    return fail(GPTQ_ERR_INVALID_ARG, "X, Y or router is NULL or misaligned");
  if (bad_ptr(packed, 256)) return fail(GPTQ_ERR_INVALID_ARG, "packed is NULL or not 256-byte aligned");
  GPTQ_TRY(check_l4_tensor("residual", residual, residual_dtype));
  if (residual && ldr < cfg->hidden) return fail(GPTQ_ERR_INVALID_ARG, "ldr=%lld < hidden", (long long)ldr);
  if (residual == Y && (residual_dtype != y_dtype || ldr != ldy))
    return fail(GPTQ_ERR_INVALID_ARG, "Y is the residual, with another type or row stride");
  if ((topk_ids && bad_ptr(topk_ids, 4)) || (topk_weights && bad_ptr(topk_weights, 4)))
    return fail(GPTQ_ERR_INVALID_ARG, "topk_ids or topk_weights is misaligned");
  const MoeWork w = plan_moe_work(*cfg, tokens);
  GPTQ_TRY(check_l4_buffers(packed_bytes, plan_moe(*cfg).stride * (size_t)cfg->experts, workspace, ws_bytes, w.total));
  GPTQ_TRY(check_l4_overlap(X, ldx, cfg->hidden, residual, residual_dtype, ldr, Y, y_dtype, ldy, cfg->hidden, tokens));
  const MoeCall c{static_cast<const uint16_t*>(X), tokens, ldx, router, router_dtype, packed, residual,
                  residual_dtype, ldr, Y, y_dtype, ldy, topk_ids, topk_weights};
  return run_moe(c, *cfg, workspace, w, static_cast<hipStream_t>(stream));
}

}  // extern "C"
