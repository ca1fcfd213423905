// Layers on packed 2/3/4-bit weights: a projection with bias, activation and
// residual in its epilogue (gptq_w4a16_linear) and the gated half of an MLP
// (gptq_w4a16_glu).
//
//   linear  Y[t][r] = act(Σ_k x[t][k]·(q[r][k] - z[r][g(k)])·s[r][g(k)] + b[r]) + R[t][r]
//   glu     Y[t][r] = act(gate[t][r] + bg[r])·(up[t][r] + bu[r])
//
// The linear's weight is gptq_w4a16_pack's; the glu's is the same layout with
// the 16-row tiles of gate and up alternating (tile 2i gate, 2i + 1 up), so a
// wave that takes a pair of tiles holds both factors of an output.
#include <algorithm>

#include "w4a16_device.hpp"

namespace gptq {
namespace {

// ---------------------------------------------------------------- pack (glu)
__global__ __launch_bounds__(256) void l4_pair_params_kernel(L4PairSource src, int64_t rows, int64_t G, int64_t Gp,
                                                             int64_t total, float2* __restrict__ params) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t tile = i / (Gp * kL4Rows), grp = (i / kL4Rows) % Gp;
  int64_t r = (tile >> 1) * kL4Rows + (i % kL4Rows);
  float2 v = make_float2(0.f, 128.f);
  if (r < rows && src.row_order) r = src.row_order[r];
  if (r >= 0 && r < src.m && grp < G) {
    const float* s = (tile & 1) ? src.scales1 : src.scales0;
    const int32_t* z = (tile & 1) ? src.zeros1 : src.zeros0;
    v = make_float2(s[r * G + grp], 128.f + (float)z[r * G + grp]);
  }
  params[i] = v;
}

__global__ __launch_bounds__(256) void l4_pair_codes_kernel(L4PairSource src, int64_t rows, int64_t words, int64_t n,
                                                            int64_t kc, int64_t total,
                                                            const int32_t* __restrict__ order,
                                                            uint32_t* __restrict__ codes) {
  const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (w >= total) return;
  const int j = (int)(w & 3), l = (int)((w >> 2) & 63);
  const int64_t tc = w >> 8, tile = tc / kc, C = tc % kc;
  const uint32_t* q = (tile & 1) ? src.qweight1 : src.qweight0;
  int64_t r = (tile >> 1) * kL4Rows + (l & 15);
  if (r < rows && src.row_order) r = src.row_order[r];
  const int64_t kb = C * kL4Chunk + 32 * j + 8 * (l >> 4);
  uint32_t word = 0;
  if (r >= 0 && r < src.m) {
    for (int e = 0; e < 8; ++e) {
      if (kb + e >= n) break;
      const int32_t col = order[kb + e];
      if (col < 0) continue;
      word |= ((q[r * words + (col >> 3)] >> (4 * (col & 7))) & 15u) << (4 * ((e & 1) * 4 + (e >> 1)));
    }
  }
  codes[w] = word;
}

// ---------------------------------------------------------------- product
struct L4Epilogue {
  int act, bias_dt, res_dt, y_dt;
  const void *bias, *bias2, *res;
  void* Y;
  int64_t ldr, ldy;
  __device__ __forceinline__ void linear(int64_t t, int64_t r, float v) const {
    if (bias) v += l4_load(bias, bias_dt, r);
    v = l4_activate(v, act);
    if (res) v += l4_load(res, res_dt, t * ldr + r);
    l4_store(Y, y_dt, t * ldy + r, v);
  }
  __device__ __forceinline__ void gated(int64_t t, int64_t r, float g, float u) const {
    if (bias) g += l4_load(bias, bias_dt, r);
    if (bias2) u += l4_load(bias2, bias_dt, r);
    l4_store(Y, y_dt, t * ldy + r, l4_activate(g, act) * u);
  }
};

struct L4StreamArgs {
  const uint16_t* Xp;     // [tokens][n128] bf16, processing order
  const float2* params;   // [tiles][Gp][16]
  const u32x4_t* codes;   // [tiles][kc][64]
  int64_t n128, kc, Gp, units, m, tokens;
  int pmul, kslog;        // waves that split K: 1 << kslog
  L4Epilogue ep;
};

// Unit = one row tile (linear) or one gate/up pair of tiles (glu).  A
// workgroup of 8 waves holds 8 >> kslog units x 16 tokens, 1 << kslog waves
// splitting the K range of each; their sums meet in LDS in wave order.
template <int GS, bool GATED>
__global__ __launch_bounds__(512) void l4_stream_kernel(L4StreamArgs a) {
  constexpr int RT = GATED ? 2 : 1;
  __shared__ float red[8][RT][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = 1 << a.kslog, upw = 8 >> a.kslog;
  const int64_t u0 = (int64_t)blockIdx.x * upw;
  const int64_t unit = std::min<int64_t>(u0 + (wave >> a.kslog), a.units - 1);
  const int sl = wave & (ks - 1);
  const int cps = (int)((a.kc + ks - 1) >> a.kslog);
  const int c0 = sl * cps, c1 = (int)std::min<int64_t>(a.kc, c0 + cps);
  const int64_t t0 = (int64_t)blockIdx.y * 16;
  const int64_t t = std::min<int64_t>(t0 + (lane & 15), a.tokens - 1);   // rows past the last: computed, not stored
  const L4GlobalA af{a.Xp + t * a.n128 + 8 * (lane >> 4), 0};
  const u32x4_t* cp[RT];
  const float2* pp[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    cp[r] = a.codes + (unit * RT + r) * a.kc * 64 + lane;
    pp[r] = a.params + (unit * RT + r) * a.Gp * kL4Rows + (lane & 15);
  }
  const L4Consts kc;
  f32x4_t y[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) y[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  l4_stream<GS, RT, 1, (GATED ? 2 : 4)>(af, cp, pp, a.pmul, c0, c1, kc, y);
#pragma unroll
  for (int r = 0; r < RT; ++r) *reinterpret_cast<f32x4_t*>(&red[wave][r][lane * 4]) = y[r];
  __syncthreads();
  // D[4·(lane/16) + v][lane % 16]: token 4·quad + v of weight row lane % 16
  for (int i = tid; i < upw * 256; i += 512) {
    const int ul = i >> 8, tl = (i >> 4) & 15, row = i & 15;
    const int at = ((tl >> 2) * 16 + row) * 4 + (tl & 3);
    const int64_t r = (u0 + ul) * kL4Rows + row;
    if (t0 + tl >= a.tokens || u0 + ul >= a.units || r >= a.m) continue;
    float v[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      v[q] = red[ul << a.kslog][q][at];
      for (int s = 1; s < ks; ++s) v[q] += red[(ul << a.kslog) + s][q][at];
    }
    if (GATED)
      a.ep.gated(t0 + tl, r, v[0], v[RT - 1]);
    else
      a.ep.linear(t0 + tl, r, v[0]);
  }
}

}  // namespace

W4Layout plan_w4a16_pair(int64_t m, int64_t n, int32_t group_size) {
  return plan_w4a16(2 * kL4Rows * ceil_div(m, kL4Rows), n, group_size);
}

gptq_status launch_l4_pair(const L4PairSource& src, int64_t rows, const W4Layout& L, const int32_t* order,
                           char* base, hipStream_t stream) {
  const int64_t np = L.mt * L.Gp * kL4Rows, nw = L.mt * L.kc * 256;
  hipLaunchKernelGGL(l4_pair_params_kernel, dim3((unsigned)ceil_div(np, 256)), dim3(256), 0, stream, src, rows, L.G,
                     L.Gp, np, reinterpret_cast<float2*>(base + L.param_off));
  GPTQ_LAUNCH_CHECK();
  hipLaunchKernelGGL(l4_pair_codes_kernel, dim3((unsigned)ceil_div(nw, 256)), dim3(256), 0, stream, src, rows,
                     ceil_div(L.n, 8), L.n, L.kc, nw, order, reinterpret_cast<uint32_t*>(base + L.code_off));
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

gptq_status run_w4a16_glu_pack(const L4PairSource& src, const int32_t* g_idx, const W4Layout& L, void* packed,
                               hipStream_t stream) {
  char* base = static_cast<char*>(packed);
  int* flag = reinterpret_cast<int*>(base + L.flag_off);
  int32_t* order = reinterpret_cast<int32_t*>(base + L.order_off);
  GPTQ_TRY(launch_w4_order(g_idx, L, order, flag, stream));
  GPTQ_TRY(launch_l4_pair(src, src.m, L, order, base, stream));
  return check_w4_order(flag, "gptq_w4a16_glu_pack", stream);
}

L4LinearPlan plan_w4a16_linear(int64_t tokens, int64_t n) {
  L4LinearPlan p;
  const int64_t n128 = ceil_div(n, kL4Chunk) * kL4Chunk;
  p.block = std::min<int64_t>(std::max<int64_t>(tokens, 1), kL4BlockTokens);
  p.xs_off = align256((size_t)(p.block * n128) * sizeof(uint16_t));
  p.total = p.xs_off + align256((size_t)(p.block * (n128 / 32 + n128 / 128)) * sizeof(float));
  return p;
}

gptq_status run_w4a16_linear(const L4Call& c, const W4Layout& L, bool gated, void* ws, const L4LinearPlan& p,
                             hipStream_t stream) {
  const char* base = static_cast<const char*>(c.packed);
  char* w = static_cast<char*>(ws);
  uint16_t* Xp = reinterpret_cast<uint16_t*>(w);
  float* xs = reinterpret_cast<float*>(w + p.xs_off);
  const int32_t* order = reinterpret_cast<const int32_t*>(base + L.order_off);
  L4StreamArgs a;
  a.Xp = Xp;
  a.params = reinterpret_cast<const float2*>(base + L.param_off);
  a.codes = reinterpret_cast<const u32x4_t*>(base + L.code_off);
  a.n128 = L.n128;
  a.kc = L.kc;
  a.Gp = L.Gp;
  a.units = gated ? L.mt / 2 : L.mt;
  a.m = c.m;
  const bool one_group = L.g >= L.n128;
  a.pmul = one_group ? 0 : kL4Rows;
  const int gs = one_group ? 4 : (int)(L.g / 32);
  a.kslog = L.kc >= 32 ? 3 : L.kc >= 16 ? 2 : L.kc >= 4 ? 1 : 0;
  const size_t ysz = c.y_dtype == GPTQ_FP32 ? 4 : 2, rsz = c.res_dtype == GPTQ_FP32 ? 4 : 2;
  for (int64_t t0 = 0; t0 < c.tokens; t0 += p.block) {
    const int64_t tk = std::min<int64_t>(p.block, c.tokens - t0);
    GPTQ_TRY(launch_w4_gather(c.X + t0 * c.ldx, c.ldx, order, L.n128, Xp, xs, xs + tk * (L.n128 / 32), tk, stream));
    a.tokens = tk;
    a.ep = L4Epilogue{c.act, c.bias_dtype, c.res_dtype, c.y_dtype, c.bias, c.bias2,
                      c.res ? static_cast<const char*>(c.res) + (size_t)(t0 * c.ldr) * rsz : nullptr,
                      static_cast<char*>(c.Y) + (size_t)(t0 * c.ldy) * ysz, c.ldr, c.ldy};
    const dim3 grid((unsigned)ceil_div(a.units, 8 >> a.kslog), (unsigned)ceil_div(tk, 16));
#define L4_STREAM(GS)                                                                            \
  if (gated)                                                                                     \
    hipLaunchKernelGGL((l4_stream_kernel<GS, true>), grid, dim3(512), 0, stream, a);             \
  else                                                                                           \
    hipLaunchKernelGGL((l4_stream_kernel<GS, false>), grid, dim3(512), 0, stream, a)
    switch (gs) {
      case 1: L4_STREAM(1); break;
      case 2: L4_STREAM(2); break;
      default: L4_STREAM(4); break;
    }
#undef L4_STREAM
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

}  // namespace gptq
