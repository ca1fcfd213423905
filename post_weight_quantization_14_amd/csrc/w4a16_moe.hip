// A mixture-of-experts layer on packed 2/3/4-bit weights, for a few tokens.
//
//   p = softmax(x·Rᵀ), e_1..e_k = the k largest (ties: the lower expert),
//   w_j = p[e_j] (divided by their sum if renormalised),
//   y = Σ_j w_j·Ŵd_e(act(Ŵg_e·x) ⊙ (Ŵu_e·x)) + residual.
//
// An expert's blob (gptq_w4a16_moe_pack) holds gate and up as one packed
// weight of alternating 16-row tiles, its rows in the down projection's
// processing order, and the down projection as its own packed weight: what
// the gate/up kernel writes is the down kernel's operand as it lies, with no
// gather between them.
//
// Launches for up to 64 tokens: router (a workgroup per token), gate/up (a
// workgroup per active expert and row tiles), down (the same), combine.
#include <algorithm>

#include "w4a16_device.hpp"

namespace gptq {
namespace {

constexpr int kMoeTokens = 64;       // tokens per launch sequence: one lane each
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 64;
constexpr int kMoeMaxPlanes = 3;     // bf16 parts of the hidden activation
constexpr int kMoePass = 16;         // tokens of one expert per pass (MFMA M)

// ---------------------------------------------------------------- router
struct MoeRouterArgs {
  const uint16_t* X;
  int64_t ldx, hidden;
  const void* R;          // [experts][hidden]
  int r_dt, experts, top_k, renorm, vec;
  int32_t* ids;           // [tokens][top_k]
  float* wts;
  int32_t* ids_out;       // the caller's copies, may be null
  float* wts_out;
};

// a before b: larger, NaN above every number, ties to the lower index
__device__ __forceinline__ bool moe_before(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na != nb) return na;
  if (!na && a != b) return a > b;
  return ia < ib;
}

// One workgroup per token.  The logits are summed in 64 bits: which experts
// are chosen hangs on the last bits of the k-th and the next, and a choice
// that falls the other way is no rounding error in the result.
__global__ __launch_bounds__(1024) void moe_router_kernel(MoeRouterArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t t = blockIdx.x, h = a.hidden;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  double* logit = reinterpret_cast<double*>(lds);
  float* x = reinterpret_cast<float*>(lds + (size_t)a.experts * sizeof(double) + (a.experts & 1) * sizeof(double));
  for (int64_t i = tid; i < h; i += blockDim.x) x[i] = __uint_as_float((uint32_t)a.X[t * a.ldx + i] << 16);
  __syncthreads();
  for (int e = wave; e < a.experts; e += waves) {
    double s0 = 0.0, s1 = 0.0;
    if (a.vec && a.r_dt == GPTQ_BF16) {
      const uint16_t* r = static_cast<const uint16_t*>(a.R) + (int64_t)e * h;
      for (int64_t i = 8 * lane; i < h; i += 512) {
        const uint4 w = *reinterpret_cast<const uint4*>(r + i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s0 += (double)(x[i + 2 * q] * __uint_as_float(ww[q] << 16));   // bf16·bf16: exact in fp32
          s1 += (double)(x[i + 2 * q + 1] * __uint_as_float(ww[q] & 0xffff0000u));
        }
      }
    } else {
      for (int64_t i = lane; i < h; i += 64) s0 = fma((double)x[i], (double)l4_load(a.R, a.r_dt, (int64_t)e * h + i), s0);
    }
    s0 += s1;
#pragma unroll
    for (int d = 32; d; d >>= 1) s0 += __shfl_xor(s0, d);
    if (lane == 0) logit[e] = s0;
  }
  __syncthreads();
  if (wave != 0) return;
  // lane l holds experts l, l + 64, ...; taken = those already chosen
  uint32_t taken = 0;
  double top = 0.0, chosen = 0.0, mine = 0.0;
  int my_id = 0;
  for (int j = 0; j < a.top_k; ++j) {
    double bv = 0.0;
    int bi = kMoeMaxExperts;   // none
    for (int e = lane, q = 0; e < a.experts; e += 64, ++q)
      if (!(taken >> q & 1) && (bi == kMoeMaxExperts || moe_before(logit[e], e, bv, bi))) {
        bv = logit[e];
        bi = e;
      }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const double ov = __shfl_xor(bv, d);
      const int oi = __shfl_xor(bi, d);
      if (oi != kMoeMaxExperts && (bi == kMoeMaxExperts || moe_before(ov, oi, bv, bi))) {
        bv = ov;
        bi = oi;
      }
    }
    if ((bi & 63) == lane) taken |= 1u << (bi >> 6);
    if (j == 0) top = bv;
    const double p = exp(bv - top);
    chosen += p;
    if (lane == j) {
      mine = p;
      my_id = bi;
    }
  }
  if (!a.renorm) {
    chosen = 0.0;
    for (int e = lane; e < a.experts; e += 64) chosen += exp(logit[e] - top);
#pragma unroll
    for (int d = 32; d; d >>= 1) chosen += __shfl_xor(chosen, d);
  }
  if (lane < a.top_k) {
    const float w = (float)(mine / chosen);
    a.ids[t * a.top_k + lane] = my_id;
    a.wts[t * a.top_k + lane] = w;
    if (a.ids_out) a.ids_out[t * a.top_k + lane] = my_id;
    if (a.wts_out) a.wts_out[t * a.top_k + lane] = w;
  }
}

// ---------------------------------------------------------------- experts
struct MoeList {
  uint32_t used[kMoeMaxExperts / 32];
  int pair[kMoeTokens];   // pairs t·top_k + j of the expert, tokens ascending
  int count;
};

// The slot-th expert that any token chose (-1: there are fewer), and its
// pairs.  Every thread calls it; ends with a barrier.
__device__ __forceinline__ int moe_expert(const int32_t* __restrict__ ids, int tokens, int top_k, int experts,
                                          int slot, MoeList& L) {
  const int tid = threadIdx.x;
  if (tid < kMoeMaxExperts / 32) L.used[tid] = 0;
  __syncthreads();
  for (int i = tid; i < tokens * top_k; i += blockDim.x) atomicOr(&L.used[ids[i] >> 5], 1u << (ids[i] & 31));
  __syncthreads();
  int e = -1, left = slot;
  for (int w = 0; w < (experts + 31) / 32; ++w) {
    uint32_t b = L.used[w];
    const int n = __popc(b);
    if (left < n) {
      while (left--) b &= b - 1;
      e = 32 * w + __ffs(b) - 1;
      break;
    }
    left -= n;
  }
  if (e >= 0 && tid < 64) {
    int p = -1;
    if (tid < tokens)
      for (int j = 0; j < top_k; ++j)
        if (ids[tid * top_k + j] == e) p = tid * top_k + j;
    const uint64_t hit = __ballot(p >= 0);
    if (p >= 0) L.pair[__popcll(hit & ((1ull << tid) - 1ull))] = p;
    if (tid == 0) L.count = __popcll(hit);
  }
  __syncthreads();
  return e;
}

struct L4LdsA {
  static constexpr bool kPrefetch = false;
  const uint16_t* row;   // this lane's token row + 8·(lane/16)
  __device__ __forceinline__ uint4 load(int c, int j, int) const {
    return *reinterpret_cast<const uint4*>(row + c * kL4Chunk + 32 * j);
  }
};

struct MoeGateUpArgs {
  const uint16_t* X;
  int64_t ldx;
  const char* packed;         // expert e's blob at e·stride
  int64_t stride;
  int64_t order_off, param_off, code_off;
  int64_t n128, kc, Gp, units, f128;
  const int32_t* ids;
  uint16_t* mid;              // [pairs][planes][f128]: bf16 parts, largest first
  int tokens, top_k, experts, pmul, kslog, act, pass, planes;
};

// act(gate)·up of one expert's tokens for 8 >> kslog tile pairs.  X' =
// X[:, order] of up to `pass` tokens sits in LDS in processing order.
template <int GS>
__global__ __launch_bounds__(512) void moe_gate_up_kernel(MoeGateUpArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ MoeList list;
  __shared__ float red[8][2][256];
  uint16_t* xsh = reinterpret_cast<uint16_t*>(lds);
  const int xrow = (int)a.n128 + 8;   // rows 16 bytes apart in the banks
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = __builtin_amdgcn_readfirstlane(moe_expert(a.ids, a.tokens, a.top_k, a.experts, blockIdx.y, list));
  if (e < 0) return;
  const char* blob = a.packed + e * a.stride;
  const int32_t* order = reinterpret_cast<const int32_t*>(blob + a.order_off);
  const int ks = 1 << a.kslog, upw = 8 >> a.kslog;
  const int64_t u0 = (int64_t)blockIdx.x * upw;
  const int64_t unit = std::min<int64_t>(u0 + (wave >> a.kslog), a.units - 1);
  const int sl = wave & (ks - 1);
  const int cps = (int)((a.kc + ks - 1) >> a.kslog);
  const int c0 = sl * cps, c1 = (int)std::min<int64_t>(a.kc, c0 + cps);
  const u32x4_t* cp[2];
  const float2* pp[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    cp[r] = reinterpret_cast<const u32x4_t*>(blob + a.code_off) + (unit * 2 + r) * a.kc * 64 + lane;
    pp[r] = reinterpret_cast<const float2*>(blob + a.param_off) + (unit * 2 + r) * a.Gp * kL4Rows + (lane & 15);
  }
  const L4Consts kc;
  for (int p0 = 0; p0 < list.count; p0 += a.pass) {
    const int np = std::min(a.pass, list.count - p0);
    for (int i = tid; i < np * (int)(a.n128 / 4); i += 512) {
      const int q = i / (int)(a.n128 / 4), p = 4 * (i % (int)(a.n128 / 4));
      const uint16_t* x = a.X + (int64_t)(list.pair[p0 + q] / a.top_k) * a.ldx;
      const int4 o = *reinterpret_cast<const int4*>(order + p);
      uint2 v;
      v.x = (o.x >= 0 ? (uint32_t)x[o.x] : 0u) | ((o.y >= 0 ? (uint32_t)x[o.y] : 0u) << 16);
      v.y = (o.z >= 0 ? (uint32_t)x[o.z] : 0u) | ((o.w >= 0 ? (uint32_t)x[o.w] : 0u) << 16);
      *reinterpret_cast<uint2*>(xsh + q * xrow + p) = v;
    }
    __syncthreads();
    const L4LdsA af{xsh + std::min(lane & 15, np - 1) * xrow + 8 * (lane >> 4)};
    f32x4_t y[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    l4_stream<GS, 2, 1, 2, false>(af, cp, pp, a.pmul, c0, c1, kc, y);
#pragma unroll
    for (int r = 0; r < 2; ++r) *reinterpret_cast<f32x4_t*>(&red[wave][r][lane * 4]) = y[r];
    __syncthreads();
    for (int i = tid; i < upw * 256; i += 512) {
      const int ul = i >> 8, q = (i >> 4) & 15, row = i & 15;
      const int at = ((q >> 2) * 16 + row) * 4 + (q & 3);
      if (q >= np || u0 + ul >= a.units) continue;
      float g = red[ul << a.kslog][0][at], u = red[ul << a.kslog][1][at];
      for (int s = 1; s < ks; ++s) {
        g += red[(ul << a.kslog) + s][0][at];
        u += red[(ul << a.kslog) + s][1][at];
      }
      // The hidden activation leaves as 2 or 3 bf16 parts (16 or 24 significant
      // bits, for a bf16 or an fp32 result), so it adds no rounding of its own;
      // a single bf16 would add as much error as the result's rounding.
      float v = l4_activate(g, a.act) * u;
      uint16_t* o = a.mid + (int64_t)list.pair[p0 + q] * a.planes * a.f128 + (u0 + ul) * kL4Rows + row;
      for (int p = 0; p < a.planes; ++p) {
        const uint16_t part = l4_bf16(v);
        const float f = __uint_as_float((uint32_t)part << 16);
        o[p * a.f128] = part;
        v = isfinite(f) ? v - f : 0.f;
      }
    }
    __syncthreads();
  }
}

struct MoeDownArgs {
  const uint16_t* mid;
  const char* packed;
  int64_t stride, param_off, code_off;
  int64_t f128, kc, Gp, units, hidden;
  const int32_t* ids;
  float* out;                 // [pairs][hidden]
  int tokens, top_k, experts, pmul, kslog;
};

template <int GS, int NP>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeDownArgs a) {
  __shared__ MoeList list;
  __shared__ float red[8][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = __builtin_amdgcn_readfirstlane(moe_expert(a.ids, a.tokens, a.top_k, a.experts, blockIdx.y, list));
  if (e < 0) return;
  const char* blob = a.packed + e * a.stride;
  const int ks = 1 << a.kslog, upw = 8 >> a.kslog;
  const int64_t u0 = (int64_t)blockIdx.x * upw;
  const int64_t unit = std::min<int64_t>(u0 + (wave >> a.kslog), a.units - 1);
  const int sl = wave & (ks - 1);
  const int cps = (int)((a.kc + ks - 1) >> a.kslog);
  const int c0 = sl * cps, c1 = (int)std::min<int64_t>(a.kc, c0 + cps);
  const u32x4_t* cp[1] = {reinterpret_cast<const u32x4_t*>(blob + a.code_off) + unit * a.kc * 64 + lane};
  const float2* pp[1] = {reinterpret_cast<const float2*>(blob + a.param_off) + unit * a.Gp * kL4Rows + (lane & 15)};
  const L4Consts kc;
  for (int p0 = 0; p0 < list.count; p0 += kMoePass) {
    const int np = std::min(kMoePass, list.count - p0);
    const L4GlobalA af{a.mid + (int64_t)list.pair[p0 + std::min(lane & 15, np - 1)] * NP * a.f128 + 8 * (lane >> 4),
                       a.f128};
    f32x4_t y[1] = {{0.f, 0.f, 0.f, 0.f}};
    l4_stream<GS, 1, NP, 2, NP == 3>(af, cp, pp, a.pmul, c0, c1, kc, y);
    *reinterpret_cast<f32x4_t*>(&red[wave][lane * 4]) = y[0];
    __syncthreads();
    for (int i = tid; i < upw * 256; i += 512) {
      const int ul = i >> 8, q = (i >> 4) & 15, row = i & 15;
      const int at = ((q >> 2) * 16 + row) * 4 + (q & 3);
      const int64_t r = (u0 + ul) * kL4Rows + row;
      if (q >= np || u0 + ul >= a.units || r >= a.hidden) continue;
      float v = red[ul << a.kslog][at];
      for (int s = 1; s < ks; ++s) v += red[(ul << a.kslog) + s][at];
      a.out[(int64_t)list.pair[p0 + q] * a.hidden + r] = v;
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ pairs, const float* __restrict__ wts,
                                                          int top_k, int64_t hidden, const void* res, int res_dt,
                                                          int64_t ldr, void* Y, int y_dt, int64_t ldy) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (r >= hidden) return;
  float v = 0.f;
  for (int j = 0; j < top_k; ++j) v = fmaf(wts[t * top_k + j], pairs[(t * top_k + j) * hidden + r], v);
  if (res) v += l4_load(res, res_dt, t * ldr + r);
  l4_store(Y, y_dt, t * ldy + r, v);
}

int ks_log(int64_t kc) { return kc >= 32 ? 3 : kc >= 16 ? 2 : kc >= 4 ? 1 : 0; }

}  // namespace

MoeLayout plan_moe(const gptq_moe_config& c) {
  MoeLayout L;
  L.f128 = ceil_div(c.inter, kL4Chunk) * kL4Chunk;
  L.gu = plan_w4a16_pair(L.f128, c.hidden, c.group_size);
  L.down = plan_w4a16(c.hidden, c.inter, c.group_size);
  L.down_off = align256(L.gu.total);
  L.stride = L.down_off + align256(L.down.total);
  return L;
}

MoeWork plan_moe_work(const gptq_moe_config& c, int64_t tokens) {
  MoeWork w;
  w.block = std::min<int64_t>(std::max<int64_t>(tokens, 1), kMoeTokens);
  const size_t pairs = (size_t)(w.block * c.top_k);
  const size_t f128 = (size_t)(ceil_div(c.inter, kL4Chunk) * kL4Chunk);
  w.wts_off = align256(pairs * sizeof(int32_t));
  w.mid_off = w.wts_off + align256(pairs * sizeof(float));
  w.out_off = w.mid_off + align256(pairs * kMoeMaxPlanes * f128 * sizeof(uint16_t));
  w.total = w.out_off + align256(pairs * (size_t)c.hidden * sizeof(float));
  return w;
}

gptq_status run_moe_pack(const gptq_moe_config& c, int expert, const L4PairSource& gate_up, const int32_t* g_idx,
                         const uint32_t* down_qweight, const float* down_scales, const int32_t* down_zeros,
                         const int32_t* down_g_idx, void* packed, hipStream_t stream) {
  const MoeLayout L = plan_moe(c);
  char* base = static_cast<char*>(packed) + (size_t)expert * L.stride;
  GPTQ_TRY(run_w4a16_pack(down_qweight, down_scales, down_zeros, down_g_idx, c.bits, L.down, base + L.down_off, stream));
  int* flag = reinterpret_cast<int*>(base + L.gu.flag_off);
  int32_t* order = reinterpret_cast<int32_t*>(base + L.gu.order_off);
  GPTQ_TRY(launch_w4_order(g_idx, L.gu, order, flag, stream));
  L4PairSource src = gate_up;
  src.row_order = reinterpret_cast<const int32_t*>(base + L.down_off + L.down.order_off);
  GPTQ_TRY(launch_l4_pair(src, L.f128, L.gu, order, base, stream));
  return check_w4_order(flag, "gptq_w4a16_moe_pack", stream);
}

gptq_status run_moe(const MoeCall& c, const gptq_moe_config& cfg, void* ws, const MoeWork& w, hipStream_t stream) {
  const MoeLayout L = plan_moe(cfg);
  char* wb = static_cast<char*>(ws);
  int32_t* ids = reinterpret_cast<int32_t*>(wb);
  float* wts = reinterpret_cast<float*>(wb + w.wts_off);
  uint16_t* mid = reinterpret_cast<uint16_t*>(wb + w.mid_off);
  float* out = reinterpret_cast<float*>(wb + w.out_off);
  const size_t ysz = c.y_dtype == GPTQ_FP32 ? 4 : 2, rsz = c.res_dtype == GPTQ_FP32 ? 4 : 2;
  const char* packed = static_cast<const char*>(c.packed);
  const int h = (int)cfg.hidden;

  MoeGateUpArgs g;
  g.ldx = c.ldx;
  g.packed = packed;
  g.stride = (int64_t)L.stride;
  g.order_off = (int64_t)L.gu.order_off;
  g.param_off = (int64_t)L.gu.param_off;
  g.code_off = (int64_t)L.gu.code_off;
  g.n128 = L.gu.n128;
  g.kc = L.gu.kc;
  g.Gp = L.gu.Gp;
  g.units = L.gu.mt / 2;
  g.f128 = L.f128;
  g.ids = ids;
  g.mid = mid;
  g.top_k = cfg.top_k;
  g.experts = cfg.experts;
  g.pmul = L.gu.g >= L.gu.n128 ? 0 : kL4Rows;
  g.kslog = ks_log(L.gu.kc);
  g.act = cfg.activation;
  g.planes = c.y_dtype == GPTQ_FP32 ? 3 : 2;
  MoeDownArgs d;
  d.mid = mid;
  d.packed = packed + L.down_off;
  d.stride = (int64_t)L.stride;
  d.param_off = (int64_t)L.down.param_off;
  d.code_off = (int64_t)L.down.code_off;
  d.f128 = L.f128;
  d.kc = L.down.kc;
  d.Gp = L.down.Gp;
  d.units = L.down.mt;
  d.hidden = cfg.hidden;
  d.ids = ids;
  d.out = out;
  d.top_k = cfg.top_k;
  d.experts = cfg.experts;
  d.pmul = L.down.g >= L.down.n128 ? 0 : kL4Rows;
  d.kslog = ks_log(L.down.kc);
  const size_t row = (size_t)(g.n128 + 8) * sizeof(uint16_t);
  // one group per row folds as groups of 128 (pmul = 0 repeats its parameters)
  auto steps = [&](const W4Layout& l) { return l.g >= l.n128 ? 4 : (int)(l.g / 32); };

  for (int64_t t0 = 0; t0 < c.tokens; t0 += w.block) {
    const int tk = (int)std::min<int64_t>(w.block, c.tokens - t0);
    MoeRouterArgs r;
    r.X = c.X + t0 * c.ldx;
    r.ldx = c.ldx;
    r.hidden = cfg.hidden;
    r.R = c.router;
    r.r_dt = c.router_dtype;
    r.experts = cfg.experts;
    r.top_k = cfg.top_k;
    r.renorm = cfg.renormalize;
    r.vec = h % 8 == 0 && (reinterpret_cast<uintptr_t>(c.router) & 15) == 0;
    r.ids = ids;
    r.wts = wts;
    r.ids_out = c.topk_ids ? c.topk_ids + t0 * cfg.top_k : nullptr;
    r.wts_out = c.topk_weights ? c.topk_weights + t0 * cfg.top_k : nullptr;
    const size_t rlds = (size_t)round_up(cfg.experts, 2) * sizeof(double) + (size_t)h * sizeof(float);
    if (rlds > 65536)
      GPTQ_HIP_CHECK(hipFuncSetAttribute((const void*)moe_router_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)rlds));
    hipLaunchKernelGGL(moe_router_kernel, dim3((unsigned)tk), dim3(1024), rlds, stream, r);
    GPTQ_LAUNCH_CHECK();

    const unsigned slots = (unsigned)std::min<int64_t>(cfg.experts, (int64_t)tk * cfg.top_k);
    g.X = r.X;
    g.tokens = d.tokens = tk;
    g.pass = (int)std::min<size_t>({(size_t)kMoePass, (size_t)tk, (size_t)(128 * 1024) / row});
    const size_t glds = row * (size_t)g.pass;
    const dim3 ggrid((unsigned)ceil_div(g.units, 8 >> g.kslog), slots);
    const dim3 dgrid((unsigned)ceil_div(d.units, 8 >> d.kslog), slots);
#define MOE_GATE_UP(GS)                                                                                          \
  do {                                                                                                           \
    if (glds > 32768)                                                                                            \
      GPTQ_HIP_CHECK(hipFuncSetAttribute((const void*)moe_gate_up_kernel<GS>,                                    \
                                         hipFuncAttributeMaxDynamicSharedMemorySize, (int)glds));                \
    hipLaunchKernelGGL(moe_gate_up_kernel<GS>, ggrid, dim3(512), glds, stream, g);                               \
  } while (0)
    switch (steps(L.gu)) {
      case 1: MOE_GATE_UP(1); break;
      case 2: MOE_GATE_UP(2); break;
      default: MOE_GATE_UP(4); break;
    }
#undef MOE_GATE_UP
    GPTQ_LAUNCH_CHECK();
#define MOE_DOWN(GS)                                                                                             \
  if (g.planes == 3)                                                                                             \
    hipLaunchKernelGGL((moe_down_kernel<GS, 3>), dgrid, dim3(512), 0, stream, d);                                \
  else                                                                                                           \
    hipLaunchKernelGGL((moe_down_kernel<GS, 2>), dgrid, dim3(512), 0, stream, d)
    switch (steps(L.down)) {
      case 1: MOE_DOWN(1); break;
      case 2: MOE_DOWN(2); break;
      default: MOE_DOWN(4); break;
    }
#undef MOE_DOWN
    GPTQ_LAUNCH_CHECK();
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)ceil_div(cfg.hidden, 256), (unsigned)tk), dim3(256), 0, stream,
                       (const float*)out, (const float*)wts, (int)cfg.top_k, cfg.hidden,
                       c.res ? (const void*)(static_cast<const char*>(c.res) + (size_t)(t0 * c.ldr) * rsz) : nullptr,
                       c.res_dtype, c.ldr, (void*)(static_cast<char*>(c.Y) + (size_t)(t0 * c.ldy) * ysz), c.y_dtype, c.ldy);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

}  // namespace gptq
