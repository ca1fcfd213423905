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
// Launches for up to 64 tokens: router (a workgroup per token; it also gathers
// the token into each chosen expert's column order; its logits come from a
// launch of their own where there are many), gate/up and down (some workgroups
// per active expert, each a share of its row tiles), combine.  A token or a few
// take two: see below.
//
// Bound by the chosen experts' codes and parameters from HBM: 64 tokens, 64
// experts of 2048 x 1024, top 6: gate/up 39 us = 4.2 TB/s, down 25 us, router
// 10 us, 81 us in all; 1 token, 8 experts of 4096 x 11008, top 2: 33 us and
// 20 us, 55 us in all.
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
  int r_dt, experts, top_k, renorm, vec, xvec, parts;
  int32_t* ids;           // [tokens][top_k]
  float* wts;
  int32_t* ids_out;       // the caller's copies, may be null
  float* wts_out;
  const char* packed;     // expert e's column order at e·stride + order_off
  int64_t stride, order_off, n128;
  uint16_t* Xp;           // [pairs][n128]
  double* logits;         // [tokens][experts] of moe_logits_kernel, or null: computed here
};

// a before b: larger, NaN above every number, ties to the lower index
__device__ __forceinline__ bool moe_before(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na != nb) return na;
  if (!na && a != b) return a > b;
  return ia < ib;
}

// A token's row in LDS ends with eight zeros, which lanes past its end read: an
// Inf of x, from anywhere else in the row, times their zero of the router would
// be NaN.  (Selecting zeros after the read: router 9.2 -> 11.3 us.)
constexpr int kMoeTail = 8;
__device__ __forceinline__ void moe_tail(uint16_t* x, int h, int i) {   // i = 0 .. 7
  x[((h + 7) & ~7) + i] = 0;
}
__device__ __forceinline__ u32x4_t moe_x(const uint16_t* x, int k, int h) {   // h % 8 == 0
  return *reinterpret_cast<const u32x4_t*>(x + (k < h ? k : h));
}

// One logit in 64 bits by one wave: `part` of `parts` interleaved 512-element
// pieces, four pieces in flight.
__device__ __forceinline__ double moe_logit(const uint16_t* x, const void* R, int r_dt, int vec, int64_t e, int h,
                                            int part, int parts) {
  const int lane = threadIdx.x & 63;
  double s0 = 0.0, s1 = 0.0;
  if (vec && r_dt == GPTQ_BF16) {
    const uint16_t* r = static_cast<const uint16_t*>(R) + e * h;
    for (int b = 512 * part; b < h; b += 2048 * parts) {
      u32x4_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = b + 512 * parts * u + 8 * lane;
        w[u] = *reinterpret_cast<const u32x4_t*>(r + (k < h ? k : 0));
        if (k >= h) w[u] = u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = b + 512 * parts * u + 8 * lane;
        const u32x4_t xv = moe_x(x, k, h);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s0 = fma((double)__uint_as_float(xv[q] << 16), (double)__uint_as_float(w[u][q] << 16), s0);
          s1 = fma((double)__uint_as_float(xv[q] & 0xffff0000u), (double)__uint_as_float(w[u][q] & 0xffff0000u), s1);
        }
      }
    }
  } else if (vec) {
    const float* r = static_cast<const float*>(R) + e * h;
    for (int b = 512 * part; b < h; b += 1024 * parts) {
      f32x4_t w[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = b + 512 * parts * u + 8 * lane;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          w[u][q] = *reinterpret_cast<const f32x4_t*>(r + (k < h ? k : 0) + 4 * q);
          if (k >= h) w[u][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = b + 512 * parts * u + 8 * lane;
        const u32x4_t xv = moe_x(x, k, h);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s0 = fma((double)__uint_as_float(xv[q] << 16), (double)w[u][q >> 1][2 * (q & 1)], s0);
          s1 = fma((double)__uint_as_float(xv[q] & 0xffff0000u), (double)w[u][q >> 1][2 * (q & 1) + 1], s1);
        }
      }
    }
  } else {
    // rows that are not 16-byte aligned: element by element, 16 in flight (the
    // type's branch outside: inside, each load is a block with its own wait)
    constexpr int U = 16;
    for (int b = 64 * part; b < h; b += 64 * U * parts) {
      float w[U];
      if (r_dt == GPTQ_FP32) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = b + 64 * parts * u + lane;
          w[u] = static_cast<const float*>(R)[e * h + (i < h ? i : 0)];
        }
      } else {
        uint16_t q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = b + 64 * parts * u + lane;
          q[u] = static_cast<const uint16_t*>(R)[e * h + (i < h ? i : 0)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = __uint_as_float((uint32_t)q[u] << 16);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = b + 64 * parts * u + lane;
        const float xi = __uint_as_float((uint32_t)x[i < h ? i : 0] << 16);
        s0 = fma(i < h ? (double)xi : 0.0, i < h ? (double)w[u] : 0.0, s0);
      }
    }
  }
  s0 += s1;
#pragma unroll
  for (int d = 32; d; d >>= 1) s0 += __shfl_xor(s0, d);
  return s0;
}

// Logits of 16 experts (grid x) for a token (grid y), a wave each: where there
// are many, on all CUs instead of one per token (64 tokens, 64 experts of
// 2048: the router's 15 us become 5 + 6).
__global__ __launch_bounds__(1024) void moe_logits_kernel(MoeRouterArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t t = blockIdx.y;
  const int h = (int)a.hidden, tid = threadIdx.x;
  const int e = blockIdx.x * 16 + (tid >> 6);
  l4_row_to_lds(a.X + t * a.ldx, h, a.xvec, lds, tid, 1024);
  if (tid < kMoeTail) moe_tail(reinterpret_cast<uint16_t*>(lds), h, tid);
  __syncthreads();
  if (e >= a.experts) return;
  const double s = moe_logit(reinterpret_cast<const uint16_t*>(lds), a.R, a.r_dt, a.vec, e, h, 0, 1);
  if ((tid & 63) == 0) a.logits[t * a.experts + e] = s;
}

// One workgroup per token.  The logits are summed in 64 bits: which experts
// are chosen hangs on the last bits of the k-th and the next, and a choice
// that falls the other way is no rounding error in the result.  `parts` waves
// share an expert's row when there are fewer experts than waves.
//
// Then every expert's rank is the number of experts before it, counted by all
// threads together (a chain of top_k wave-wide maxima took three times as
// long), and the token is gathered into the column order of each chosen one.
__global__ __launch_bounds__(1024) void moe_router_kernel(MoeRouterArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int chosen[kMoeMaxTopK];
  __shared__ double total[16];
  const int64_t t = blockIdx.x;
  const int h = (int)a.hidden, E = a.experts;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  double* logit = reinterpret_cast<double*>(lds);                      // [parts][experts]
  int* rank = reinterpret_cast<int*>(logit + (((size_t)a.parts * E + 1) & ~(size_t)1));
  uint16_t* x = reinterpret_cast<uint16_t*>(rank + ((E + 3) & ~3));
  const int part = wave % a.parts, wpe = 16 / a.parts, e0 = wave / a.parts;
  const bool fast = a.vec && a.r_dt == GPTQ_BF16;
  const uint16_t* R = static_cast<const uint16_t*>(a.R);
  // four 512-element pieces of a row; past its end zeros
  auto fetch = [&](int e, int i, u32x4_t (&w)[4]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = i + 512 * a.parts * u;
      const bool in = k < h && e < E;
      w[u] = *reinterpret_cast<const u32x4_t*>(R + (in ? (int64_t)e * h + k : 0));
      if (!in) w[u] = u32x4_t{0u, 0u, 0u, 0u};
    }
  };
  const int i0 = 8 * lane + 512 * part, istep = 2048 * a.parts;
  u32x4_t w[4], nx[4];
  if (fast && !a.logits) fetch(e0, i0, w);   // in flight while the token is copied
  l4_row_to_lds(a.X + t * a.ldx, h, a.xvec, reinterpret_cast<uint8_t*>(x), tid, 1024);
  if (tid < kMoeTail) moe_tail(x, h, tid);
  for (int e = tid; e < E; e += 1024) rank[e] = 0;
  __syncthreads();
  if (a.logits)
    for (int e = tid; e < E; e += 1024) logit[e] = a.logits[t * E + e];
  for (int e = a.logits ? E : e0; e < E; e += wpe) {
    double s0 = 0.0, s1 = 0.0;
    if (fast) {
      for (int i = i0; i - 8 * lane < h; i += istep) {
        const bool more = i + istep - 8 * lane < h;
        fetch(more ? e : e + wpe, more ? i + istep : i0, nx);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = i + 512 * a.parts * u;
          const u32x4_t xv = moe_x(x, k, h);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            s0 = fma((double)__uint_as_float(xv[q] << 16), (double)__uint_as_float(w[u][q] << 16), s0);
            s1 = fma((double)__uint_as_float(xv[q] & 0xffff0000u), (double)__uint_as_float(w[u][q] & 0xffff0000u), s1);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = nx[u];
      }
      s0 += s1;
#pragma unroll
      for (int d = 32; d; d >>= 1) s0 += __shfl_xor(s0, d);
    } else {
      s0 = moe_logit(x, a.R, a.r_dt, a.vec, e, h, part, a.parts);
    }
    if (lane == 0) logit[part * E + e] = s0;
  }
  __syncthreads();
  if (a.parts > 1) {
    if (tid < E)
      for (int p = 1; p < a.parts; ++p) logit[tid] += logit[p * E + tid];
    __syncthreads();
  }
  // segs threads per expert, each comparing it with every segs-th other
  int slog = 0;
  while ((E << (slog + 1)) <= 1024) ++slog;
  for (int i = tid; i < E << slog; i += 1024) {
    const int e = i >> slog;
    const double mine = logit[e];
    int before = 0;
    for (int o = i & ((1 << slog) - 1); o < E; o += 1 << slog) before += o != e && moe_before(logit[o], o, mine, e);
    if (before) atomicAdd(&rank[e], before);
  }
  __syncthreads();
  for (int e = tid; e < E; e += 1024)
    if (rank[e] < a.top_k) chosen[rank[e]] = e;
  __syncthreads();
  const double top = logit[chosen[0]];
  if (!a.renorm) {   // the sum over all experts, wave by wave
    double s = 0.0;
    for (int e = tid; e < E; e += 1024) s += exp(logit[e] - top);
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) total[wave] = s;
    __syncthreads();
  }
  if (wave == 0) {
    const double mine = lane < a.top_k ? exp(logit[chosen[lane]] - top) : 0.0;
    double sum = 0.0;
    if (a.renorm) {
      sum = mine;
#pragma unroll
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    } else {
      for (int v = 0; v < 16; ++v) sum += total[v];
    }
    if (lane < a.top_k) {
      const float wt = (float)(mine / sum);
      const int64_t at = t * a.top_k + lane;
      a.ids[at] = chosen[lane];
      a.wts[at] = wt;
      if (a.ids_out) a.ids_out[at] = chosen[lane];
      if (a.wts_out) a.wts_out[at] = wt;
    }
  }
  // the token in the column order of each of its experts
  const int quarter = (int)(a.n128 / 4);
  for (int i = tid; i < a.top_k * quarter; i += 1024) {
    const int j = i / quarter, p = 4 * (i % quarter);
    const int4 o = *reinterpret_cast<const int4*>(a.packed + chosen[j] * a.stride + a.order_off + (int64_t)p * 4);
    const uint32_t v0 = x[std::max(o.x, 0)], v1 = x[std::max(o.y, 0)], v2 = x[std::max(o.z, 0)], v3 = x[std::max(o.w, 0)];
    uint2 v;
    v.x = (o.x >= 0 ? v0 : 0u) | (o.y >= 0 ? v1 : 0u) << 16;
    v.y = (o.z >= 0 ? v2 : 0u) | (o.w >= 0 ? v3 : 0u) << 16;
    *reinterpret_cast<uint2*>(a.Xp + (t * a.top_k + j) * a.n128 + p) = v;
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

struct MoeExpertArgs {
  const char* packed;         // expert e's weight at e·stride
  int64_t stride, param_off, code_off;
  L4Stream st;
  const uint16_t* A;          // [pairs][planes][k128], processing order
  int64_t k128;               // positions of the product's input
  const int32_t* ids;
  int tokens, top_k, experts, pass, quads, act, planes, slices;
  int64_t rows;               // gate/up: f128 (positions); down: hidden
  uint16_t* mid;              // gate/up's result [pairs][planes][rows]: bf16 parts, largest first
  float* out;                 // down's result [slices][pairs][rows]
};

// act(gate)·up of one pair and row.  It leaves as 2 or 3 bf16 parts (16 or 24
// significant bits, for a bf16 or an fp32 result), so it adds no rounding of
// its own; a single bf16 would add as much error as the result's rounding.
template <int RT>
__device__ __forceinline__ void moe_hidden(const MoeExpertArgs& a, int64_t pair, int64_t r, const float (&z)[RT]) {
  float v = l4_activate(z[0], a.act) * z[RT - 1];
  uint16_t* o = a.mid + pair * a.planes * a.rows + r;
  for (int p = 0; p < a.planes; ++p) {
    uint16_t part = l4_bf16(v);
    if ((part & 0x7fff) == 0x7f80) part = (uint16_t)(__float_as_uint(v) >> 16);   // finite v that rounds to Inf: cut
    const float f = __uint_as_float((uint32_t)part << 16);
    o[p * a.rows] = part;
    v = isfinite(f) ? v - f : 0.f;
  }
}

// A workgroup's share of one expert's units, NP planes of A per token.  LDS:
// the rows of a pass are copied into LDS, else every fragment is read from
// memory.  GATE_UP: RT = 2, act(gate)·up to `mid`; else to `out`.
template <int GS, bool GATE_UP, int NP, bool LDS>
__device__ __forceinline__ void moe_expert_units(const MoeExpertArgs& a, MoeList& list, uint8_t* lds) {
  constexpr int RT = GATE_UP ? 2 : 1;
  // batches that leave the wave within 128 registers
  constexpr int B = LDS ? (GATE_UP ? (GS == 1 ? 1 : 2) : (GS == 4 ? 4 : 2)) : 1;
  const int e = __builtin_amdgcn_readfirstlane(moe_expert(a.ids, a.tokens, a.top_k, a.experts, blockIdx.y, list));
  if (e < 0) return;
  const char* blob = a.packed + e * a.stride;
  L4Stream st = a.st;
  st.codes = reinterpret_cast<const u32x4_t*>(blob + a.code_off);
  st.params = reinterpret_cast<const float2*>(blob + a.param_off);
  const int lane = threadIdx.x & 63, tid = threadIdx.x;
  const int upw = kL4Waves >> st.kslog;
  const int64_t first = (int64_t)blockIdx.x * upw, step = (int64_t)gridDim.x * upw;
  // grid z: passes of an expert of many tokens, and slices of K whose rows fit
  const int slice = GATE_UP ? 0 : (int)(blockIdx.z % a.slices), z0 = GATE_UP ? blockIdx.z : blockIdx.z / a.slices;
  const int zn = GATE_UP ? gridDim.z : gridDim.z / a.slices;
  if (!GATE_UP) {
    st.kcount = (int)((st.kc + a.slices - 1) / a.slices);
    st.kfirst = slice * st.kcount;
    st.kcount = std::min(st.kcount, (int)st.kc - st.kfirst);
  }
  const int per = GATE_UP ? (int)st.kc : (int)((st.kc + a.slices - 1) / a.slices);   // chunks of a row in LDS
  const int xrow = per * kL4Chunk + kL4Pad;
  uint16_t* xsh = reinterpret_cast<uint16_t*>(lds);
  float* red = reinterpret_cast<float*>(lds + (LDS ? (size_t)a.pass * NP * xrow * 2 : 0));
  bool again = false;
  for (int p0 = z0 * a.pass; p0 < list.count; p0 += zn * a.pass) {
    const int np = std::min(a.pass, list.count - p0);
    auto fill = [&] {
      if (!LDS) return;
      if (again) __syncthreads();   // the pass before has been read
      const int pieces = st.kcount * (kL4Chunk / 8);
      for (int i = tid; i < np * NP * pieces; i += kL4Threads) {
        const int q = i / pieces, k = 8 * (i % pieces);   // row q = token q / NP, plane q % NP
        *reinterpret_cast<uint4*>(xsh + q * xrow + k) =
            *reinterpret_cast<const uint4*>(a.A + ((int64_t)list.pair[p0 + q / NP] * NP + q % NP) * a.k128 + st.kfirst * kL4Chunk + k);
      }
      __syncthreads();
    };
    auto end = [&](int64_t unit, const f32x4_t (&y)[RT]) {
      l4_finish<RT>(red, a.quads, np, st.kslog, unit, y, [&](int64_t u, int q, int row, const float (&z)[RT]) {
        const int64_t r = u * kL4Rows + row, pair = list.pair[p0 + q];
        if (u >= st.units || r >= a.rows) return;
        if (GATE_UP) {
          moe_hidden(a, pair, r, z);
        } else {
          a.out[((int64_t)slice * a.tokens * a.top_k + pair) * a.rows + r] = z[0];
        }
      });
    };
    const int q = std::min(lane & 15, np - 1);   // rows past the last: computed, not stored
    if (LDS) {
      const L4LdsA af{xsh + q * NP * xrow + 8 * (lane >> 4), xrow, GATE_UP ? 0 : st.kfirst};
      l4_units<GS, RT, NP, B, NP == 3>(st, first, step, af, fill, end);
    } else {
      const L4GlobalA af{a.A + (int64_t)list.pair[p0 + q] * NP * a.k128 + 8 * (lane >> 4), a.k128};
      l4_units<GS, RT, NP, B, NP == 3>(st, first, step, af, fill, end);
    }
    again = true;
  }
}

template <int GS, bool LDS>
__global__ __launch_bounds__(kL4Threads) void moe_gate_up_kernel(MoeExpertArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ MoeList list;
  moe_expert_units<GS, true, 1, LDS>(a, list, lds);
}

template <int GS, int NP, bool LDS>
__global__ __launch_bounds__(kL4Threads) void moe_down_kernel(MoeExpertArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ MoeList list;
  moe_expert_units<GS, false, NP, LDS>(a, list, lds);
}

// ---------------------------------------------------------------- a token or a few: two launches
// While the router's work is small (tokens x experts x hidden), every
// gate/up workgroup does all of it for itself and gathers its expert's tokens,
// and the down kernel adds all experts of a row tile: two launches instead of
// four, with no pass of ids, X' or pair results through memory between them.
constexpr int kSmallTokens = 16;
constexpr int kSmallPairs = 64;
constexpr int kSmallLogits = 64;

struct MoeSmallArgs {
  MoeExpertArgs x;        // gate/up: A unused; down: the combine's part below
  const uint16_t* X;
  int64_t ldx, order_off;
  int hidden, renorm, vec, xvec, r_dt;
  const void* R;
  int32_t *ids, *ids_out;
  float *wts, *wts_out;
};

template <int GS>
__global__ __launch_bounds__(kL4Threads) void moe_small_gate_up_kernel(MoeSmallArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ MoeList list;
  __shared__ double logit[kSmallLogits];
  __shared__ double part_sum[16];
  __shared__ int rank[kSmallLogits];
  __shared__ int32_t ids[kSmallPairs];
  const MoeExpertArgs& g = a.x;
  const int T = g.tokens, E = g.experts, K = g.top_k, h = a.hidden, hrow = ((h + 7) & ~7) + kMoeTail;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int xrow = (int)g.k128 + kL4Pad;
  uint16_t* xsh = reinterpret_cast<uint16_t*>(lds);                    // X' [pass][xrow]
  uint16_t* raw = xsh + (size_t)g.pass * xrow;                         // X [T][hrow]
  float* red = reinterpret_cast<float*>(raw);                          // after the gather
  for (int t = 0; t < T; ++t)
    l4_row_to_lds(a.X + t * a.ldx, h, a.xvec, reinterpret_cast<uint8_t*>(raw + t * hrow), tid, kL4Threads);
  if (tid < T * kMoeTail) moe_tail(raw + (tid / kMoeTail) * hrow, h, tid % kMoeTail);
  const int pairs = T * E;
  for (int i = tid; i < pairs; i += kL4Threads) rank[i] = 0;
  __syncthreads();
  int parts = 1;
  while (parts < 16 && pairs * parts * 2 <= 16) parts *= 2;
  for (int i = wave / parts; i < pairs; i += 16 / parts) {
    const int t = i / E, e = i - t * E, part = wave % parts;
    const double s = moe_logit(raw + t * hrow, a.R, a.r_dt, a.vec, e, h, part, parts);
    if (lane == 0) {
      if (parts == 1)
        logit[i] = s;
      else
        part_sum[wave] = s;   // pairs * parts <= 16: each wave has one
    }
  }
  __syncthreads();
  if (parts > 1) {
    if (tid < pairs) {
      double s = part_sum[tid * parts];
      for (int p = 1; p < parts; ++p) s += part_sum[tid * parts + p];
      logit[tid] = s;
    }
    __syncthreads();
  }
  int slog = 0;
  while ((pairs << (slog + 1)) <= kL4Threads && (1 << slog) < E) ++slog;
  for (int i = tid; i < pairs << slog; i += kL4Threads) {
    const int at = i >> slog, t = at / E, e = at - t * E;
    const double mine = logit[at];
    int before = 0;
    for (int o = i & ((1 << slog) - 1); o < E; o += 1 << slog)
      before += o != e && moe_before(logit[t * E + o], o, mine, e);
    if (before) atomicAdd(&rank[at], before);
  }
  __syncthreads();
  if (tid < pairs && rank[tid] < K) ids[(tid / E) * K + rank[tid]] = tid % E;
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave < T) {   // one workgroup leaves them for the down kernel
    const double* lg = logit + wave * E;
    const double top = lg[ids[wave * K]];
    const double mine = lane < K ? exp(lg[ids[wave * K + lane]] - top) : 0.0;
    double sum = mine;
    if (!a.renorm) {
      sum = 0.0;
      for (int e = lane; e < E; e += 64) sum += exp(lg[e] - top);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane < K) {
      const int at = wave * K + lane;
      const float wt = (float)(mine / sum);
      a.ids[at] = ids[at];
      a.wts[at] = wt;
      if (a.ids_out) a.ids_out[at] = ids[at];
      if (a.wts_out) a.wts_out[at] = wt;
    }
  }
  const int e = __builtin_amdgcn_readfirstlane(moe_expert(ids, T, K, E, blockIdx.y, list));
  if (e < 0) return;
  const char* blob = g.packed + e * g.stride;
  L4Stream st = g.st;
  st.codes = reinterpret_cast<const u32x4_t*>(blob + g.code_off);
  st.params = reinterpret_cast<const float2*>(blob + g.param_off);
  const int np = list.count;   // at most the pass: one pass
  auto fill = [&] {
    const int32_t* order = reinterpret_cast<const int32_t*>(blob + a.order_off);
    for (int p = 4 * tid; p < (int)g.k128; p += 4 * kL4Threads) {
      const int4 o = *reinterpret_cast<const int4*>(order + p);
      for (int q = 0; q < np; ++q) {
        const uint16_t* x = raw + (list.pair[q] / K) * hrow;
        const uint32_t v0 = x[std::max(o.x, 0)], v1 = x[std::max(o.y, 0)], v2 = x[std::max(o.z, 0)], v3 = x[std::max(o.w, 0)];
        uint2 v;
        v.x = (o.x >= 0 ? v0 : 0u) | (o.y >= 0 ? v1 : 0u) << 16;
        v.y = (o.z >= 0 ? v2 : 0u) | (o.w >= 0 ? v3 : 0u) << 16;
        *reinterpret_cast<uint2*>(xsh + q * xrow + p) = v;
      }
    }
    __syncthreads();
  };
  auto end = [&](int64_t unit, const f32x4_t (&y)[2]) {
    l4_finish<2>(red, g.quads, np, st.kslog, unit, y, [&](int64_t u, int q, int row, const float (&z)[2]) {
      if (u < st.units) moe_hidden(g, list.pair[q], u * kL4Rows + row, z);
    });
  };
  const int upw = kL4Waves >> st.kslog, q = std::min(lane & 15, np - 1);
  const L4LdsA af{xsh + q * xrow + 8 * (lane >> 4), 0};
  l4_units<GS, 2, 1, (GS == 1 ? 1 : 2), false>(st, (int64_t)blockIdx.x * upw, (int64_t)gridDim.x * upw, af, fill, end);
}

struct MoeSmallDownArgs {
  MoeExpertArgs x;
  const float* wts;
  const void* res;
  int res_dt, y_dt;
  int64_t ldr, ldy;
  void* Y;
};

// Y = Σ over the active experts, in ascending order, of w·(down product) +
// residual.  A workgroup takes row tiles; its 16 waves share the chunks of all
// active experts, laid end to end, in equal runs; where a run passes from one
// expert to the next the sums so far are weighted and put by.
template <int GS, int NP>
__global__ __launch_bounds__(kL4Threads) void moe_small_down_kernel(MoeSmallDownArgs a) {
  constexpr int NG = 4 / GS, B = GS == 4 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint32_t used[kMoeMaxExperts / 32];
  __shared__ int expert[kSmallPairs];
  __shared__ int active;
  __shared__ __attribute__((aligned(16))) float weight[kSmallPairs][16];    // [slot][token]
  __shared__ __attribute__((aligned(16))) int pair_of[kSmallPairs][16];     // the token's pair, -1: it did not choose the expert
  const MoeExpertArgs& g = a.x;
  const int T = g.tokens, K = g.top_k;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int xrow = (int)g.k128 + kL4Pad;
  uint16_t* xsh = reinterpret_cast<uint16_t*>(lds);                                    // [pairs][NP][xrow]
  float* red = reinterpret_cast<float*>(xsh + (size_t)T * K * NP * xrow);
  if (tid < kMoeMaxExperts / 32) used[tid] = 0;
  for (int i = tid; i < kSmallPairs * 16; i += kL4Threads) {
    (&weight[0][0])[i] = 0.f;
    (&pair_of[0][0])[i] = -1;
  }
  __syncthreads();
  const int my = tid < T * K ? g.ids[tid] : 0;
  if (tid < T * K) atomicOr(&used[my >> 5], 1u << (my & 31));
  const int pieces = (int)(g.k128 / 8);
  for (int i = tid; i < T * K * NP * pieces; i += kL4Threads)
    *reinterpret_cast<uint4*>(xsh + (i / pieces) * xrow + 8 * (i % pieces)) =
        *reinterpret_cast<const uint4*>(g.A + (int64_t)(i / pieces) * g.k128 + 8 * (i % pieces));
  __syncthreads();
  if (tid < T * K) {
    int slot = __popc(used[my >> 5] & ((1u << (my & 31)) - 1u));
    for (int w = 0; w < (my >> 5); ++w) slot += __popc(used[w]);
    expert[slot] = my;
    weight[slot][tid / K] = a.wts[tid];
    pair_of[slot][tid / K] = tid;
  }
  if (tid == 0) {
    int n = 0;
    for (int w = 0; w < (g.experts + 31) / 32; ++w) n += __popc(used[w]);
    active = n;
  }
  __syncthreads();
  const int kc = (int)g.st.kc, total = active * kc, per = (total + 15) / 16;
  const int i0 = std::min(total, wave * per), i1 = std::min(total, i0 + per);
  const L4Consts k;
  struct Batch {
    u32x4_t cw[B];
    float2 p[B][NG];
  };
  auto load = [&](int64_t unit, int i, int n, Batch& b) {   // n >= 1 chunks from item i of one slot
    const int slot = i / kc, c = i - slot * kc;
    const char* blob = g.packed + (int64_t)__builtin_amdgcn_readfirstlane(expert[slot]) * g.stride;
    const u32x4_t* cp = reinterpret_cast<const u32x4_t*>(blob + g.code_off) + unit * kc * 64 + lane;
    const float2* pp = reinterpret_cast<const float2*>(blob + g.param_off) + unit * g.st.Gp * kL4Rows + (lane & 15);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int cc = c + std::min(j, n - 1);
      b.cw[j] = cp[(int64_t)cc * 64];
#pragma unroll
      for (int q = 0; q < NG; ++q) b.p[j][q] = pp[(int64_t)(cc * NG + q) * g.st.pmul];
    }
  };
  // chunks of a batch from item i: up to B, within the slot and the run
  auto count = [&](int i) { return std::min(std::min(B, i1 - i), kc - i % kc); };
  f32x4_t y[1];
  const int64_t first = blockIdx.x, step = gridDim.x;
  Batch cur, nxt;
  if (i0 < i1) load(std::min<int64_t>(first, g.st.units - 1), i0, count(i0), cur);
  for (int r = 0; r < g.st.rounds; ++r) {
    const int64_t unit = first + r * step;
    y[0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    f32x4_t z = {0.f, 0.f, 0.f, 0.f};
    for (int i = i0; i < i1;) {
      const int n = count(i), slot = i / kc, c = i - slot * kc;
      const bool more = i + n < i1;
      const int ni = more ? i + n : i0;
      load(std::min<int64_t>(more ? unit : unit + step, g.st.units - 1), ni, count(ni), nxt);
      const uint16_t* row = xsh + (size_t)std::max(pair_of[slot][lane & 15], 0) * NP * xrow + 8 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (j >= n) break;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          f32x4_t sx = {0.f, 0.f, 0.f, 0.f}, acc = {0.f, 0.f, 0.f, 0.f};
          const float s = cur.p[j][q].x, y0 = cur.p[j][q].y;
#pragma unroll
          for (int st = q * GS; st < q * GS + GS; ++st) {
            const bf16x8_t w = NP == 3 ? k.unpack_centred(cur.cw[j][st], l4_centre_off(y0)) : k.unpack(cur.cw[j][st]);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              const bf16x8_t av = __builtin_bit_cast(
                  bf16x8_t, *reinterpret_cast<const uint4*>(row + p * xrow + (c + j) * kL4Chunk + 32 * st));
              sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, k.ones(), sx, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, w, acc, 0, 0, 0);
            }
          }
          const float zp = NP == 3 ? y0 - 128.f - l4_centre(y0) : l4_zero(y0);
#pragma unroll
          for (int v = 0; v < 4; ++v) z[v] = fmaf(s, fmaf(-zp, sx[v], acc[v]), z[v]);
        }
      }
      i += n;
      if (i >= i1 || i % kc == 0) {   // the run leaves this expert
        const f32x4_t wt = *reinterpret_cast<const f32x4_t*>(&weight[slot][4 * (lane >> 4)]);
        const int4 po = *reinterpret_cast<const int4*>(&pair_of[slot][4 * (lane >> 4)]);
        const int chose[4] = {po.x, po.y, po.z, po.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) y[0][v] = chose[v] >= 0 ? fmaf(wt[v], z[v], y[0][v]) : y[0][v];
        z = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      cur = nxt;
    }
    l4_finish<1>(red, g.quads, T, 4, unit + wave / 16, y, [&](int64_t u, int t, int row, const float (&v)[1]) {
      const int64_t c = u * kL4Rows + row;
      if (u >= g.st.units || c >= g.rows) return;
      float o = v[0];
      if (a.res) o += l4_load(a.res, a.res_dt, t * a.ldr + c);
      l4_store(a.Y, a.y_dt, t * a.ldy + c, o);
    });
  }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ pairs, const float* __restrict__ wts,
                                                          int top_k, int slices, int64_t hidden, const void* res, int res_dt,
                                                          int64_t ldr, void* Y, int y_dt, int64_t ldy) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (r >= hidden) return;
  float v = 0.f;
  const int64_t slice = (int64_t)gridDim.y * top_k * hidden;
  for (int j = 0; j < top_k; ++j) {
    const float* p = pairs + (t * top_k + j) * hidden + r;
    float d = p[0];
    for (int s = 1; s < slices; ++s) d += p[s * slice];
    v = fmaf(wts[t * top_k + j], d, v);
  }
  if (res) v += l4_load(res, res_dt, t * ldr + r);
  l4_store(Y, y_dt, t * ldy + r, v);
}

constexpr int64_t kMoeLogitsElsewhere = 1 << 16;   // logit products from which they get a launch of their own
// Logit products that every workgroup repeats: up to here it costs less than
// the launches it saves (64 experts of 2048, 1 token: 34.5 us by four launches,
// 27.2 by two; 16 of 2048, 4 tokens: 32.5 and 34.1).
constexpr int64_t kSmallRouter = 65536, kSmallRouter2 = 131072;   // the latter for one or two tokens
constexpr size_t kMoeMaxLds = 150 * 1024;

// The fewest tokens that are worth a pass: twice an expert's mean, six at most
// (8 experts of 4096 x 11008, top 2, passes of 3 against slices of K with full
// ones: 4 tokens 137 us and 181 from memory, 8 tokens 169 and 159, 16 tokens 194
// and 175).
int moe_least(int64_t tokens, int64_t top_k, int64_t experts) {
  return (int)std::min<int64_t>(6, ceil_div(2 * tokens * top_k, experts));
}
// Slices of the down product's K: one where moe_least tokens' hidden activation
// fits in LDS, else as many as make a full pass fit; the combine kernel adds
// their results in slice order.  Up to 256 MB of those, beyond that one slice,
// read from memory (the same experts, 32 tokens: 245 us from memory, 180 in
// slices; 64 tokens 448 and 303).
int moe_slices(const gptq_moe_config& c, int64_t tokens, int planes) {
  const int64_t kc = ceil_div(c.inter, kL4Chunk), pass = std::min<int64_t>(kMoePass, tokens);
  auto bytes = [&](int64_t rows, int64_t chunks) {   // and the waves' sums
    return (size_t)rows * planes * (size_t)(chunks * kL4Chunk + kL4Pad) * 2 + (size_t)kL4Waves * ceil_div(rows, 4) * 256;
  };
  if (bytes(std::min<int64_t>(pass, moe_least(tokens, c.top_k, c.experts)), kc) <= kMoeMaxLds) return 1;
  int64_t s = 2;
  while (bytes(pass, ceil_div(kc, s)) > kMoeMaxLds) ++s;
  s = ceil_div(kc, ceil_div(kc, s));   // none is empty
  return (size_t)(s * tokens * c.top_k) * (size_t)c.hidden * sizeof(float) <= (size_t)256 << 20 ? (int)s : 1;
}

// fills the launch-dependent fields; returns the dynamic LDS bytes, 0 < lds
// with *in_lds when the rows of a pass fit
size_t moe_plan(MoeExpertArgs& a, int tokens, int planes, int rt, int64_t wgs, bool* in_lds) {
  const int64_t per = ceil_div(a.st.kc, (int64_t)a.slices);   // chunks
  const L4Split sp = l4_split(a.st.units, wgs, per, rt);
  a.st.kslog = sp.kslog;
  a.st.rounds = sp.rounds;
  // as many tokens a pass as LDS holds, down to moe_least; fewer would stream the
  // codes too often, and fragments are read from memory instead (8 experts of
  // 4096 x 2048, 64 tokens: 114 us from memory, 80 in passes of 14)
  const int least = moe_least(tokens, a.top_k, a.experts);
  for (a.pass = std::min(kMoePass, tokens);; --a.pass) {
    a.quads = (int)ceil_div(a.pass, 4);
    const size_t red = sp.kslog ? (size_t)kL4Waves * rt * a.quads * 64 * sizeof(float) : 0;
    const size_t rows = (size_t)a.pass * planes * (size_t)(per * kL4Chunk + kL4Pad) * 2;
    *in_lds = rows + red <= kMoeMaxLds;
    if (*in_lds) return rows + red;
    if (a.pass <= least) break;
  }
  a.pass = std::min(kMoePass, tokens);
  a.quads = (int)ceil_div(a.pass, 4);
  return sp.kslog ? (size_t)kL4Waves * rt * a.quads * 64 * sizeof(float) : 0;
}

// Whether a call of `tokens` tokens takes the two-launch form.
bool moe_is_small(const gptq_moe_config& c, int64_t tokens, int planes, const MoeLayout& L) {
  const size_t x = (size_t)tokens * (size_t)(L.gu.n128 + kL4Pad) * 2 + (size_t)tokens * (size_t)round_up(c.hidden, 8) * 2;
  const size_t mid = (size_t)(tokens * c.top_k * planes) * (size_t)(L.f128 + kL4Pad) * 2;
  return tokens <= kSmallTokens && tokens * c.top_k <= kSmallPairs && tokens * c.experts <= kSmallLogits &&
         tokens * c.experts * c.hidden <= (tokens <= 2 ? kSmallRouter2 : kSmallRouter) && x <= 64 * 1024 && mid <= 100 * 1024;
}

// The form of a call of `tk` tokens: the two launches, or the split over the GPU
// and the passes of gate/up and down (launch-dependent fields of g and d).
struct MoeForm {
  bool small, logits, gu_in_lds, down_in_lds;   // logits: in a launch of their own
  int64_t slots, passes;
  size_t gu_lds, down_lds;
  dim3 gu_grid, down_grid;
};
MoeForm moe_form(const gptq_moe_config& c, int tk, const MoeLayout& L, MoeExpertArgs& g, MoeExpertArgs& d) {
  MoeForm f{};
  f.small = moe_is_small(c, tk, d.planes, L);
  f.logits = !f.small && (int64_t)tk * c.experts * c.hidden > kMoeLogitsElsewhere && c.experts > 16;
  // the workgroups of the GPU dealt over the experts that can be active; where an
  // expert has more tokens than a pass on average, passes side by side
  f.slots = std::min<int64_t>(c.experts, (int64_t)tk * c.top_k);
  f.passes = ceil_div((int64_t)tk * c.top_k, (int64_t)c.experts * kMoePass);
  const int64_t share = std::max<int64_t>(1, 256 / (f.slots * f.passes));
  g.tokens = d.tokens = tk;
  d.slices = moe_slices(c, tk, d.planes);
  const int64_t gw = std::min<int64_t>(share, g.st.units);
  f.gu_lds = moe_plan(g, tk, 1, 2, gw, &f.gu_in_lds);
  f.gu_grid = dim3((unsigned)std::min<int64_t>(gw, ceil_div(g.st.units, kL4Waves >> g.st.kslog)), (unsigned)f.slots,
                   (unsigned)f.passes);
  const int64_t dw = std::min<int64_t>(std::max<int64_t>(1, share / d.slices), d.st.units);
  f.down_lds = moe_plan(d, tk, d.planes, 1, dw, &f.down_in_lds);
  f.down_grid = dim3((unsigned)std::min<int64_t>(dw, ceil_div(d.st.units, kL4Waves >> d.st.kslog)), (unsigned)f.slots,
                     (unsigned)(f.passes * d.slices));
  return f;
}

int moe_planes(int y_dtype) { return y_dtype == GPTQ_FP32 ? 3 : 2; }

// Sizes of a product; one group per row folds as groups of 128 (pmul = 0 repeats
// its parameters)
void moe_sizes(MoeExpertArgs& a, const gptq_moe_config& c, const W4Layout& l, int64_t units, int planes) {
  a.st = L4Stream{nullptr, nullptr, l.kc, l.Gp, units, l.g >= l.n128 ? 0 : kL4Rows, 0, 1, 0, (int)l.kc};
  a.slices = 1;
  a.k128 = l.n128;
  a.top_k = c.top_k;
  a.experts = c.experts;
  a.planes = planes;
}

template <class A, class K>
gptq_status moe_launch(K kernel, dim3 grid, size_t lds, const A& a, hipStream_t stream) {
  if (lds > 32768)
    GPTQ_HIP_CHECK(hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  hipLaunchKernelGGL(kernel, grid, dim3(kL4Threads), lds, stream, a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

template <int GS>
gptq_status launch_gate_up(dim3 grid, size_t lds, bool in_lds, const MoeExpertArgs& a, hipStream_t stream) {
  return in_lds ? moe_launch(moe_gate_up_kernel<GS, true>, grid, lds, a, stream)
                : moe_launch(moe_gate_up_kernel<GS, false>, grid, lds, a, stream);
}

template <int GS>
gptq_status launch_down(dim3 grid, size_t lds, bool in_lds, const MoeExpertArgs& a, hipStream_t stream) {
  if (a.planes == 3)
    return in_lds ? moe_launch(moe_down_kernel<GS, 3, true>, grid, lds, a, stream)
                  : moe_launch(moe_down_kernel<GS, 3, false>, grid, lds, a, stream);
  return in_lds ? moe_launch(moe_down_kernel<GS, 2, true>, grid, lds, a, stream)
                : moe_launch(moe_down_kernel<GS, 2, false>, grid, lds, a, stream);
}

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
  const size_t h128 = (size_t)(ceil_div(c.hidden, kL4Chunk) * kL4Chunk);
  w.xp_off = w.wts_off + align256(pairs * sizeof(float));
  w.mid_off = w.xp_off + align256(pairs * h128 * sizeof(uint16_t));
  w.out_off = w.mid_off + align256(pairs * kMoeMaxPlanes * f128 * sizeof(uint16_t));
  int slices = 1;   // of either result type, of a full block and of the last
  for (int64_t tk : {w.block, tokens % w.block})
    if (tk > 0) slices = std::max({slices, moe_slices(c, tk, 2), moe_slices(c, tk, 3)});
  w.logits_off = w.out_off + align256(pairs * (size_t)slices * (size_t)c.hidden * sizeof(float));
  w.total = w.logits_off + align256((size_t)w.block * (size_t)c.experts * sizeof(double));
  return w;
}

MoePath moe_path(const gptq_moe_config& c, int64_t tokens, int y_dtype) {
  const MoeLayout L = plan_moe(c);
  MoeExpertArgs g{}, d{};
  moe_sizes(g, c, L.gu, L.gu.mt / 2, moe_planes(y_dtype));
  moe_sizes(d, c, L.down, L.down.mt, moe_planes(y_dtype));
  const MoeForm f = moe_form(c, (int)std::min<int64_t>(tokens, kMoeTokens), L, g, d);
  return {f.small, f.logits, f.gu_in_lds, g.pass, f.down_in_lds, d.pass, d.slices};
}

// The slices of K change with the tokens (none where a few fit in LDS, none
// again where their results pass 256 MB), so the largest of all counts up to
// `tokens`: 1 .. 64, and 64 with every rest.
size_t moe_workspace(const gptq_moe_config& c, int64_t tokens) {
  size_t most = plan_moe_work(c, tokens).total;
  for (int64_t t = 1; t < std::min<int64_t>(tokens, 2 * kMoeTokens); ++t) most = std::max(most, plan_moe_work(c, t).total);
  return most;
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
  double* logits = reinterpret_cast<double*>(wb + w.logits_off);
  const size_t ysz = c.y_dtype == GPTQ_FP32 ? 4 : 2, rsz = c.res_dtype == GPTQ_FP32 ? 4 : 2;
  const char* packed = static_cast<const char*>(c.packed);
  const int h = (int)cfg.hidden;

  uint16_t* Xp = reinterpret_cast<uint16_t*>(wb + w.xp_off);
  auto weight = [&](MoeExpertArgs& a, const W4Layout& l, const char* base, int64_t units) {
    a.packed = base;
    a.stride = (int64_t)L.stride;
    a.param_off = (int64_t)l.param_off;
    a.code_off = (int64_t)l.code_off;
    moe_sizes(a, cfg, l, units, moe_planes(c.y_dtype));
    a.ids = ids;
    a.act = cfg.activation;
    a.mid = mid;
    a.out = out;
  };
  auto steps = [&](const W4Layout& l) { return l.g >= l.n128 ? 4 : (int)(l.g / 32); };
  MoeExpertArgs g, d;
  weight(g, L.gu, packed, L.gu.mt / 2);
  weight(d, L.down, packed + L.down_off, L.down.mt);
  g.A = Xp;
  g.rows = L.f128;
  d.A = mid;
  d.rows = cfg.hidden;

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
    r.xvec = (reinterpret_cast<uintptr_t>(c.X) & 15) == 0 && c.ldx % 8 == 0;
    r.parts = cfg.experts > 8 ? 1 : cfg.experts > 4 ? 2 : cfg.experts > 2 ? 4 : 8;
    r.ids = ids;
    r.wts = wts;
    r.ids_out = c.topk_ids ? c.topk_ids + t0 * cfg.top_k : nullptr;
    r.wts_out = c.topk_weights ? c.topk_weights + t0 * cfg.top_k : nullptr;
    r.packed = packed;
    r.stride = (int64_t)L.stride;
    r.order_off = (int64_t)L.gu.order_off;
    r.n128 = L.gu.n128;
    r.Xp = Xp;
    const MoeForm f = moe_form(cfg, tk, L, g, d);
    r.logits = f.logits ? logits : nullptr;
    if (r.logits) r.parts = 1;
    const void* res = c.res ? (const void*)(static_cast<const char*>(c.res) + (size_t)(t0 * c.ldr) * rsz) : nullptr;
    void* Y = static_cast<char*>(c.Y) + (size_t)(t0 * c.ldy) * ysz;
    if (f.small) {
      MoeSmallArgs sa;
      sa.x = g;
      sa.X = r.X;
      sa.ldx = c.ldx;
      sa.order_off = r.order_off;
      sa.hidden = h;
      sa.renorm = cfg.renormalize;
      sa.vec = r.vec;
      sa.xvec = r.xvec;
      sa.r_dt = c.router_dtype;
      sa.R = c.router;
      sa.ids = ids;
      sa.wts = wts;
      sa.ids_out = r.ids_out;
      sa.wts_out = r.wts_out;
      const size_t rows = (size_t)g.pass * (size_t)(g.k128 + kL4Pad) * 2;
      const size_t raw = (size_t)tk * (size_t)(round_up(h, 8) + kMoeTail) * 2, red = (size_t)kL4Waves * 2 * g.quads * 64 * sizeof(float);
      size_t lds = rows + std::max(raw, red);
      switch (steps(L.gu)) {
        case 1: GPTQ_TRY(moe_launch(moe_small_gate_up_kernel<1>, f.gu_grid, lds, sa, stream)); break;
        case 2: GPTQ_TRY(moe_launch(moe_small_gate_up_kernel<2>, f.gu_grid, lds, sa, stream)); break;
        default: GPTQ_TRY(moe_launch(moe_small_gate_up_kernel<4>, f.gu_grid, lds, sa, stream)); break;
      }
      MoeSmallDownArgs sd;
      sd.x = d;
      sd.wts = wts;
      sd.res = res;
      sd.res_dt = c.res_dtype;
      sd.y_dt = c.y_dtype;
      sd.ldr = c.ldr;
      sd.ldy = c.ldy;
      sd.Y = Y;
      const int64_t wgs = std::min<int64_t>(d.st.units, 256);
      sd.x.quads = g.quads;
      sd.x.st.rounds = (int)ceil_div(d.st.units, wgs);
      lds = (size_t)(tk * cfg.top_k * d.planes) * (size_t)(d.k128 + kL4Pad) * 2 +
            (size_t)kL4Waves * sd.x.quads * 64 * sizeof(float);
      const dim3 sgrid((unsigned)wgs);
#define MOE_SMALL_DOWN(GS)                                                                                       \
  GPTQ_TRY(d.planes == 3 ? moe_launch(moe_small_down_kernel<GS, 3>, sgrid, lds, sd, stream)                  \
                         : moe_launch(moe_small_down_kernel<GS, 2>, sgrid, lds, sd, stream))
      switch (steps(L.down)) {
        case 1: MOE_SMALL_DOWN(1); break;
        case 2: MOE_SMALL_DOWN(2); break;
        default: MOE_SMALL_DOWN(4); break;
      }
#undef MOE_SMALL_DOWN
      continue;
    }
    const size_t xlds = (size_t)(round_up(h, 8) + kMoeTail) * 2;   // a token's row
    if (r.logits)
      GPTQ_TRY(moe_launch(moe_logits_kernel, dim3((unsigned)ceil_div(cfg.experts, 16), (unsigned)tk), xlds, r, stream));
    GPTQ_TRY(moe_launch(moe_router_kernel, dim3((unsigned)tk),
                        (size_t)round_up((int64_t)r.parts * cfg.experts, 2) * sizeof(double) +
                            (size_t)round_up(cfg.experts, 4) * sizeof(int) + xlds,
                        r, stream));
    switch (steps(L.gu)) {
      case 1: GPTQ_TRY(launch_gate_up<1>(f.gu_grid, f.gu_lds, f.gu_in_lds, g, stream)); break;
      case 2: GPTQ_TRY(launch_gate_up<2>(f.gu_grid, f.gu_lds, f.gu_in_lds, g, stream)); break;
      default: GPTQ_TRY(launch_gate_up<4>(f.gu_grid, f.gu_lds, f.gu_in_lds, g, stream)); break;
    }
    switch (steps(L.down)) {
      case 1: GPTQ_TRY(launch_down<1>(f.down_grid, f.down_lds, f.down_in_lds, d, stream)); break;
      case 2: GPTQ_TRY(launch_down<2>(f.down_grid, f.down_lds, f.down_in_lds, d, stream)); break;
      default: GPTQ_TRY(launch_down<4>(f.down_grid, f.down_lds, f.down_in_lds, d, stream)); break;
    }
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)ceil_div(cfg.hidden, 256), (unsigned)tk), dim3(256), 0, stream,
                       (const float*)out, (const float*)wts, (int)cfg.top_k, d.slices, cfg.hidden, res, c.res_dtype, c.ldr, Y,
                       c.y_dtype, c.ldy);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

}  // namespace gptq
