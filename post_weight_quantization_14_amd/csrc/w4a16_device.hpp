// Device pieces shared by the layers built on packed 2/3/4-bit weights
// (w4a16_linear.hip, w4a16_moe.hip): operand unpacking, the K loop of a
// 16-row tile, activations and typed loads and stores.
#pragma once

#include <algorithm>

#include "gptq_internal.hpp"

namespace gptq {

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kL4Rows = 16;     // weight rows per packed tile (MFMA N)
constexpr int kL4Chunk = 128;   // positions per packed chunk (4 MFMA k-steps of 32)

// ---------------------------------------------------------------- operands
// A 4-bit code q becomes the bf16 (16 + q)·2^-12 with one shift and one AND-OR:
// bf16 numbers in [16, 32)·2^-12 are spaced 2^-15, so q sits in mantissa bits
// 3..6 of 0x3B80.  Then
//   Σ_k x_k·(q_k - z) = Σ_k x_k·(16 + q_k) - (16 + z)·Σ_k x_k,
// with exact bf16 x bf16 products on the left.  16 is the smallest offset
// whose binade holds every 4-bit code: the two sums are then at most ~5x the
// difference for codes around the middle, and fp32 sums lose 2-3 bits to
// the subtraction (an offset of 128 loses 5).
//
// Both sums are held times 2^-12, and a result is multiplied by 2^12 when it is
// whole: 128 positions·31 < 2^12, so no sum of a group overflows for any finite
// x, where x·(16 + q) alone would from 1.1e37 on, with a result of Inf - Inf.
// The factor is exact: other results keep their bits (of groups whose x are all
// below 2^-102 some are lost to the smallest numbers of fp32 and of bf16 planes).
constexpr float kL4Down = 0x1p-12f, kL4Up = 0x1p12f;

struct L4Consts {
  uint32_t m, c, one;
  // hidden from constant folding: VOP3 takes no literals, so as visible
  // constants each AND-OR would compile to two instructions
  __device__ __forceinline__ L4Consts() : m(0x00780078u), c(0x3B803B80u), one(0x39803980u) {
    asm volatile("" : "+v"(m), "+v"(c), "+v"(one));
  }
  __device__ __forceinline__ bf16x8_t unpack(uint32_t w) const {
    u32x4_t r;
    r[0] = ((w << 3) & m) | c;
    r[1] = ((w >> 1) & m) | c;
    r[2] = ((w >> 5) & m) | c;
    r[3] = ((w >> 9) & m) | c;
    return __builtin_bit_cast(bf16x8_t, r);
  }
  // (q - zc)·2^-12 for an integer 0 <= zc <= 15 (off = (16 + zc)·2^-12): exact in
  // bf16, so the upper halves of the fp32 differences are the operand itself
  __device__ __forceinline__ bf16x8_t unpack_centred(uint32_t w, float off) const {
    const u32x4_t r = __builtin_bit_cast(u32x4_t, unpack(w));
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(r[i] << 16) - off, hi = __uint_as_float(r[i] & 0xffff0000u) - off;
      o[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
    }
    return __builtin_bit_cast(bf16x8_t, o);
  }
  // each 2^-12
  __device__ __forceinline__ bf16x8_t ones() const {
    return __builtin_bit_cast(bf16x8_t, u32x4_t{one, one, one, one});
  }
};

// packed group parameters hold (s, 128 + z)
__device__ __forceinline__ float l4_zero(float y) { return y - 112.f; }
__device__ __forceinline__ float l4_centre(float y) { return fminf(fmaxf(y - 128.f, 0.f), 15.f); }
__device__ __forceinline__ float l4_centre_off(float y) { return fmaf(l4_centre(y), kL4Down, 16.f * kL4Down); }

// ---------------------------------------------------------------- few tokens
// The kernels of up to 16 tokens are bound by the code stream from HBM.  A
// workgroup of 16 waves takes `rounds` rounds of units (a unit is RT row tiles
// of 16 weight rows), 16 / ks units a round with ks waves splitting the K
// range of each, and every wave keeps B·RT KB of codes in flight through all
// of its rounds: the next batch, of the same unit or the next one, is loaded
// before the current one is multiplied.
constexpr int kL4Waves = 16;
constexpr int kL4Threads = 64 * kL4Waves;

struct L4Stream {
  const u32x4_t* codes;    // [units·RT][kc][64]
  const float2* params;    // [units·RT][Gp][16]: (s, 128 + z)
  int64_t kc, Gp, units;
  int pmul;                // distance of groups in params: 16, or 0 for one group per row
  int kslog, rounds;
  int kfirst, kcount;      // the chunks of this call: all kc, or a slice of them
};

// Runs a wave's share.  GS = 32-position steps per group (1, 2, 4); one group
// per row is GS = 4 with pmul = 0: its scale is folded in after every chunk
// (the formula is linear in the chunk), which keeps the offset sums short.
// NP: planes of A that are summed (x = plane 0 + plane 1 + ..).
//   fill()            puts A where `af` reads it; called by every wave once,
//                     after the first batch of codes has been requested
//   af.load(c, j, p)  8 positions 128c + 32j + 8·(lane/16) of token lane % 16
//   end(unit, y)      2^-12 of the wave's sums of its K share of a unit, every round
// The group sum Σx comes from the matrix cores too (A times a tile of ones):
// in D's layout it already sits where the fold needs it, and the matrix cores
// are idle in a product that is bound by its codes.
// CENTRED: the operand is q - zc with zc the zero point clamped to 0..15, and
// only z - zc (0 for a zero point in the code range) is taken off the group
// sum.  Activations of 24 bits fill the fp32 sums, whose rounding the offset
// would then magnify (2-bit codes: 1.8e-6 against 4e-7 for the result); it
// takes 28 VALU instructions per operand instead of 8, so only they use it.
template <int GS, int RT, int NP, int B, bool CENTRED, class AF, class FF, class EF>
__device__ __forceinline__ void l4_units(const L4Stream& st, int64_t first, int64_t step, const AF& af, const FF& fill,
                                         const EF& end) {
  constexpr int NG = 4 / GS;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int ks = 1 << st.kslog, sl = wave & (ks - 1);
  const int cps = (st.kcount + ks - 1) >> st.kslog;
  const int c0 = st.kfirst + sl * cps, c1 = std::min(st.kfirst + st.kcount, c0 + cps);
  const int64_t u0 = first + (wave >> st.kslog);
  const L4Consts kc;
  struct Batch {
    u32x4_t cw[B][RT];
    float2 p[B][RT][NG];
    uint4 a[AF::kPrefetch ? B : 1][AF::kPrefetch ? 4 : 1][NP];
  };
  auto load = [&](int r, int c, Batch& b) {
    const int64_t unit = std::min<int64_t>(u0 + r * step, st.units - 1);   // past the last: computed, not stored
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const u32x4_t* cp = st.codes + (unit * RT + t) * st.kc * 64 + lane;
      const float2* pp = st.params + (unit * RT + t) * st.Gp * kL4Rows + (lane & 15);
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int cc = std::max(0, std::min(c + i, c1 - 1));   // past the end: the last chunk again, not used
        b.cw[i][t] = cp[(int64_t)cc * 64];
#pragma unroll
        for (int g = 0; g < NG; ++g) b.p[i][t][g] = pp[(int64_t)(cc * NG + g) * st.pmul];
      }
    }
    if (AF::kPrefetch) {
#pragma unroll
      for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            b.a[AF::kPrefetch ? i : 0][AF::kPrefetch ? j : 0][p] = af.load(std::max(0, std::min(c + i, c1 - 1)), j, p);
    }
  };
  f32x4_t y[RT];
  auto compute = [&](int c, const Batch& b) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (c + i >= c1) break;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t sx = {0.f, 0.f, 0.f, 0.f};
        f32x4_t acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < GS; ++q) {
          const int j = g * GS + q;
          bf16x8_t a[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p)
            a[p] = __builtin_bit_cast(
                bf16x8_t, AF::kPrefetch ? b.a[AF::kPrefetch ? i : 0][AF::kPrefetch ? j : 0][p] : af.load(c + i, j, p));
#pragma unroll
          for (int p = 0; p < NP; ++p) sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], kc.ones(), sx, 0, 0, 0);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const bf16x8_t w = CENTRED ? kc.unpack_centred(b.cw[i][t][j], l4_centre_off(b.p[i][t][g].y))
                                       : kc.unpack(b.cw[i][t][j]);
#pragma unroll
            for (int p = 0; p < NP; ++p) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], w, acc[t], 0, 0, 0);
          }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const float s = b.p[i][t][g].x, y0 = b.p[i][t][g].y;
          const float z = CENTRED ? y0 - 128.f - l4_centre(y0) : l4_zero(y0);
#pragma unroll
          for (int v = 0; v < 4; ++v) y[t][v] = fmaf(s, fmaf(-z, sx[v], acc[t][v]), y[t][v]);
        }
      }
    }
  };
  Batch cur, nxt;
  load(0, c0, cur);
  fill();
  for (int r = 0; r < st.rounds; ++r) {
#pragma unroll
    for (int t = 0; t < RT; ++t) y[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c < c1; c += B) {
      const bool more = c + B < c1;
      load(more ? r : std::min(r + 1, st.rounds - 1), more ? c + B : c0, nxt);
      compute(c, cur);
      cur = nxt;
    }
    end(u0 + r * step, y);
  }
}

// 2^12 times the sums of the ks waves of each unit, added in wave order through
// LDS.  red: [16 waves][RT][quads][64] floats, quads = 4-token groups that hold
// tokens.  Calls out(unit, token, row, value[RT]) once per result; every wave
// calls it.
template <int RT, class OF>
__device__ __forceinline__ void l4_finish(float* red, int quads, int tokens, int kslog, int64_t unit,
                                          const f32x4_t (&y)[RT], const OF& out) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (kslog == 0) {   // every wave holds its whole unit: D[4·(lane/16) + v][lane % 16]
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (4 * (lane >> 4) + v >= tokens) break;
      float z[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) z[t] = y[t][v] * kL4Up;
      out(unit, 4 * (lane >> 4) + v, lane & 15, z);
    }
    return;
  }
  const int ks = 1 << kslog, upw = kL4Waves >> kslog;
  if ((lane >> 4) < quads) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
      *reinterpret_cast<f32x4_t*>(red + ((wave * RT + t) * quads + (lane >> 4)) * 64 + (lane & 15) * 4) = y[t];
  }
  __syncthreads();
  const int64_t base = unit - (wave >> kslog);   // the round's first unit
  for (int i = tid; i < upw * quads * 64; i += kL4Threads) {
    const int ul = i / (quads * 64), tok = (i >> 4) % (quads * 4), row = i & 15;
    if (tok >= tokens) continue;
    float z[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float* p = red + (((ul << kslog) * RT + t) * quads + (tok >> 2)) * 64 + row * 4 + (tok & 3);
      z[t] = p[0];
      for (int s = 1; s < ks; ++s) z[t] += p[s * RT * quads * 64];
      z[t] *= kL4Up;
    }
    out(base + ul, tok, row, z);
  }
  __syncthreads();
}

// A fragments from memory: rows in processing order, planes `plane` elements apart
struct L4GlobalA {
  static constexpr bool kPrefetch = true;
  const uint16_t* row;   // this lane's token row + 8·(lane/16)
  int64_t plane;
  __device__ __forceinline__ uint4 load(int c, int j, int p) const {
    return *reinterpret_cast<const uint4*>(row + p * plane + c * kL4Chunk + 32 * j);
  }
};

// A fragments from LDS: rows 16 bytes apart in the banks
constexpr int kL4Pad = 8;
struct L4LdsA {
  static constexpr bool kPrefetch = false;
  const uint16_t* row;
  int plane, first = 0;   // the chunk that the rows begin with
  __device__ __forceinline__ uint4 load(int c, int j, int p) const {
    return *reinterpret_cast<const uint4*>(row + p * plane + (c - first) * kL4Chunk + 32 * j);
  }
};

// Host: the split of `units` units (of rt row tiles) over `wgs` workgroups, ks
// = 1 << kslog waves sharing a unit.  A round costs a wave its chunks (about
// 1 us for each of 16 waves' KB at the HBM's pace) and, where waves share,
// the sums through LDS and their two barriers (about the same).  Fullest
// rounds alone chose 7 rounds of 2 chunks over 1 of 16 for 64 units on 5
// workgroups: 61 us instead of 35.
struct L4Split {
  int kslog, rounds;
};
inline L4Split l4_split(int64_t units, int64_t wgs, int64_t kc, int rt) {
  L4Split best{0, 1};
  int64_t least = -1;
  for (int lg = 0; lg <= 4; ++lg) {
    if (lg > 0 && (int64_t(1) << lg) > kc) break;
    const int64_t rounds = ceil_div(units, wgs * (kL4Waves >> lg)), cps = (kc + (1 << lg) - 1) >> lg;
    const int64_t cost = rounds * (cps * rt * 5 + (lg ? 5 : 1));
    if (least < 0 || cost < least) {
      least = cost;
      best = L4Split{lg, (int)rounds};
    }
  }
  return best;
}

// one row of n bf16 into LDS (16-byte pieces when the row is 16-byte aligned)
__device__ __forceinline__ void l4_row_to_lds(const uint16_t* __restrict__ x, int64_t n, int vec, uint8_t* lds, int tid,
                                              int threads) {
  int64_t done = 0;
  if (vec) {
    const int pieces = (int)(n / 8);
    for (int i = tid; i < pieces; i += threads)
      reinterpret_cast<uint4*>(lds)[i] = reinterpret_cast<const uint4*>(x)[i];
    done = (int64_t)pieces * 8;
  }
  for (int64_t i = done + tid; i < n; i += threads) reinterpret_cast<uint16_t*>(lds)[i] = x[i];
}

// X' = X[:, order] of `tokens` rows into LDS (rows n128 + 8 apart), through raw
// copies of `batch` rows at a time: LDS serves scattered 2-byte reads in a few
// cycles where the memory pipe takes one or more per lane.
__device__ __forceinline__ void l4_gather_lds(const uint16_t* __restrict__ X, int64_t ldx, int n, int vec,
                                              const int32_t* __restrict__ order, int n128, int tokens, int batch,
                                              uint16_t* xsh, uint8_t* raw) {
  const int tid = threadIdx.x, rrow = (n + 7) & ~7;   // raw rows start 16-byte aligned
  for (int t0 = 0; t0 < tokens; t0 += batch) {
    const int nt = std::min(batch, tokens - t0);
    if (t0) __syncthreads();   // the batch before has been gathered
    for (int t = 0; t < nt; ++t)
      l4_row_to_lds(X + (t0 + t) * ldx, n, vec, raw + (size_t)t * rrow * 2, tid, kL4Threads);
    __syncthreads();
    for (int p = 4 * tid; p < n128; p += 4 * kL4Threads) {
      const int4 o = *reinterpret_cast<const int4*>(order + p);
      const int a = std::max(o.x, 0), b = std::max(o.y, 0), c = std::max(o.z, 0), d = std::max(o.w, 0);
      for (int t = 0; t < nt; ++t) {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(raw) + (size_t)t * rrow;
        const uint32_t xa = x[a], xb = x[b], xc = x[c], xd = x[d];
        uint2 v;
        v.x = (o.x >= 0 ? xa : 0u) | (o.y >= 0 ? xb : 0u) << 16;
        v.y = (o.z >= 0 ? xc : 0u) | (o.w >= 0 ? xd : 0u) << 16;
        *reinterpret_cast<uint2*>(xsh + (t0 + t) * (n128 + kL4Pad) + p) = v;
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- values
__device__ __forceinline__ float l4_load(const void* p, int dtype, int64_t i) {
  if (dtype == GPTQ_FP32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ uint16_t l4_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }   // nearest even

__device__ __forceinline__ void l4_store(void* p, int dtype, int64_t i, float v) {
  if (dtype == GPTQ_FP32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = l4_bf16(v);
}

__device__ __forceinline__ float l4_activate(float x, int act) {
  switch (act) {
    case GPTQ_ACT_RELU: return x < 0.f ? 0.f : x;   // NaN stays NaN
    case GPTQ_ACT_SILU: return x / (1.f + expf(-x));
    case GPTQ_ACT_GELU: return 0.5f * x * erfcf(-0.70710678118654752f * x);
    // ½x(1 + tanh u) = x / (1 + e^(-2u)), without the cancellation of 1 + tanh
    case GPTQ_ACT_GELU_TANH: return x / (1.f + expf(-1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.f)));
    default: return x;
  }
}

}  // namespace gptq
