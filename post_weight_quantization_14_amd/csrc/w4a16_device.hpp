// Device pieces shared by the layers built on packed 2/3/4-bit weights
// (w4a16_linear.hip, w4a16_moe.hip): operand unpacking, the K loop of a
// 16-row tile, activations and typed loads and stores.
#pragma once

#include "gptq_internal.hpp"

namespace gptq {

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kL4Rows = 16;     // weight rows per packed tile (MFMA N)
constexpr int kL4Chunk = 128;   // positions per packed chunk (4 MFMA k-steps of 32)

// ---------------------------------------------------------------- operands
// A 4-bit code q becomes the bf16 16 + q with one shift and one AND-OR: bf16
// numbers in [16, 32) are spaced 1/8, so q sits in mantissa bits 3..6 of
// 0x4180.  Then
//   Σ_k x_k·(q_k - z) = Σ_k x_k·(16 + q_k) - (16 + z)·Σ_k x_k,
// with exact bf16 x bf16 products on the left.  16 is the smallest offset
// whose binade holds every 4-bit code: the two sums are then at most ~5x the
// difference for codes around the middle, and fp32 sums lose 2-3 bits to
// the subtraction (an offset of 128 loses 5).
struct L4Consts {
  uint32_t m, c, one;
  // hidden from constant folding: VOP3 takes no literals, so as visible
  // constants each AND-OR would compile to two instructions
  __device__ __forceinline__ L4Consts() : m(0x00780078u), c(0x41804180u), one(0x3F803F80u) {
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
  // q - zc for an integer 0 <= zc <= 15 (off = 16 + zc): exact in bf16, so the
  // upper halves of the fp32 differences are the operand itself
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
  __device__ __forceinline__ bf16x8_t ones() const {
    return __builtin_bit_cast(bf16x8_t, u32x4_t{one, one, one, one});
  }
};

// packed group parameters hold (s, 128 + z)
__device__ __forceinline__ float l4_zero(float y) { return y - 112.f; }
__device__ __forceinline__ float l4_centre(float y) { return fminf(fmaxf(y - 128.f, 0.f), 15.f); }

// ---------------------------------------------------------------- the K loop
// y[r] += the product of one 16-token tile with RT row tiles over chunks
// [c0, c1), NP planes of A summed (x = plane 0 + plane 1).  GS = 32-position
// steps per group (1, 2, 4); one group per row is passed as GS = 4 with
// pmul = 0, which folds the group's scale in after every chunk (the formula is
// linear in the chunk) and keeps the offset sums short.
//   cp[r]  codes of row tile r, this lane's u32x4 of chunk 0
//   pp[r]  (s, 128 + z) of this lane's row, group 0; groups are pmul (16) apart
//   af     A fragments: load(c, j, p) = 8 positions 128c + 32j + 8·(lane/16)
//          of this lane's token row (lane % 16), plane p
// The group sum Σx comes from the matrix cores too (A times a tile of ones):
// in D's layout it already sits where the fold needs it, and the matrix cores
// are idle in a product that is bound by the code stream.
// Loads run one batch ahead of the products in registers.
// CENTRED: the operand is q - zc with zc the zero point clamped to 0..15, and
// only z - zc (0 for a zero point in the code range) is taken off the group
// sum.  Activations of 24 bits fill the fp32 sums, whose rounding the offset
// would then magnify (2-bit codes: 1.8e-6 against 4e-7 for the result); it
// takes 28 VALU instructions per operand instead of 8, so only they use it.
template <int GS, int RT, int NP, int B, bool CENTRED, class AF>
__device__ __forceinline__ void l4_stream(const AF& af, const u32x4_t* const (&cp)[RT],
                                          const float2* const (&pp)[RT], int pmul, int c0, int c1,
                                          const L4Consts& kc, f32x4_t (&y)[RT]) {
  constexpr int NG = 4 / GS;
  struct Batch {
    u32x4_t cw[B][RT];
    float2 p[B][RT][NG];
    uint4 a[B][AF::kPrefetch ? 4 : 1][NP];
  };
  const int last = c1 - 1;
  auto load = [&](int c, Batch& b) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int cc = c + i < last ? c + i : last;   // past the end: the last chunk again, not used
#pragma unroll
      for (int r = 0; r < RT; ++r) b.cw[i][r] = cp[r][(int64_t)cc * 64];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int g = 0; g < NG; ++g) b.p[i][r][g] = pp[r][(int64_t)(cc * NG + g) * pmul];
      if (AF::kPrefetch) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < NP; ++p) b.a[i][AF::kPrefetch ? j : 0][p] = af.load(cc, j, p);
      }
    }
  };
  auto compute = [&](int c, const Batch& b) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (c + i >= c1) break;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t sx = {0.f, 0.f, 0.f, 0.f};
        f32x4_t acc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < GS; ++q) {
          const int j = g * GS + q;
          bf16x8_t a[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p)
            a[p] = __builtin_bit_cast(bf16x8_t, AF::kPrefetch ? b.a[i][AF::kPrefetch ? j : 0][p] : af.load(c + i, j, p));
#pragma unroll
          for (int p = 0; p < NP; ++p) sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], kc.ones(), sx, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const bf16x8_t w = CENTRED ? kc.unpack_centred(b.cw[i][r][j], 16.f + l4_centre(b.p[i][r][g].y))
                                       : kc.unpack(b.cw[i][r][j]);
#pragma unroll
            for (int p = 0; p < NP; ++p) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p], w, acc[r], 0, 0, 0);
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float s = b.p[i][r][g].x, y0 = b.p[i][r][g].y;
          const float z = CENTRED ? y0 - 128.f - l4_centre(y0) : l4_zero(y0);
#pragma unroll
          for (int v = 0; v < 4; ++v) y[r][v] = fmaf(s, fmaf(-z, sx[v], acc[r][v]), y[r][v]);
        }
      }
    }
  };
  if (c0 >= c1) return;
  Batch cur, nxt;
  load(c0, cur);
  for (int c = c0; c < c1; c += B) {
    load(c + B, nxt);
    compute(c, cur);
    cur = nxt;
  }
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
