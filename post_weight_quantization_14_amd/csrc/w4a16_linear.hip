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
  // N tokens (runs of 4, 8 apart, from t) of one row.  The residual loads of
  // them all are in flight together, a caller's further blocks may be loaded
  // before the first is finished: under the type's branch and a range check
  // each, they would be one memory latency apart.
  template <int N>
  __device__ __forceinline__ void residual(int64_t t, int64_t tokens, int64_t r, int64_t m, float (&rv)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) rv[i] = 0.f;
    if (!res || r >= m || t >= tokens) return;
    if (res_dt == GPTQ_FP32) {
#pragma unroll
      for (int i = 0; i < N; ++i)   // past the last token: the last one's, not used
        rv[i] = static_cast<const float*>(res)[std::min<int64_t>(t + 8 * (i / 4) + (i & 3), tokens - 1) * ldr + r];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        rv[i] = __uint_as_float(
            (uint32_t) static_cast<const uint16_t*>(res)[std::min<int64_t>(t + 8 * (i / 4) + (i & 3), tokens - 1) * ldr + r]
            << 16);
    }
  }
  template <int N, bool GATED>
  __device__ __forceinline__ void block(int64_t t, int64_t tokens, int64_t r, int64_t m, const float (&v)[N],
                                        const float (&u)[N], const float (&rv)[N]) const {
    if (r >= m || t >= tokens) return;
    const float b0 = bias ? l4_load(bias, bias_dt, r) : 0.f;
    float z[N];
    if (GATED) {
      const float b1 = bias2 ? l4_load(bias2, bias_dt, r) : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = l4_activate(v[i] + b0, act) * (u[i] + b1);
    } else if (act == GPTQ_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = v[i] + b0 + rv[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = l4_activate(v[i] + b0, act) + rv[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t ti = t + 8 * (i / 4) + (i & 3);
      if (ti < tokens) l4_store(Y, y_dt, ti * ldy + r, z[i]);
    }
  }
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

struct L4DecodeArgs {
  L4Stream st;
  const uint16_t* X;      // in-kernel gather: the activations and the order
  const int32_t* order;
  int64_t ldx, n;
  const uint16_t* Xp;     // else X' [tokens][n128]
  int64_t n128, m;
  int tokens, quads, vec, batch;   // batch: raw rows gathered at a time
  L4Epilogue ep;
};

// Few tokens: 16 of them (grid y), whose X' fits in LDS.  Unit = one row tile
// (linear) or one gate/up pair of tiles (glu).  X' is gathered here (GATHER) or
// copied from X' in memory.  Bound by the code stream from HBM, at small sizes
// by the chain launch - row - order - codes - sums and the call itself:
// 4096 x 4096, 1 token 6.9 us (9.4 with Python's call), 11008 x 4096 pair
// 16.4 us = 3.1 TB/s, 8192 x 29568 33.7 us = 4.1 TB/s.
template <int GS, bool GATED, bool GATHER>
__global__ __launch_bounds__(kL4Threads) void l4_decode_kernel(L4DecodeArgs a) {
  constexpr int RT = GATED ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int xrow = (int)a.n128 + kL4Pad;
  const int t0 = blockIdx.y * 16, tokens = std::min(16, a.tokens - t0);
  uint16_t* xsh = reinterpret_cast<uint16_t*>(lds);
  uint8_t* rest = lds + (size_t)std::min(16, a.tokens) * xrow * 2;
  float* red = reinterpret_cast<float*>(rest);   // after the gather, over its raw rows
  auto fill = [&] {
    if (GATHER) {
      l4_gather_lds(a.X + t0 * a.ldx, a.ldx, (int)a.n, a.vec, a.order, (int)a.n128, tokens, a.batch, xsh, rest);
    } else {
      const int pieces = (int)(a.n128 / 8);
      const uint16_t* xp = a.Xp + t0 * a.n128;
      for (int i = threadIdx.x; i < tokens * pieces; i += kL4Threads)
        *reinterpret_cast<uint4*>(xsh + (i / pieces) * xrow + 8 * (i % pieces)) =
            *reinterpret_cast<const uint4*>(xp + (int64_t)(i / pieces) * a.n128 + 8 * (i % pieces));
      __syncthreads();
    }
  };
  const int upw = kL4Waves >> a.st.kslog;
  auto end = [&](int64_t unit, const f32x4_t (&y)[RT]) {
    l4_finish<RT>(red, a.quads, tokens, a.st.kslog, unit, y, [&](int64_t u, int t, int row, const float (&z)[RT]) {
      const int64_t r = u * kL4Rows + row;
      if (u >= a.st.units || r >= a.m) return;
      if (GATED)
        a.ep.gated(t0 + t, r, z[0], z[RT - 1]);
      else
        a.ep.linear(t0 + t, r, z[0]);
    });
  };
  const int t = std::min(lane & 15, tokens - 1);   // rows past the last: computed, not stored
  // batches that leave the wave within 128 registers (16 waves on a CU)
  constexpr int B = GATED ? (GS == 1 ? 1 : 2) : (GS == 4 ? 4 : GS == 2 ? 3 : 2);
  const L4LdsA af{xsh + t * xrow + 8 * (lane >> 4), 0};
  l4_units<GS, RT, 1, B, false>(a.st, (int64_t)blockIdx.x * upw, (int64_t)gridDim.x * upw, af, fill, end);
}

// ---------------------------------------------------------------- many tokens
// v = h + m + l, exactly: 8 of its 24 bits each
struct L4Planes {
  uint32_t h, m, l;   // bf16 values in the upper halves
};
__device__ __forceinline__ L4Planes l4_planes(float v) {
  const uint32_t h = __float_as_uint(v) & 0xffff0000u;
  const float r = v - __uint_as_float(h);
  const uint32_t m = __float_as_uint(r) & 0xffff0000u;
  return {h, m, __float_as_uint(r - __uint_as_float(m))};
}

constexpr float kL4SumDown = 0x1p-7f;

// X' = X[:, order] and 2^-7 of its group sums (128 of them stay finite; the zero
// points take the other 2^-5, bf16 planes end at 2^-133), groups-major
// (sums[c·NG + g][t], for the tile kernel's contiguous copies, cut into three
// bf16 planes: an operand).  A row of X is read once, 16 bytes a
// thread, into LDS and gathered from there: 2-byte loads at scattered columns
// cost the memory pipe a cycle or more a lane (2048 x 4096: 13 us, through
// LDS 8.5), LDS serves 64 of them in a few cycles.  Thread: 8 positions; GS·4
// threads make one group's sum; a workgroup covers 4096 positions of a token.
// One token per workgroup: eight in a row, each behind a barrier, took 12 us.
template <int GS, bool LDS>
__global__ __launch_bounds__(512) void l4_gather_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                        const int32_t* __restrict__ order, int64_t n, int64_t n128,
                                                        uint16_t* __restrict__ Xp, uint2* __restrict__ sums,
                                                        int64_t tokens, int64_t tpad, int vec) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x;
  const int64_t p0 = (int64_t)blockIdx.y * 4096 + 8 * tid;
  const bool live = p0 < n128;   // n128 is a multiple of 128: whole 16-thread groups agree
  int oi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) oi[e] = -1;
  if (live) {
    const int4 o0 = *reinterpret_cast<const int4*>(order + p0), o1 = *reinterpret_cast<const int4*>(order + p0 + 4);
    oi[0] = o0.x, oi[1] = o0.y, oi[2] = o0.z, oi[3] = o0.w;
    oi[4] = o1.x, oi[5] = o1.y, oi[6] = o1.z, oi[7] = o1.w;
  }
  const int64_t t = blockIdx.x;
  const uint16_t* x = X + t * ldx;
  if (LDS) {
    l4_row_to_lds(x, n, vec, lds, tid, 512);
    __syncthreads();
    x = reinterpret_cast<const uint16_t*>(lds);
  }
  if (!live) return;
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {   // unconditional reads, all in flight together
    const uint16_t xe = x[oi[e] >= 0 ? oi[e] : 0];
    v[e] = oi[e] >= 0 ? xe : 0u;
  }
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(__uint_as_float(v[e] << 16), kL4SumDown, s);
  *reinterpret_cast<u32x4_t*>(Xp + t * n128 + p0) =
      u32x4_t{v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
#pragma unroll
  for (int d = 1; d < 4 * GS; d <<= 1) s += __shfl_xor(s, d);
  if ((tid & (4 * GS - 1)) == 0) {
    const L4Planes p = l4_planes(s);
    sums[(p0 / (32 * GS)) * tpad + t] = make_uint2((p.h >> 16) | p.m, p.l >> 16);
  }
}

typedef __attribute__((address_space(3))) void lds_void_t;

struct L4GemmArgs {
  const uint16_t* Xp;     // [tokens][n128]
  const uint2* sums;      // [kc·NG][tpad]: three bf16 planes
  const float2* params;
  const u32x4_t* codes;
  float* part;            // split tiles: [splits][tiles - whole][fragments]
  int64_t n128, kc, Gp, mt, m, tokens, tpad;
  // 32 bits, like all that is divided: 64-bit divisions before the first load
  // took 1 us of a small call
  uint32_t tblocks;
  uint32_t whole, parted; // tiles 0 .. whole - 1 take the whole K range, the other `parted` `splits` slices
  int pmul, splits, chunks;   // K slices, chunks per slice
  L4Epilogue ep;
};

// Tile: 32·MT·TG tokens x 32·NB·RG rows; TG·RG waves of 32·MT tokens x 32·NB
// rows on v_mfma_f32_32x32x16_bf16, and KG such groups of waves that take every
// KG-th chunk of the slice (few tokens: the chain of chunks is latency, and a
// workgroup's groups run KG of them side by side).
//
// X' comes through LDS (direct copies, two slots), the codes straight into
// registers in operand order: 4 bits a weight would be 16 as operands in LDS.
// Bound by issue: 2048 x 22016 x 4096 takes 358 us = 1.03 PFLOP/s in 675 000
// cycles at 1.89 GHz, and the matrix instructions' 396 000 and the others'
// 282 000 add up to that: the two waves of a SIMD leave the same barrier and
// unpack and multiply in step, so neither hides the other's vector work.  (The
// library's bf16 product of that shape takes 424 us.)  A wave of 128 tokens x
// 32 rows unpacks an operand once for four products; one of 64 x 64, which
// halves the LDS reads instead, took 3 % longer.  The zero points' term is one
// more product per group, not a fold with the sums: 16 vector instructions and 4
// LDS reads fewer for each 32 x 32 (2 % of the time).  Tried and not kept: two
// chunks in flight behind a second barrier (+2 %), the fold between the next
// products (+7 %: it reads the A fragments twice), A fragments two steps ahead
// (0 %), waves of 128 x 64, one per SIMD (+35 %).
template <int GS, int MT, int NB, int TG, int RG, int KG>
struct L4Tile {
  static constexpr int kTokens = 32 * MT * TG, kRows = 32 * NB * RG, kGroup = TG * RG, kThreads = 64 * kGroup * KG;
  static constexpr int kNG = 4 / GS;
  static constexpr int kX = kTokens * 256;                                 // X' of one chunk
  static constexpr int kBytes = kX + kNG * kTokens * 8;   // and its group sums
  static constexpr int kXCopies = kX / 1024 / kGroup;                      // 1 KB copies per wave
  static_assert(kX % (2048 * kGroup) == 0, "copies split evenly over the waves, two at a time");
  static_assert(kTokens <= 128, "the sums of a group are one copy of up to 64 lanes, two tokens each");
};

template <int GS, int MT, int NB, int TG, int RG, int KG, bool GATED>
__device__ __forceinline__ void l4_gemm_tile(const L4GemmArgs& a, uint8_t* __restrict__ s0, uint8_t* __restrict__ s1) {
  using Tl = L4Tile<GS, MT, NB, TG, RG, KG>;
  constexpr int NG = Tl::kNG, U = Tl::kXCopies;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kg = wave / Tl::kGroup, gw = wave % Tl::kGroup, rg = gw % RG, tg = gw / RG;
  // whole tiles first, then the slices of the others, slice by slice; tiles
  // run along the token blocks of a row block
  uint32_t i = blockIdx.x;
  const int64_t parted = a.parted;
  const bool split = i >= a.whole && a.splits > 1;
  int sl = 0;
  if (split) {
    const uint32_t j = i - a.whole;
    sl = (int)(j / a.parted);
    i = a.whole + j % a.parted;
  }
  const int64_t tb = i % a.tblocks, rb = i / a.tblocks;
  const int64_t t0 = tb * Tl::kTokens;
  const int c0 = sl * a.chunks, nch = split ? std::min(a.chunks, (int)a.kc - c0) : (int)a.kc;
  const int steps = (nch + KG - 1) / KG;   // this wave's chunk of step s: s·KG + kg

  // X' rows past the last token lie outside the descriptor and read as zero
  const int64_t trows = std::min<int64_t>(Tl::kTokens, a.tokens - t0);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(a.Xp + t0 * a.n128), 0, (int32_t)(trows * a.n128 * 2), 0x00020000);
  int32_t xoff[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // 1 KB = 4 token rows of 16 pieces; row t keeps piece p in slot p ^ (t mod 16)
    const int q = (gw * U + u) * 64 + lane, t = q >> 4, pc = (q & 15) ^ (t & 15);
    xoff[u] = (int32_t)(t * a.n128 * 2 + pc * 16);
  }
  // copies of the sums, two tokens a lane, a group's each, spread over the waves
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint2*>(a.sums + t0), 0, (int32_t)std::min<int64_t>((a.kc * NG * a.tpad - t0) * 8, 0x7fffffff),
      0x00020000);
  auto issue = [&](int s, uint8_t* slots, int u0, int u1) {   // copies u0 .. u1 - 1; the sums with the first
    uint8_t* slot = slots + kg * Tl::kBytes;
    const int cc = c0 + std::min(s * KG + kg, nch - 1);
#pragma unroll
    for (int u = u0; u < u1; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(slot + (gw * U + u) * 1024), 16, xoff[u], cc * 256, 0, 0);
    if (u0) return;
#pragma unroll
    for (int k = 0; k < (NG + Tl::kGroup - 1) / Tl::kGroup; ++k) {
      const int g = k * Tl::kGroup + gw;
      if ((NG % Tl::kGroup == 0 || g < NG) && (Tl::kTokens == 128 || lane < Tl::kTokens / 2))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(slot + Tl::kX + g * Tl::kTokens * 8), 16, lane * 16,
                                                (int32_t)((cc * NG + g) * a.tpad * 8), 0, 0);
    }
  };

  // operand b of a wave's 32·NB rows: lane l feeds row l % 32 of 32, which is
  // row l % 16 of packed tile 2b + (l / 16) % 2; for two operands of gate/up
  // pairs, whose tiles alternate, tile b + 2·((l / 16) % 2): b = 0 all gate,
  // b = 1 all up (one operand holds a gate tile and its up tile side by side).
  // Positions 32j + 16h + 8(l / 32).. of a chunk are word j of the packed lane
  // 16·(2h + l / 32) + l % 16.
  const int half = (lane >> 4) & 1;
  const u32x4_t* cp[NB][2];
  const float2* pp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t tile =
        std::min<int64_t>((rb * RG + rg) * 2 * NB + (GATED && NB == 2 ? b + 2 * half : 2 * b + half), a.mt - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      cp[b][h] = a.codes + (tile * a.kc + c0) * 64 + 16 * (2 * h + (lane >> 5)) + (lane & 15);
    pp[b] = a.params + tile * a.Gp * kL4Rows + (lane & 15) + (int64_t)c0 * NG * a.pmul;
  }
  struct Codes {
    u32x4_t w[NB][2];
    float2 p[NB][NG];
  };
  auto fetch = [&](int c, Codes& k) {
    const int cc = std::min(c * KG + kg, nch - 1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) k.w[b][h] = cp[b][h][(int64_t)cc * 64];
#pragma unroll
      for (int g = 0; g < NG; ++g) k.p[b][g] = pp[b][(int64_t)(cc * NG + g) * a.pmul];
    }
  };

  const L4Consts kc;
  f32x16_t y[MT][NB];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) y[mt][b][v] = 0.f;

  const int trow = lane & 31;   // + 32·(MT·tg + mt): (t mod 16) is lane mod 16
  // One chunk.  Per 16-position step: the next step's A fragments are read
  // from LDS, this step's NB operands are unpacked and MT·NB products issued;
  // the scheduling barriers spread the VALU work between the matrix
  // instructions (left alone the compiler unpacks a whole group first, and
  // reads each fragment right before its use).
  auto compute = [&](const uint8_t* cur, const Codes& k, auto&& ahead) {
    auto frag = [&](int st, int mt) {
      const int t = 32 * (MT * tg + mt) + trow;
      return *reinterpret_cast<const u32x4_t*>(cur + t * 256 + (((2 * st + (lane >> 5)) ^ (t & 15)) * 16));
    };
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x16_t acc[MT][NB];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[mt][b][v] = 0.f;
      // -(16 + z)·Σx on the matrix cores too, both in exact bf16 planes: lanes
      // 0..31 hold the sum's three against z's first two, the others against
      // its third
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const L4Planes z = l4_planes(l4_zero(k.p[b][g].y) * -(kL4Down / kL4SumDown));
        const uint32_t z0 = lane < 32 ? z.h : z.l, z1 = lane < 32 ? z.m : 0u;
        const bf16x8_t zp = __builtin_bit_cast(bf16x8_t, u32x4_t{z0 | (z0 >> 16), z0 >> 16, z1 | (z1 >> 16), z1 >> 16});
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint2 sx = *reinterpret_cast<const uint2*>(cur + Tl::kX + (g * Tl::kTokens + 32 * (MT * tg + mt) + trow) * 8);
          acc[mt][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, u32x4_t{sx.x, sx.y, sx.x, sx.y}),
                                                               zp, acc[mt][b], 0, 0, 0);
        }
      }
      u32x4_t av[2][MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) av[0][mt] = frag(g * 2 * GS, mt);
#pragma unroll
      for (int q = 0; q < 2 * GS; ++q) {
        const int st = g * 2 * GS + q;
        ahead(st);
        if (q + 1 < 2 * GS) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) av[(q + 1) & 1][mt] = frag(st + 1, mt);
        }
        bf16x8_t w[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) w[b] = kc.unpack(k.w[b][st & 1][st >> 1]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[mt][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, av[q & 1][mt]), w[b],
                                                                 acc[mt][b], 0, 0, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, MT, 0);   // LDS reads
#pragma unroll
        for (int u = 0; u < NB * MT; ++u) {
          __builtin_amdgcn_sched_group_barrier(0x002, 8 / MT, 0);       // VALU
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // MFMA
        }
      }
      // D: lane l, v: token 8·(v / 4) + 4·(l / 32) + v % 4, row l % 32
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int v = 0; v < 16; ++v) y[mt][b][v] = fmaf(k.p[b][g].x, acc[mt][b][v], y[mt][b][v]);
    }
  };

  Codes k0, k1;
  issue(0, s0, 0, U);
  fetch(0, k0);
  // One step: every copy of this step has landed (all waves', after the
  // barrier) and every wave is done with the other slot, which the next refills,
  // two copies at a time between this step's products (all at once right after
  // the barrier they block the wave: 4 % of the 2048-token pair).  The wait is
  // the builtin: of one in inline asm the compiler does not know that it covers
  // the codes, and puts another before their first use.
#define L4_STEP(s, cur, kcur, nxt, knxt)                                          \
  {                                                                               \
    asm volatile("" ::: "memory");                                                \
    __builtin_amdgcn_s_waitcnt(0x0070);   /* vmcnt(0) lgkmcnt(0) */               \
    __builtin_amdgcn_s_barrier();                                                 \
    asm volatile("" ::: "memory");                                                \
    if ((s) * KG + kg < nch)                                                      \
      compute(cur + kg * Tl::kBytes, kcur, [&](int st) {                          \
        if (2 * st >= U) return;                                                \
        issue((s) + 1, nxt, 2 * st, 2 * st + 2);                            \
        if (st == 0) fetch((s) + 1, knxt);                                        \
      });                                                                         \
  }
  for (int s = 0; s < steps; s += 2) {
    L4_STEP(s, s0, k0, s1, k1)
    L4_STEP(s + 1, s1, k1, s0, k0)
  }
#undef L4_STEP
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy may land after the workgroup ends

  if constexpr (KG > 1) {
    // The groups' sums through LDS: every wave leaves its fragments, then each
    // group adds and finishes its share of them (4 tokens of a row, gate and
    // up together), so the epilogue runs on all waves.
    constexpr int F = MT * 8, SHARE = MT * 4 / KG;
    static_assert(KG == 1 || (NB == 2 && (MT * 4) % KG == 0), "the fragments split evenly over the groups");
    static_assert(KG == 1 || (KG / 2) * Tl::kGroup * F * 1024 <= KG * Tl::kBytes, "half of the groups fit in each array");
    __syncthreads();   // every copy into the slots and every read of them is done
    auto at = [&](int k, int f) {
      return reinterpret_cast<f32x4_t*>(k < KG / 2 ? s0 : s1) + (((k % (KG / 2)) * Tl::kGroup + gw) * F + f) * 64 + lane;
    };
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const f32x16_t& v = y[f >> 3][(f >> 2) & 1];
      *at(kg, f) = f32x4_t{v[4 * (f & 3)], v[4 * (f & 3) + 1], v[4 * (f & 3) + 2], v[4 * (f & 3) + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SHARE; ++j) {
      const int c = kg * SHARE + j, mt = c >> 2, q = c & 3;
      f32x4_t z[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        z[b] = *at(0, mt * 8 + b * 4 + q);
#pragma unroll
        for (int k = 1; k < KG; ++k) z[b] += *at(k, mt * 8 + b * 4 + q);
        z[b] *= kL4Up;
      }
      if (split) {
        if (t0 + 32 * (MT * tg + mt) + 8 * q >= a.tokens) continue;   // not read
        f32x4_t* out = reinterpret_cast<f32x4_t*>(a.part) +
                       ((((int64_t)sl * parted + i - a.whole) * Tl::kGroup + gw) * F + mt * 8 + q) * 64 + lane;
        out[0] = z[0];
        out[256] = z[1];
        continue;
      }
      const int64_t t = t0 + 32 * (MT * tg + mt) + 8 * q + 4 * (lane >> 5);
      const int64_t r = (rb * RG + rg) * (GATED ? 32 : 64) + (lane & 31);
      const float g4[4] = {z[0][0], z[0][1], z[0][2], z[0][3]}, u4[4] = {z[1][0], z[1][1], z[1][2], z[1][3]};
      float r0[4], r1[4];
      if (!GATED) {
        a.ep.residual(t, a.tokens, r, a.m, r0);
        a.ep.residual(t, a.tokens, r + 32, a.m, r1);
      }
      a.ep.template block<4, GATED>(t, a.tokens, r, a.m, g4, u4, r0);
      if (!GATED) a.ep.template block<4, false>(t, a.tokens, r + 32, a.m, u4, u4, r1);
    }
    return;
  }

#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) y[mt][b][v] *= kL4Up;
  if (split) {
    // fragments as they lie: [slice][tile][wave][mt][b][q][lane] float4
    f32x4_t* out = reinterpret_cast<f32x4_t*>(a.part) +
                   (((int64_t)sl * parted + i - a.whole) * Tl::kGroup + gw) * (MT * NB * 4 * 64) + lane;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (t0 + 32 * (MT * tg + mt) + 8 * q < a.tokens)   // the others are not read
            out[((mt * NB + b) * 4 + q) * 64] =
                f32x4_t{y[mt][b][4 * q], y[mt][b][4 * q + 1], y[mt][b][4 * q + 2], y[mt][b][4 * q + 3]};
    return;
  }
  const int64_t rbase = (rb * RG + rg) * (GATED ? 16 : 32) + (lane & (GATED ? 15 : 31));
  static_assert(KG > 1 || NB == 1, "the tiles of one group of waves have one operand");
  float rv[MT][16];
  if (!GATED) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) a.ep.residual(t0 + 32 * (MT * tg + mt) + 4 * (lane >> 5), a.tokens, rbase, a.m, rv[mt]);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int64_t t = t0 + 32 * (MT * tg + mt) + 4 * (lane >> 5);
    if (!GATED) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = y[mt][0][i];
      a.ep.template block<16, false>(t, a.tokens, rbase, a.m, v, v, rv[mt]);
      continue;
    }
    // gate sits in the lower 16 lanes of each 32, up in the upper: of each 8
    // tokens (t + 8q + {0..3, 8..11}) they trade, and finish four each
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      float g4[4], u4[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float lo = y[mt][0][4 * q + v], hi = y[mt][0][4 * q + 4 + v];
        const float got = __shfl_xor(half ? lo : hi, 16);
        g4[v] = half ? got : lo;
        u4[v] = half ? hi : got;
      }
      a.ep.template block<4, true>(t + 8 * (q + half), a.tokens, rbase, a.m, g4, u4, u4);
    }
  }
}

template <int GS, int MT, int NB, int TG, int RG, int KG, bool GATED>
__global__ __launch_bounds__(64 * TG * RG * KG, 2) void l4_gemm_kernel(L4GemmArgs a) {
  using Tl = L4Tile<GS, MT, NB, TG, RG, KG>;
  // two arrays, not one indexed at run time: a read of one is then known not
  // to alias the copies in flight into the other
  __shared__ __attribute__((aligned(16))) uint8_t s0[KG * Tl::kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s1[KG * Tl::kBytes];
  l4_gemm_tile<GS, MT, NB, TG, RG, KG, GATED>(a, s0, s1);
}

// Sums the K slices in slice order and finishes.  Thread: one float4 fragment
// (4 tokens of one row; gate and up together for a pair).
template <int MT, int NB, int TG, int RG, bool GATED>
__global__ __launch_bounds__(256) void l4_reduce_kernel(L4GemmArgs a) {
  constexpr int FR = TG * RG * MT * NB * 4 * 64;   // fragments of one tile
  constexpr bool kPair = GATED && NB == 2;
  const int64_t per = a.parted;
  const uint32_t f = blockIdx.x * 256 + threadIdx.x;
  constexpr uint32_t PER = kPair ? FR / 2 : FR;
  if (f >= a.parted * PER) return;   // whole waves: PER is a multiple of 64
  const uint32_t i = f / PER;
  int k = (int)(f % PER);
  const int lane = k & 63, q = (k >> 6) & 3;
  k >>= 8;
  int b = 0;
  if (!kPair) {
    b = k % NB;
    k /= NB;
  }
  const int mt = k % MT, wave = k / MT, rg = wave % RG, tg = wave / RG;
  const uint32_t tile = a.whole + i;
  const int64_t tb = tile % a.tblocks, rb = tile / a.tblocks;
  const int64_t t = tb * (32 * MT * TG) + 32 * (MT * tg + mt) + 8 * q + 4 * (lane >> 5);
  if (t - 4 * (lane >> 5) >= a.tokens) return;   // whole waves
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.part) + (int64_t)i * FR + ((wave * MT + mt) * NB + b) * 256 + q * 64 + lane;
  f32x4_t v0 = p[0], v1 = {0.f, 0.f, 0.f, 0.f};
  if (kPair) v1 = p[256];
  for (int s = 1; s < a.splits; ++s) {
    v0 += p[(int64_t)s * per * FR];
    if (kPair) v1 += p[(int64_t)s * per * FR + 256];
  }
  if (GATED && NB == 1) {   // up is 16 lanes on
#pragma unroll
    for (int v = 0; v < 4; ++v) v1[v] = __shfl_xor(v0[v], 16);
    if (lane & 16) return;
  }
  const int64_t r = (rb * RG + rg) * (GATED ? 16 * NB : 32 * NB) + 32 * b + (lane & (GATED && NB == 1 ? 15 : 31));
  const float g4[4] = {v0[0], v0[1], v0[2], v0[3]}, u4[4] = {v1[0], v1[1], v1[2], v1[3]};
  float rv[4];
  if (!GATED) a.ep.residual(t, a.tokens, r, a.m, rv);
  a.ep.template block<4, GATED>(t, a.tokens, r, a.m, g4, u4, rv);
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

namespace {
// a tile, and the K slices that fill the GPU
struct L4Shape {
  int tokens = 128;                 // 32, 64 or 128, x 128 packed rows
  int64_t tblocks = 0, rblocks = 0;
  int64_t whole = 0;                // tiles that are not split
  int splits = 1, chunks = 0;
  double us = 0.0;                  // estimate of its kernels
};
// Full rounds of workgroups take whole tiles; what is left over, or a call of
// less than a round, is split along K to fill one (11008 x 4096, 256 tokens:
// 54 us with 172 whole tiles, 43 us with each in two slices).
L4Shape l4_tile(int tile_tokens, int64_t tokens, int64_t packed_rows, int64_t kc) {
  L4Shape s;
  s.tokens = tile_tokens;
  s.tblocks = ceil_div(tokens, s.tokens);
  s.rblocks = ceil_div(packed_rows, 128);
  const int64_t tiles = s.tblocks * s.rblocks;
  const int64_t round = s.tokens == 128 ? 512 : 256;   // workgroups that run at once
  const int64_t left = tiles % round;
  // four chunks at least in a slice: one step of the 4 groups, or 4 steps
  // (up to 12 chunks are not split at all: three steps of the 4 groups cost
  // less than the launch that adds the slices)
  const int64_t want = left == 0 || (kc <= 12 && s.tokens <= 64) ? 1 : std::min<int64_t>(kc / 4, round / left);
  s.chunks = (int)kc;
  if (want > 1) {
    s.chunks = (int)ceil_div(kc, want);
    s.splits = (int)ceil_div(kc, s.chunks);
  }
  s.whole = s.splits > 1 ? tiles - left : tiles;
  // Microseconds, fitted to runs of 4096..11008 wide weights: a step (a chunk;
  // four, of the tiles with four groups) and a workgroup's start and end.  Two
  // 128-token workgroups share a CU and take as long as one after the other.
  const double step = s.tokens == 128 ? 1.15 : s.tokens == 64 ? 2.6 : 1.9, over = s.tokens == 128 ? 7.0 : 5.0;
  auto rounds_us = [&](int64_t wgs, int64_t chunks) {
    const double steps = s.tokens == 128 ? (double)chunks : (double)ceil_div(chunks, 4);
    return (double)ceil_div(wgs, 256) * steps * step + (double)ceil_div(wgs, round) * over;
  };
  s.us = (s.whole ? rounds_us(s.whole, kc) : 0.0) + (s.splits > 1 ? rounds_us(left * s.splits, s.chunks) + 4.0 : 0.0);
  return s;
}
L4Shape l4_shape(int64_t tokens, int64_t packed_rows, int64_t kc) {
  L4Shape best = l4_tile(32, tokens, packed_rows, kc);
  for (int t : {64, 128}) {
    const L4Shape s = l4_tile(t, tokens, packed_rows, kc);
    if (s.us < best.us) best = s;
  }
  return best;
}
constexpr size_t kL4GatherLds = 65536;    // rows up to 32768 columns are gathered through LDS
// the decode kernel's tiles of 16 tokens against the tiled product: its start,
// and rounds of workgroups that take a share of the chunks and about 1 us of
// their own; and one launch less (4096 x 4096, 64 tokens: 14.5 us in four tiles
// of 16, 18.1 in one of 64; 80 tokens: 20.0 and 17.1 in tiles of 32)
double l4_decode_us(int64_t tiles, int64_t units, int64_t kc, int rt) {
  return 2.5 + (double)ceil_div(tiles * units, 256) * ((double)(kc * rt) / 16.0 + 1.0);
}
constexpr int64_t kL4GatherMax = 65536;   // up to this many elements of X' it gathers them itself
constexpr size_t kL4MaxLds = 158 * 1024;
constexpr int64_t kL4Cus = 256;

template <int GS, bool GATED>
gptq_status launch_l4_source(const L4DecodeArgs& d, bool gather, dim3 grid, size_t lds, hipStream_t stream) {
  const void* fn = gather ? (const void*)l4_decode_kernel<GS, GATED, true> : (const void*)l4_decode_kernel<GS, GATED, false>;
  if (lds > 65536) GPTQ_HIP_CHECK(hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  L4DecodeArgs args = d;
  void* argv[] = {&args};
  GPTQ_HIP_CHECK(hipLaunchKernel(fn, grid, dim3(kL4Threads), argv, lds, stream));
  return GPTQ_OK;
}

gptq_status launch_l4_decode(const L4DecodeArgs& d, int gs, bool gated, bool gather, dim3 grid, size_t lds,
                             hipStream_t stream) {
  switch (gs) {
    case 1: return gated ? launch_l4_source<1, true>(d, gather, grid, lds, stream) : launch_l4_source<1, false>(d, gather, grid, lds, stream);
    case 2: return gated ? launch_l4_source<2, true>(d, gather, grid, lds, stream) : launch_l4_source<2, false>(d, gather, grid, lds, stream);
    default: return gated ? launch_l4_source<4, true>(d, gather, grid, lds, stream) : launch_l4_source<4, false>(d, gather, grid, lds, stream);
  }
}

template <int GS, int MT, int NB, int TG, int RG, int KG, bool GATED>
gptq_status launch_l4_tile(const L4GemmArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((l4_gemm_kernel<GS, MT, NB, TG, RG, KG, GATED>), dim3(g.whole + g.parted * g.splits),
                     dim3(64 * TG * RG * KG), 0, stream, g);
  GPTQ_LAUNCH_CHECK();
  if (g.splits > 1) {
    const int64_t frags = (int64_t)g.parted * TG * RG * MT * NB * 4 * 64 / (GATED && NB == 2 ? 2 : 1);
    hipLaunchKernelGGL((l4_reduce_kernel<MT, NB, TG, RG, GATED>), dim3((unsigned)ceil_div(frags, 256)), dim3(256), 0,
                       stream, g);
    GPTQ_LAUNCH_CHECK();
  }
  return GPTQ_OK;
}

template <int GS, bool GATED>
gptq_status launch_l4_shape(const L4GemmArgs& g, const L4Shape& s, hipStream_t stream) {
  if (s.tokens == 32) return launch_l4_tile<GS, 1, 2, 1, 2, 4, GATED>(g, stream);
  if (s.tokens == 64) return launch_l4_tile<GS, 2, 2, 1, 2, 4, GATED>(g, stream);
  return launch_l4_tile<GS, 4, 1, 1, 4, 1, GATED>(g, stream);
}

gptq_status launch_l4_gemm(const L4GemmArgs& g, const L4Shape& s, int gs, bool gated, hipStream_t stream) {
  switch (gs) {
    case 1: return gated ? launch_l4_shape<1, true>(g, s, stream) : launch_l4_shape<1, false>(g, s, stream);
    case 2: return gated ? launch_l4_shape<2, true>(g, s, stream) : launch_l4_shape<2, false>(g, s, stream);
    default: return gated ? launch_l4_shape<4, true>(g, s, stream) : launch_l4_shape<4, false>(g, s, stream);
  }
}
}  // namespace

namespace {
// What a launch sequence of tk tokens runs.  Few tokens whose X' and sums fit in
// LDS take the decode kernel, which gathers X' itself where that is a barrier or
// two of work; the others the tiles of `shape`.
struct L4Choice {
  bool decode = false, gather = false;
  int quads = 0, batch = 0;   // decode: 4-token groups of a tile, raw rows gathered at a time
  size_t lds = 0;
  L4Shape shape;
};
L4Choice l4_choose(int64_t tk, const W4Layout& L, bool gated) {
  L4Choice c;
  const int rt = gated ? 2 : 1;
  const int64_t ttiles = ceil_div(tk, 16);
  c.shape = l4_shape(tk, L.mt * kL4Rows, L.kc);
  if (ttiles > 1 && l4_decode_us(ttiles, L.mt / rt, L.kc, rt) >= c.shape.us + 3.0) return c;
  const int64_t tt = std::min<int64_t>(tk, 16);   // tokens of a tile
  c.quads = (int)ceil_div(tt, 4);
  const size_t rows = (size_t)tt * (size_t)(L.n128 + kL4Pad) * 2;
  const size_t red = (size_t)kL4Waves * rt * c.quads * 64 * sizeof(float);
  const size_t raw = (size_t)round_up(L.n * 2, 16);
  c.decode = rows + red <= kL4MaxLds;
  if (!c.decode) return c;
  c.batch = (int)std::min<int64_t>(tt, (int64_t)((kL4MaxLds - rows) / raw));
  c.gather = 2 * c.batch >= tt && tt * L.n128 <= kL4GatherMax;
  c.lds = rows + std::max(red, c.gather ? raw * (size_t)c.batch : 0);
  return c;
}

// the K slices' partial sums of a launch sequence of tk tokens
size_t l4_part_bytes(int64_t tk, int64_t packed_rows, int64_t kc) {
  const L4Shape s = l4_shape(tk, packed_rows, kc);
  if (s.splits == 1) return 0;
  return align256((size_t)(s.splits * (s.tblocks * s.rblocks - s.whole)) * (size_t)(s.tokens * 128) * sizeof(float));
}
}  // namespace

L4LinearPlan plan_w4a16_linear(int64_t tokens, int64_t n, int64_t packed_rows) {
  L4LinearPlan p;
  const int64_t kc = ceil_div(n, kL4Chunk), n128 = kc * kL4Chunk;
  p.block = std::min<int64_t>(std::max<int64_t>(tokens, 1), kL4BlockTokens);
  p.tpad = round_up(p.block, 256);
  p.xs_off = align256((size_t)(p.block * n128) * sizeof(uint16_t));
  p.part_off = p.xs_off + align256((size_t)(p.tpad * (n128 / 32)) * sizeof(uint2));
  p.total = p.part_off;
  // the last, shorter block of a long call may take more slices than the others
  for (int64_t tk : {p.block, tokens % p.block})
    if (tk > 0) p.total = std::max(p.total, p.part_off + l4_part_bytes(tk, packed_rows, kc));
  return p;
}

L4Path w4a16_linear_path(int64_t tokens, const W4Layout& L, bool gated) {
  const L4Choice c = l4_choose(std::min(tokens, kL4BlockTokens), L, gated);
  if (c.decode) return {16, c.gather, 0, 0, 1};
  return {c.shape.tokens, 0, (int)c.shape.whole, (int)(c.shape.tblocks * c.shape.rblocks - c.shape.whole), c.shape.splits};
}

// Fewer tokens may be cut into more slices (2048 tokens of 4096 x 4096 fill the
// GPU with whole tiles, 1024 take two slices), so the largest of the partial
// sums of any count up to `tokens` is taken: the tiles change every 32 tokens,
// 128 counts at most (5 us on the host, which is why a call checks its own
// plan's size instead).
size_t w4a16_linear_workspace(int64_t tokens, int64_t n, int64_t packed_rows) {
  const L4LinearPlan p = plan_w4a16_linear(tokens, n, packed_rows);
  size_t part = 0;
  for (int64_t t = 32; t < p.block + 32; t += 32)
    part = std::max(part, l4_part_bytes(std::min(t, p.block), packed_rows, ceil_div(n, kL4Chunk)));
  return p.part_off + part;
}

gptq_status run_w4a16_linear(const L4Call& c, const W4Layout& L, bool gated, void* ws, const L4LinearPlan& p,
                             hipStream_t stream) {
  const char* base = static_cast<const char*>(c.packed);
  char* w = static_cast<char*>(ws);
  uint16_t* Xp = reinterpret_cast<uint16_t*>(w);
  uint2* xs = reinterpret_cast<uint2*>(w + p.xs_off);
  const int32_t* order = reinterpret_cast<const int32_t*>(base + L.order_off);
  L4Stream st;
  st.params = reinterpret_cast<const float2*>(base + L.param_off);
  st.codes = reinterpret_cast<const u32x4_t*>(base + L.code_off);
  st.kc = L.kc;
  st.Gp = L.Gp;
  st.units = gated ? L.mt / 2 : L.mt;
  const bool one_group = L.g >= L.n128;
  st.pmul = one_group ? 0 : kL4Rows;
  const int gs = one_group ? 4 : (int)(L.g / 32);
  const size_t ysz = c.y_dtype == GPTQ_FP32 ? 4 : 2, rsz = c.res_dtype == GPTQ_FP32 ? 4 : 2;
  const int vec = (reinterpret_cast<uintptr_t>(c.X) & 15) == 0 && c.ldx % 8 == 0;
  for (int64_t t0 = 0; t0 < c.tokens; t0 += p.block) {
    const int64_t tk = std::min<int64_t>(p.block, c.tokens - t0);
    const uint16_t* X = c.X + t0 * c.ldx;
    const L4Epilogue ep{c.act, c.bias_dtype, c.res_dtype, c.y_dtype, c.bias, c.bias2,
                        c.res ? static_cast<const char*>(c.res) + (size_t)(t0 * c.ldr) * rsz : nullptr,
                        static_cast<char*>(c.Y) + (size_t)(t0 * c.ldy) * ysz, c.ldr, c.ldy};
    const L4Choice ch = l4_choose(tk, L, gated);
    const L4Shape& sh = ch.shape;
    if (!ch.gather) {
      const size_t glds = (size_t)L.n * 2 <= kL4GatherLds ? (size_t)round_up(L.n * 2, 16) : 0;
      const dim3 ggrid((unsigned)tk, (unsigned)ceil_div(L.n128, 4096));
#define L4_GATHER(GS)                                                                                             \
  if (glds)                                                                                                       \
    hipLaunchKernelGGL((l4_gather_kernel<GS, true>), ggrid, dim3(512), glds, stream, X, c.ldx, order, L.n, L.n128, \
                       Xp, xs, tk, p.tpad, vec);                                                                  \
  else                                                                                                            \
    hipLaunchKernelGGL((l4_gather_kernel<GS, false>), ggrid, dim3(512), 0, stream, X, c.ldx, order, L.n, L.n128,  \
                       Xp, xs, tk, p.tpad, vec)
      switch (gs) {
        case 1: L4_GATHER(1); break;
        case 2: L4_GATHER(2); break;
        default: L4_GATHER(4); break;
      }
#undef L4_GATHER
      GPTQ_LAUNCH_CHECK();
    }
    if (ch.decode) {
      const int64_t ttiles = ceil_div(tk, 16);
      L4DecodeArgs d;
      d.quads = ch.quads;
      d.batch = ch.batch;
      d.X = X;
      d.order = order;
      d.ldx = c.ldx;
      d.n = L.n;
      d.Xp = Xp;
      d.n128 = L.n128;
      d.m = c.m;
      d.tokens = (int)tk;
      d.vec = vec;
      d.ep = ep;
      const int64_t wgs = std::min<int64_t>(st.units, std::max<int64_t>(1, kL4Cus / ttiles));
      const L4Split sp = l4_split(st.units, wgs, L.kc, gated ? 2 : 1);
      st.kslog = sp.kslog;
      st.rounds = sp.rounds;
      st.kfirst = 0;
      st.kcount = (int)L.kc;
      d.st = st;
      // workgroups that the split leaves without units are not launched
      const unsigned grid = (unsigned)std::min<int64_t>(wgs, ceil_div(st.units, kL4Waves >> sp.kslog));
      GPTQ_TRY(launch_l4_decode(d, gs, gated, ch.gather, dim3(grid, (unsigned)ttiles), ch.lds, stream));
      continue;
    }
    L4GemmArgs g;
    g.Xp = Xp;
    g.sums = xs;
    g.params = st.params;
    g.codes = st.codes;
    g.part = reinterpret_cast<float*>(w + p.part_off);
    g.n128 = L.n128;
    g.kc = L.kc;
    g.Gp = L.Gp;
    g.mt = L.mt;
    g.m = c.m;
    g.tokens = tk;
    g.tpad = p.tpad;
    g.tblocks = (uint32_t)sh.tblocks;
    g.pmul = st.pmul;
    g.whole = (uint32_t)sh.whole;
    g.parted = (uint32_t)(sh.tblocks * sh.rblocks - sh.whole);
    g.splits = sh.splits;
    g.chunks = sh.chunks;
    g.ep = ep;
    GPTQ_TRY(launch_l4_gemm(g, sh, gs, gated, stream));
  }
  return GPTQ_OK;
}

}  // namespace gptq
