// Causal attention over whole prompts of different lengths, packed one after the
// other: Y_i = Σ_{j <= i} softmax_j(scale·Q_i·K_j)·V_j within each sequence,
// `heads / kv_heads` query heads to a key head.
#include "attention.hpp"

namespace gptq {
namespace {

#define INLINE __attribute__((always_inline))

constexpr int kWaves = 4, kThreads = 64 * kWaves;
// Queries of a workgroup: 32 a wave, or 32 for the KH waves that take a part of a
// tile's keys each.
template <int KH>
constexpr int kBM = 32 * kWaves / KH;
constexpr int kBN = 64;            // keys of a tile
constexpr float kNone = -3e38f;

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4i16_t;
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ float half_max(float x) {   // with lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Tiles in LDS are rows of D bf16 in pieces of 16 bytes; piece c of row t lies at
// c ^ swz(t), so that 16 rows' reads of one piece (keys) and 8 rows' reads of
// four pieces (values, transposed) each meet every bank equally often.
template <int D>
__device__ __forceinline__ int swz(int t) {
  return D == 128 ? ((t & 3) << 2 | (t >> 2 & 3)) : ((t >> 1 & 1) << 2 | (t >> 2 & 3));
}
template <int D>
__device__ __forceinline__ int lds_at(int t, int c) {   // in bytes
  return t * (D * 2) + (c ^ swz<D>(t)) * 16;
}

struct Prompt {
  HeadRows Q, K, V, Y;
  const int32_t* cu;
  int64_t batch, tokens, tiles;
  int64_t fold;     // tiles of each head that go from the last to the first; those after them the other way
  int kv_heads, share;
  float scale;      // times log2(e), positive: a masked logit times it stays -Inf
  uint32_t keep, flip;   // Q's bits and signs: a scale of 0 clears it, a negative one flips it
};

// Sᵀ = K·Qᵀ and Oᵀ = Vᵀ·Pᵀ: a lane then holds weights of one query, 32 of a tile's
// 64 keys, and they are the second product's operand as they stand; a wave keeps
// its 32 queries and their results in registers, and keys and values come through
// LDS once for the four waves.  One pass with a running maximum; weights are
// rounded to bf16 (2^-8 of each, as the result is), their sum is of the unrounded.  In two
// parts 2048 tokens of 32 heads would take 68 us instead of 52, 6 x 4000 of 64 heads 2201
// instead of 1557, for an error against 64 bits of 0.0016 instead of 0.0018 to 0.0021, of
// which 0.0016 is the result's rounding.
//   Long prompts are bound by issue.  6 of up to 8192 tokens, 64 heads on 8: 2.38 ms, 1.05
// PFLOP/s, 68% of a large product of the library; the matrix cores are busy 59% of the cycles
// (75% in that product), the vector unit 51%, and waves wait 42% of theirs for an
// instruction to issue: the two of a SIMD put no more products beside weights.  Power takes
// its part: the clock under these counters was 1.57 GHz, 1.71 in that product, 2.43 in decoding.
//   One prompt is bound by its longest workgroup: 2048 tokens of 32 heads 49 us, of
// one head 38 where a wave takes all keys, 32 tiles in a row, and 28 where it takes half.
//   Heads of 64 run three waves a SIMD, where the rarely taken second pass spills:
// 23 prompts of 200 tokens 14.3 us, two waves 16.7; 8192 tokens of 32 heads 293 and 317;
// 2048 31 and 34.
template <int D, bool VEC, int KH>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void prompt_attention_kernel(Prompt a) {
  constexpr int KS = D / 16, DT = D / 32, CH = D / 8, TB = kBN * D * 2, BM = kBM<KH>, U = 2 / KH;   // U: 32 keys each
  // Keys and values of a tile and of the next.  Two objects: the compiler makes a
  // read wait for every copy in flight that may go to the object it reads.
  __shared__ __attribute__((aligned(16))) uint8_t lds0[2 * TB], lds1[2 * TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int n32 = lane & 31, half = lane >> 5;
  const int part = KH == 2 ? wave & 1 : 0;   // of a tile's keys

  // Workgroup i runs on XCD i % 8.  The heads that share a key head stay together
  // on one, which then reads those keys from its own L2; tiles with the most keys
  // go first, so that the last workgroups to start are the shortest.  Where all run at
  // once, two a CU, the second half goes the other way: the longest share a CU with the
  // shortest (2 x 900 tokens of 32 heads 32.1 us instead of 35.8, 2048 52.4 instead of 52.9).
  const int64_t slot = blockIdx.x >> 3, group = slot / a.share * 8 + (blockIdx.x & 7);
  const int64_t kvh = group % a.kv_heads, head = kvh * a.share + slot % a.share;
  if (group >= a.tiles * a.kv_heads) return;
  int64_t b = 0, at = 0, row0 = 0;
  int from, len = 0;
  auto count = [&](int64_t i) {   // tiles of sequence i
    const int64_t r0 = a.cu[i], r1 = a.cu[i + 1];
    row0 = r0 < 0 ? 0 : r0 > a.tokens ? a.tokens : r0;
    const int64_t past = r1 > a.tokens ? a.tokens : r1;
    len = past > row0 ? (int)(past - row0) : 0;
    return (int64_t)((len + BM - 1) / BM);
  };
  const int64_t rank = group / a.kv_heads;
  if (!ragged_find(rank < a.fold ? a.tiles - 1 - rank : rank - a.fold, a.batch, count, &b, &at, &from)) return;
  row0 = lane_value(row0, from);
  len = __builtin_amdgcn_readlane(len, from);
  const int q0 = (int)at * BM, w0 = q0 + wave / KH * 32;   // the workgroup's and the wave's first query
  const int iq = w0 + n32;                             // the lane's query
  const int keys = std::min(len, q0 + BM);            // that any of its queries sees
  const int tiles = (keys + kBN - 1) / kBN;

  const uint16_t* Kp = static_cast<const uint16_t*>(a.K.p) + row0 * a.K.ld + kvh * a.K.hs;
  const uint16_t* Vp = static_cast<const uint16_t*>(a.V.p) + row0 * a.V.ld + kvh * a.V.hs;

  bf16x8_t qf[KS];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.Q.p) + (row0 + std::min(iq, len - 1)) * a.Q.ld + head * a.Q.hs + half * 8;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4_t x;
      if (VEC) {
        x = *reinterpret_cast<const u32x4_t*>(qp + ks * 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = qp[ks * 16 + 2 * i] | (uint32_t)qp[ks * 16 + 2 * i + 1] << 16;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (x[i] & a.keep) ^ a.flip;
      qf[ks] = __builtin_bit_cast(bf16x8_t, x);
    }
  }

  // A tile's rows into LDS, straight from memory (descriptor bounds: rows past the
  // last key read as zeros).  Piece i·256 + tid of a tile is row i·(256 / CH) +
  // tid / CH, whose pieces lie as those of row tid / CH do: one address a lane.
  const int t0 = tid / CH, c0 = (tid % CH ^ swz<D>(t0)) * 8;
  const int kvoff = (int)(t0 * a.K.ld + c0) * 2, vvoff = (int)(t0 * a.V.ld + c0) * 2;
  auto fetch = [&](int tile, uint8_t* buf) {
    constexpr int kRows = kThreads / CH;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t ld = v ? a.V.ld : a.K.ld;
      const uint16_t* X = (v ? Vp : Kp) + (int64_t)tile * kBN * ld;
      if (VEC) {
        const int64_t left = ((int64_t)(keys - 1 - tile * kBN) * ld + D) * 2;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(X), 0, (int)std::min<int64_t>(left, 0x7fffffff), 0x00020000);
#pragma unroll
        for (int i = 0; i < kBN / kRows; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(buf + v * TB + (i * kThreads + wave * 64) * 16), 16,
                                                   v ? vvoff : kvoff, (int)(i * kRows * ld * 2), 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < kBN / kRows; ++i) {
          const int t = i * kRows + t0;
          const bool there = tile * kBN + t < keys;
          u32x4_t x;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = there ? X[t * ld + c0 + 2 * j] | (uint32_t)X[t * ld + c0 + 2 * j + 1] << 16 : 0;
          *reinterpret_cast<u32x4_t*>(buf + v * TB + (i * kThreads + tid) * 16) = x;
        }
      }
    }
  };

  // Where the lane's operands lie in a buffer: keys (row n32, pieces 2·ks + half)
  // and values (transposed reads: four rows of a column at vlo, four at vhi).
  // Whole offsets: behind a longer chain of sums the compiler loses sight of which
  // buffer a read is of.
  int kat[KS], vlo[DT], vhi[DT];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) kat[ks] = lds_at<D>(n32, ks * 2 + half) + part * 32 * D * 2;   // 32 rows further: the same swizzle
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int t = part * 32 + half * 4 + (lane >> 2 & 3), c = d * 32 + (lane >> 4 & 1) * 16 + (lane & 3) * 4;
    vlo[d] = lds_at<D>(t, c >> 3) + (c & 7) * 2;
    vhi[d] = lds_at<D>(t + 8, c >> 3) + (c & 7) * 2;
  }

  f32x16_t o[DT];
  float m, l, by;   // weights are 2^(logit·by - m)
  // A maximum with a rest lies here while the wave has one: its logits are then taken
  // relative to it before their weights, and m is 0, by 1.  (In registers, heads of 64
  // reloaded one a tile, behind the copies in flight: 98 -> 117 us for 8192 tokens of 8.)
  __shared__ float far_m[kThreads], far_rest[kThreads];
  uint64_t far;     // lanes with a rest
  // A masked value meets a weight of 0, and 0·Inf is NaN.  Such values can only
  // be in the last tiles; a result that is not finite is computed once more,
  // carefully: what is not finite is left out of the product there, and counted
  // for the queries that see it.
  auto pass = [&](auto mode) {
    constexpr bool careful = decltype(mode)::value;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
    m = kNone;
    l = 0.f;
    by = a.scale;
    far = 0;
    fetch(0, lds0);
    auto step = [&](int tile, uint8_t* cur, uint8_t* nxt) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0): this wave's copies have landed
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (tile + 1 < tiles) fetch(tile + 1, nxt);
      const int k0 = tile * kBN + part * 32;   // the wave's first key
      if (k0 > w0 + 31) return;   // the wave's queries see none of it (no barrier is skipped)
      f32x16_t s[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[u][r] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int u = 0; u < U; ++u) {   // two sums by turns: a product need not wait for the one before
          const bf16x8_t k = *reinterpret_cast<const bf16x8_t*>(cur + (kat[ks] + u * 32 * D * 2));
          s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, qf[ks], s[u], 0, 0, 0);
        }
      constexpr int kAhead = U * KS < 8 ? U * KS : 8;
      __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);   // operands are read eight products ahead
#pragma unroll
      for (int i = 0; i < U * KS - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
      const bool edge = k0 + 32 * U > w0 + 1;   // some query does not see some key
      if (edge) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (k0 + u * 32 + 8 * (r >> 2) + 4 * half + (r & 3) > iq) s[u][r] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int r = 1; r < 16 * U; ++r) top = fmaxf(top, s[r >> 4][r & 15]);
      top = half_max(top);
      if (far | __ballot(fmaf(top, a.scale, -m) > 8.f)) {   // sums are scaled again only when the maximum grows by more than 2^8
        float rest = 0.f;
        if (__builtin_expect(far != 0, 0)) m = far_m[tid], rest = far_rest[tid];
        const float f = raise_to(top, a.scale, &m, &rest);
        far = __ballot(rest != 0.f);
        by = a.scale;
        if (__builtin_expect(far != 0, 0)) {
          far_m[tid] = m;
          far_rest[tid] = rest;
#pragma unroll
          for (int r = 0; r < 16 * U; ++r) s[r >> 4][r & 15] = fmaf(s[r >> 4][r & 15], a.scale, -m) - rest;
          m = 0.f;
          by = 1.f;
        }
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= f;
      }
      bf16x8_t p[2 * U];
#pragma unroll
      for (int r = 0; r < 16 * U; ++r) {
        const float e = __builtin_amdgcn_exp2f(fmaf(s[r >> 4][r & 15], by, -m));
        l += e;
        p[r >> 3][r & 7] = (__bf16)e;
      }
      auto columns = [&](int d, int kk) INLINE {   // 16 rows further: the same swizzle
        const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(cur + (vlo[d] + (TB + kk * 16 * D * 2))));
        const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(cur + (vhi[d] + (TB + kk * 16 * D * 2))));
        const auto both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8_t, both);
      };
      if constexpr (!careful) {
#pragma unroll
        for (int kk = 0; kk < 2 * U; ++kk)
#pragma unroll
          for (int d = 0; d < DT; ++d)
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(columns(d, kk), p[kk], o[d], 0, 0, 0);
      } else {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x16_t more, less;   // counts
#pragma unroll
          for (int r = 0; r < 16; ++r) more[r] = less[r] = 0.f;
#pragma unroll
          for (int kk = 0; kk < 2 * U; ++kk) {
            bf16x8_t v = columns(d, kk);
            if (edge) {
              bf16x8_t up, down, seen;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x = (float)v[e];
                const bool odd = !(fabsf(x) < INFINITY);
                up[e] = (__bf16)(odd && !(x < 0.f) ? 1.f : 0.f);
                down[e] = (__bf16)(odd && !(x > 0.f) ? 1.f : 0.f);
                v[e] = odd ? (__bf16)0.f : v[e];
                const int key = k0 + kk * 16 + (e >> 2) * 8 + half * 4 + (e & 3);
                seen[e] = (__bf16)(key <= iq ? 1.f : 0.f);
              }
              more = __builtin_amdgcn_mfma_f32_32x32x16_bf16(up, seen, more, 0, 0, 0);
              less = __builtin_amdgcn_mfma_f32_32x32x16_bf16(down, seen, less, 0, 0, 0);
            }
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[kk], o[d], 0, 0, 0);
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] += (more[r] > 0.f ? INFINITY : 0.f) + (less[r] > 0.f ? -INFINITY : 0.f);
        }
      }
    };
    for (int tile = 0; tile < tiles; tile += 2) {
      step(tile, lds0, lds1);
      if (tile + 1 < tiles) step(tile + 1, lds1, lds0);
    }
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) sum += o[d][r] * 0.f;   // NaN if any is not finite
    return __syncthreads_or(iq < len && sum != sum);
  };
  if (pass(std::false_type{})) pass(std::true_type{});

  l = half_sum(l);
  if constexpr (KH == 2) {   // the odd wave's sums to the even one, by way of LDS
    // [DT][4][64 lanes] pieces of 16 bytes for each two waves, then maxima and sums
    static_assert(DT * 4 * 64 * 16 <= 2 * TB && kWaves == 4, "");
    uint8_t* mine = wave < 2 ? lds0 : lds1;
    __shared__ float om[2][64], orest[2][64], ol[2][64];
    float rest = 0.f;
    if (far) m = far_m[tid], rest = far_rest[tid];
    __syncthreads();
    if (part) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<f32x4_t*>(mine + ((d * 4 + r) * 64 + lane) * 16) =
              f32x4_t{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
      om[wave >> 1][lane] = m;
      orest[wave >> 1][lane] = rest;
      ol[wave >> 1][lane] = l;
    }
    __syncthreads();
    if (part) return;
    const float m1 = om[wave >> 1][lane], rest1 = orest[wave >> 1][lane], more = (m1 - m) + (rest1 - rest);
    const float f0 = more > 0.f ? exp2f(-more) : 1.f, f1 = more > 0.f ? 1.f : exp2f(more);   // NaN: an infinite logit was seen
    l = l * f0 + ol[wave >> 1][lane] * f1;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x4_t other = *reinterpret_cast<const f32x4_t*>(mine + ((d * 4 + r) * 64 + lane) * 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[d][4 * r + c] = o[d][4 * r + c] * f0 + other[c] * f1;
      }
  }
  if (iq < len) {
    const float inv = 1.f / l;
    uint16_t* yp = const_cast<uint16_t*>(static_cast<const uint16_t*>(a.Y.p)) + (row0 + iq) * a.Y.ld + head * a.Y.hs + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint16_t h[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) h[c] = __builtin_bit_cast(uint16_t, (__bf16)(o[d][r * 4 + c] * inv));
        if (VEC) {
          *reinterpret_cast<u32x2_t*>(yp + d * 32 + r * 8) = u32x2_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) yp[d * 32 + r * 8 + c] = h[c];
        }
      }
  }
}

template <int KH>
gptq_status launch(const PromptCall& c, hipStream_t stream) {
  constexpr int BM = kBM<KH>;
  const int64_t tiles = (c.tokens + (BM - 1) * std::min(c.batch, c.tokens)) / BM;   // n tokens take at most (n + BM - 1) / BM
  Prompt a{c.Q, c.K, c.V, c.Y, c.cu, c.batch, c.tokens, tiles, tiles * c.heads <= 512 ? 256 / c.heads : tiles, c.kv_heads, c.heads / c.kv_heads,
           c.scale == 0.f ? 1.f : fabsf(c.scale) * 1.44269504088896340736f, c.scale == 0.f ? 0u : ~0u,
           c.scale < 0.f ? 0x80008000u : 0u};
  const unsigned grid = (unsigned)(ceil_div(tiles * c.kv_heads, 8) * 8 * (c.heads / c.kv_heads));
  const int64_t most = int64_t(1) << 23;   // a tile's rows are 32-bit offsets apart
  const bool vec = c.Q.vec && c.K.vec && c.V.vec && c.Y.vec && c.K.ld < most && c.V.ld < most;
  if (c.dim == 128)
    vec ? prompt_attention_kernel<128, true, KH><<<grid, kThreads, 0, stream>>>(a)
        : prompt_attention_kernel<128, false, KH><<<grid, kThreads, 0, stream>>>(a);
  else
    vec ? prompt_attention_kernel<64, true, KH><<<grid, kThreads, 0, stream>>>(a)
        : prompt_attention_kernel<64, false, KH><<<grid, kThreads, 0, stream>>>(a);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

// Two waves share 32 queries, each with half of every tile's keys, where workgroups
// of 128 queries leave CUs idle: their chain of tiles is what is waited for.  us
// (shared / not): 8 heads of 128, 2048 tokens (128 workgroups of 128) 30 / 40, 4096
// (256) 59 / 74, 8192 (512) 164 / 161; 32 heads, 500 tokens 12.5 / 15.5, 2048 (512) 54 /
// 50; 8 heads of 64, 8192 (512) 89 / 107, but 16 (1024) 170 / 162 and 23 prompts of 200, 14
// heads (812) 16.8 / 13.6.  Prompts of one tile have nothing to share: 64 tokens 7.5 / 6.8.
gptq_status run_prompt_attention(const PromptCall& c, hipStream_t stream) {
  const int64_t wgs = (c.tokens + 127 * std::min(c.batch, c.tokens)) / 128 * c.heads;
  return wgs <= (c.dim == 64 ? 512 : 256) && c.tokens > kBN * c.batch ? launch<2>(c, stream) : launch<1>(c, stream);
}

}  // namespace gptq
