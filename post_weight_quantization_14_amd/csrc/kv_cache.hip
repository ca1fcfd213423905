// Keys and values quantized to 4 bits as they are written to a paged cache, and
// read back (layout: attention.hpp).
//
// The grid of a group x of 32, 64 or 128 neighbouring channels of one token and
// head, with lo = min x, hi = max x, a = max |x|:
//   s = the smallest bf16 with 15·s >= hi - lo, 4096·s >= a and s >= 2^-100,
//   z = -rint(lo/s),  q = clamp(rint(x/s) + z, 0, 15),  x̂ = (q - z)·s.
// Rounding s up lets 15 steps span the group, so |x - x̂| <= s/2 for every x;
// the bound by a keeps |z| <= 4096 and |x/s| <= 4096, so that z fits 16 bits,
// x̂ has at most 21 significant bits (exact in fp32), and a constant group reads
// back to 2^-13 of its value.  A group that holds NaN, Inf or a magnitude above
// 2^64 gets s = NaN: it reads back as NaN.
#include "attention.hpp"

namespace gptq {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- grid
struct Grid {
  float s, inv;
};

// Both decisions that decide a code are made exactly.  s here: the guess (a little
// low, then cut to bf16 from above) is the wanted bf16 or the one below it, and
// 64-bit arithmetic tells which: 15·s and 4096·s are exact and have 12 bits, so hi - lo,
// rounded once to 53, compares with 15·s as it would unrounded unless it is rounded to it
// (15 and a negative 2^-60): there the rounding error's sign tells.
__device__ __forceinline__ Grid make_grid(float lo, float hi, uint32_t top) {
  Grid g;
  const float a = __uint_as_float(top);
  const float want = fmaxf(fmaxf((hi - lo) * (1.f / 15.f), a * 0x1p-12f) * (1.f - 0x1p-20f), 0x1p-100f);
  uint32_t bits = (__float_as_uint(want) + 0xffffu) & 0xffff0000u;
  const double range = (double)hi - (double)lo;
  const double sd = (double)__uint_as_float(bits);
  bool low = sd * 15. < range || sd * 4096. < (double)a;
  if (sd * 15. == range) {   // exact: of two terms' sum the error is a sum of what each lost
    const double back = range - hi;
    low |= (hi - (range - back)) - (lo + back) > 0.;
  }
  if (low) bits += 0x10000u;
  if (!(top <= 0x5f800000u)) bits = 0x7fc00000u;   // 2^64; NaN and Inf have larger bits
  g.s = __uint_as_float(bits);
  g.inv = __builtin_amdgcn_rcpf(g.s);
  return g;
}

// rint(x/s), ties to even, plus 0x4b400000 (NaN: anything).  |x/s| <= 4096, and
// x·inv is off by at most 2 units of 2^-23.
//   bf16 x: one correction by the remainder.  At a tie x/s is representable, so the
// remainder is exact and the corrected quotient is the tie itself; off a tie x/s is
// at least 2^-9 (of 1 or of itself) away from it, as x and s have eight bits, and the
// error is below 2^-11.  Adding 1.5·2^23 rounds to an integer, in the low bits.
__device__ __forceinline__ uint32_t steps(float x, const Grid& g, uint16_t) {
  const float q = x * g.inv;
  return __float_as_uint(fmaf(fmaf(-q, g.s, x), g.inv, q) + 12582912.f);
}
//   fp32 x: the integer next to x·inv is the nearest of x/s or, near a tie, its
// neighbour; the remainder x - r·s (exact by one fused step: r·s has 21 bits and
// x lies within a factor of two of it, or r is 0) tells.
__device__ __forceinline__ uint32_t steps(float x, const Grid& g, float) {
  float r = rintf(x * g.inv);
  const float t = fmaf(-r, g.s, x), half = 0.5f * g.s;
  const bool odd = (int)r & 1;
  if (t > half || (t == half && odd)) r += 1.f;
  if (t < -half || (t == -half && odd)) r -= 1.f;
  return __float_as_uint(r + 12582912.f);
}

// with the lanes that share a group (4, 8 or 16 neighbours), by DPP: quads, then
// halves of rows and rows mirrored, whose lanes agree within quads by then
template <int N, class F>
__device__ __forceinline__ uint32_t among(uint32_t x, const F& f) {
  x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xb1, 0xf, 0xf, true));
  x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4e, 0xf, 0xf, true));
  if constexpr (N > 4) x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xf, 0xf, true));
  if constexpr (N > 8) x = f(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xf, 0xf, true));
  return x;
}

template <int D, int G>
struct Rec {
  static constexpr int kWords = kv_rec_bytes(D, G) / 4, kCodeWords = kv_code_bytes(D) / 4;
  static constexpr int kParams = kv_param_bytes(D, G) / 4, kChunks = D / 8, kNg = D / G;
  // where byte b (0 .. 3) of chunk j's value codes lies, in bytes from the record's start
  static __device__ __forceinline__ int value_byte(int t, int j, int b) {
    constexpr int U = D / 32;   // bytes of a unit
    return kCodeWords * 4 + (((t >> 2) * 16 + (j & 3) * 4 + b) * 4 + (t & 3)) * U + (j >> 2);
  }
  // the word of chunk j's key codes
  static __device__ __forceinline__ int key_word(int t, int j) { return ((j & 3) * 16 + t) * (D / 32) + (j >> 2); }
  static __device__ __forceinline__ int param_word(int v, int t, int g) {
    return 2 * kCodeWords + v * kParams + g * kKvRec + t;
  }
  // the position (of 16) that record word w belongs to; value words of D = 64 hold two: the first
  static __device__ __forceinline__ int position(int w) {
    if (w < kCodeWords) return w / (D / 32) % 16;
    if (w < 2 * kCodeWords) {
      w -= kCodeWords;
      return D == 128 ? (w >> 6) * 4 + (w & 3) : (w >> 5) * 4 + (w & 1) * 2;
    }
    return (w - 2 * kCodeWords) % kKvRec;
  }
};

// eight neighbouring channels, as they lie in memory and as numbers
template <class T>
struct Eight {
  u32x4_t w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const u32x4_t*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4)
          w[i / 4][i % 4] = __float_as_uint(p[i]);
        else
          w[0][i / 2] = (i & 1 ? w[0][i / 2] : 0u) | (uint32_t)p[i] << (16 * (i & 1));
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i / 4][i % 4]);
    else
      return __uint_as_float(i & 1 ? w[0][i / 2] & 0xffff0000u : w[0][i / 2] << 16);
  }
};

// A sequence whose tokens all have a position: one with fewer positions than
// tokens is out of range here.
__device__ __forceinline__ KvSeq written_seq(const KvSeqs& q, const KvLayout& L, int64_t b) {
  KvSeq s = kv_seq(q, b, std::min<int64_t>(q.width * L.recs * kKvRec, kKvMost));
  if (s.n > s.len) {
    s.bad = true;
    s.len = s.n;
  }
  return s;
}

// The 16-position blocks that sequence s's tokens touch.
__device__ __forceinline__ int64_t blocks_of(const KvSeq& s) {
  return s.n > 0 ? (s.len - 1) / kKvRec - (s.len - s.n) / kKvRec + 1 : 0;
}

struct Block {
  int64_t b;
  KvSeq s;
  int blk;        // of 16 positions, from the sequence's start
  int p0, p1;     // the positions of it that the call's tokens hold
  int64_t page;   // or -1
};

// Block blockIdx.x of the batch's; false past the last.  Whole waves.
__device__ __forceinline__ bool find_block(const KvSeqs& q, const KvLayout& L, Block* k) {
  int64_t at = 0;
  if (q.cu == nullptr) {   // one token each: block = sequence
    k->b = blockIdx.x;
    if (k->b >= q.batch) return false;
    k->s = uniform(written_seq(q, L, k->b));
  } else {
    KvSeq mine;
    int l;
    auto count = [&](int64_t b) {
      mine = written_seq(q, L, b);
      return blocks_of(mine);
    };
    if (!ragged_find(blockIdx.x, q.batch, count, &k->b, &at, &l)) return false;
    k->s = lane_value(mine, l);
  }
  const int first = k->s.len - k->s.n;
  k->blk = first / kKvRec + (int)at;
  k->p0 = std::max(first, k->blk * kKvRec);
  k->p1 = std::min(k->s.len, (k->blk + 1) * kKvRec);
  k->page = -1;
  if (k->s.bad) return true;
  const int64_t page = q.table[k->b * q.stride + (k->blk >> L.rec_shift)];
  if (page >= 0 && page < q.pages) k->page = page;
  return true;
}

// A sequence with something out of range may have no block to say so: the first
// workgroups look at the batch.
__device__ __forceinline__ void report(const KvSeqs& q, const KvLayout& L) {
  for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < q.batch; b += (int64_t)gridDim.x * kThreads)
    if (written_seq(q, L, b).bad) kv_bad(q.status);
}

// ---------------------------------------------------------------- append
// One workgroup per record (16 positions of one head): a thread quantizes eight
// neighbouring channels (16 bytes of bf16) of a token, lanes of a group share
// their extremes by swaps, the codes are put in order in LDS and leave in whole
// rows.  Bound by memory for prompts (2 bytes in, 0.56 out per value): 8 of 2048
// tokens, 8 heads of 128, groups of 64 (86 MB) 22.5 us, 3.8 TB/s, from fp32 (153 MB) 34.6,
// 4.4 TB/s; by launch and three dependent loads (sequence, page, tokens) for a decode step:
// 16 sequences of 32 heads 5.3 us.
template <int D, int G, class T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvLayout L, HeadRows K, HeadRows V, KvSeqs q,
                                                             uint8_t* __restrict__ pages) {
  using R = Rec<D, G>;
  __shared__ __attribute__((aligned(16))) uint32_t recs[2][R::kWords];   // of this head and, while it leaves, of the next
  const int tid = threadIdx.x;
  if (blockIdx.y == 0 && q.status) report(q, L);
  Block k;
  if (!find_block(q, L, &k)) return;
  constexpr int kItems = 2 * kKvRec * R::kChunks / kThreads, kLanes = G / 8;
  const T* src[kItems];
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int it = n * kThreads + tid, v = it / (kKvRec * R::kChunks), t = it / R::kChunks % kKvRec, j = it % R::kChunks;
    // positions that are not the call's: its nearest token once more, not written
    const int p = min(max(k.blk * kKvRec + t, k.p0), k.p1 - 1);
    const HeadRows& X = v ? V : K;
    src[n] = static_cast<const T*>(X.p) + (k.s.row + (p - (k.s.len - k.s.n))) * X.ld + j * 8;
  }
  Eight<T> raw[kItems], ahead[kItems];
  auto load = [&](int head, Eight<T> (&x)[kItems]) {   // all in flight at once, a head ahead
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const HeadRows& X = n * kThreads + tid < kKvRec * R::kChunks ? K : V;
      x[n].load(src[n] + head * X.hs, X.vec);
    }
  };
  load(blockIdx.y, ahead);
  if (k.page < 0) {
    if (tid == 0) kv_bad(q.status);
    return;
  }
  for (int head = blockIdx.y, turn = 0; head < L.heads; head += gridDim.y, ++turn) {
    uint32_t* rec = recs[turn & 1];
#pragma unroll
    for (int n = 0; n < kItems; ++n) raw[n] = ahead[n];
    if (head + (int)gridDim.y < L.heads) load(head + gridDim.y, ahead);
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int it = n * kThreads + tid, v = it / (kKvRec * R::kChunks), t = it / R::kChunks % kKvRec, j = it % R::kChunks;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = raw[n].at(i);
      float lo = x[0], hi = x[0];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        top = std::max(top, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      auto f32 = [](uint32_t u) { return __uint_as_float(u); };
      lo = f32(among<kLanes>(__float_as_uint(lo), [&](uint32_t a, uint32_t b) { return __float_as_uint(fminf(f32(a), f32(b))); }));
      hi = f32(among<kLanes>(__float_as_uint(hi), [&](uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(f32(a), f32(b))); }));
      top = among<kLanes>(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const Grid g = make_grid(lo, hi, top);
      const bool nan = g.s != g.s;
      const int z = nan ? 0 : 0x4b400000 - (int)steps(lo, g, T{}), shift = z - 0x4b400000;
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = std::min(std::max((int)steps(x[i], g, T{}) + shift, 0), 15);   // NaN: any code
      if (v == 0) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (uint32_t)c[i] << (4 * (4 * (i & 1) + (i >> 1)));
        rec[R::key_word(t, j)] = w;
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          reinterpret_cast<uint8_t*>(rec)[R::value_byte(t, j, b)] = (uint8_t)(c[2 * b] | c[2 * b + 1] << 4);
      }
      if (j % kLanes == 0)
        rec[R::param_word(v, t, j / kLanes)] = __float_as_uint(g.s) | (uint32_t)(uint16_t)(int16_t)z;
    }
    __syncthreads();
    uint8_t* out = pages + (k.page * L.heads + head) * L.recs * (int64_t)(R::kWords * 4) +
                   (int64_t)(k.blk & (L.recs - 1)) * (R::kWords * 4);
    if (k.p1 - k.p0 == kKvRec) {
      for (int w = tid; w < R::kWords / 4; w += kThreads)
        reinterpret_cast<u32x4_t*>(out)[w] = reinterpret_cast<const u32x4_t*>(rec)[w];
      continue;
    }
    const int t0 = k.p0 - k.blk * kKvRec, t1 = k.p1 - k.blk * kKvRec;
    for (int w = tid; w < R::kWords; w += kThreads) {
      const int t = R::position(w);
      const bool first = t >= t0 && t < t1;
      if (D == 64 && w >= R::kCodeWords && w < 2 * R::kCodeWords) {   // two positions, 16 bits each
        const bool second = t + 1 >= t0 && t + 1 < t1;
        if (first) reinterpret_cast<uint16_t*>(out)[2 * w] = (uint16_t)rec[w];
        if (second) reinterpret_cast<uint16_t*>(out)[2 * w + 1] = (uint16_t)(rec[w] >> 16);
      } else if (first) {
        reinterpret_cast<uint32_t*>(out)[w] = rec[w];
      }
    }
  }
}

// ---------------------------------------------------------------- read
// The same records and threads the other way: whole rows to LDS, a thread makes
// eight channels of a token, (c - z)·s exactly.  Bound by memory: 8 prompts
// of 2048 tokens, 8 heads of 128, groups of 64 (86 MB) 16.7 us, 5.1 TB/s, part of it from
// the last cache; to fp32 (153 MB) 43 us, 3.5 TB/s, four bytes of five written.
template <int D, int G, class T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvLayout L, HeadRows K, HeadRows V, KvSeqs q,
                                                           const uint8_t* __restrict__ pages) {
  using R = Rec<D, G>;
  __shared__ __attribute__((aligned(16))) uint32_t recs[2][R::kWords];
  const int tid = threadIdx.x;
  if (blockIdx.y == 0 && q.status) report(q, L);
  Block k;
  if (!find_block(q, L, &k)) return;
  if (k.page < 0 && tid == 0) kv_bad(q.status);
  constexpr bool kTwice = R::kWords / 4 > kThreads;   // whether a record is more than a piece of 16 bytes a thread
  static_assert(R::kWords / 4 <= 2 * kThreads, "");
  u32x4_t ahead = {}, more = {};
  auto load = [&](int head) {   // a head ahead
    const u32x4_t* in = reinterpret_cast<const u32x4_t*>(
        pages + ((k.page < 0 ? 0 : k.page) * L.heads + head) * L.recs * (int64_t)(R::kWords * 4) +
        (int64_t)(k.blk & (L.recs - 1)) * (R::kWords * 4));
    if (tid < R::kWords / 4) ahead = in[tid];
    if (kTwice && tid + kThreads < R::kWords / 4) more = in[tid + kThreads];
  };
  load(blockIdx.y);
  for (int head = blockIdx.y, turn = 0; head < L.heads; head += gridDim.y, ++turn) {
    uint32_t* rec = recs[turn & 1];
    if (tid < R::kWords / 4) reinterpret_cast<u32x4_t*>(rec)[tid] = ahead;
    if (kTwice && tid + kThreads < R::kWords / 4) reinterpret_cast<u32x4_t*>(rec)[tid + kThreads] = more;
    if (head + (int)gridDim.y < L.heads) load(head + gridDim.y);
    __syncthreads();
    constexpr int kItems = 2 * kKvRec * R::kChunks;
#pragma unroll
    for (int it = tid; it < kItems; it += kThreads) {
      const int v = it / (kKvRec * R::kChunks), t = it / R::kChunks % kKvRec, j = it % R::kChunks;
      const int p = k.blk * kKvRec + t;
      if (p < k.p0 || p >= k.p1) continue;
      const uint32_t pw = k.page < 0 ? 0x7fc00000u : rec[R::param_word(v, t, j * 8 / G)];
      const float s = __uint_as_float(pw & 0xffff0000u);
      const int z = (int16_t)(uint16_t)pw;
      float x[8];
      if (v == 0) {
        const uint32_t w = rec[R::key_word(t, j)];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)((int)(w >> (4 * (4 * (i & 1) + (i >> 1))) & 15) - z) * s;
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int w = reinterpret_cast<const uint8_t*>(rec)[R::value_byte(t, j, b)];
          x[2 * b] = (float)((w & 15) - z) * s;
          x[2 * b + 1] = (float)((w >> 4) - z) * s;
        }
      }
      const HeadRows& X = v ? V : K;
      const int64_t row = k.s.row + (p - (k.s.len - k.s.n));
      T* out = const_cast<T*>(static_cast<const T*>(X.p)) + row * X.ld + head * X.hs + j * 8;
      if constexpr (sizeof(T) == 4) {
        if (X.vec) {
          reinterpret_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
          reinterpret_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] = x[i];
        }
      } else {
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
        if (X.vec) {
          u32x4_t o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
          *reinterpret_cast<u32x4_t*>(out) = o;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) out[i] = h[i];
        }
      }
    }
  }
}

// Blocks of 16 positions that the tokens can touch: n tokens touch at most (n + 30) / 16.
int64_t most_blocks(const KvSeqs& q) { return q.cu ? (q.tokens + 30 * std::min(q.batch, q.tokens)) / 16 : q.batch; }

// The heads are shared by as many workgroups as fill the card (8 a CU); each takes
// every so manieth head of its 16 positions, whose place it finds once (8 prompts of
// 2048 written and read 39.2 us; 41.7 with twice as many, 49.1 with one for each head).
dim3 grid_of(const KvLayout& L, const KvSeqs& q) {
  const int64_t blocks = most_blocks(q);
  return dim3((unsigned)blocks, (unsigned)std::min<int64_t>(L.heads, ceil_div(2048, blocks)));
}

template <class F>
gptq_status by_shape(const KvLayout& L, int dtype, const F& f) {
  auto typed = [&](auto d, auto g) { return dtype == GPTQ_FP32 ? f(d, g, float{}) : f(d, g, uint16_t{}); };
  using std::integral_constant;
  if (L.dim == 128 && L.group == 128) return typed(integral_constant<int, 128>{}, integral_constant<int, 128>{});
  if (L.dim == 128 && L.group == 64) return typed(integral_constant<int, 128>{}, integral_constant<int, 64>{});
  if (L.dim == 128) return typed(integral_constant<int, 128>{}, integral_constant<int, 32>{});
  if (L.group == 64) return typed(integral_constant<int, 64>{}, integral_constant<int, 64>{});
  return typed(integral_constant<int, 64>{}, integral_constant<int, 32>{});
}

}  // namespace

gptq_status run_kv_append(const KvLayout& L, const HeadRows& K, const HeadRows& V, int dtype, const KvSeqs& q,
                          void* pages, hipStream_t stream) {
  return by_shape(L, dtype, [&](auto d, auto g, auto t) {
    kv_append_kernel<d.value, g.value, decltype(t)><<<grid_of(L, q), kThreads, 0, stream>>>(
        L, K, V, q, static_cast<uint8_t*>(pages));
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  });
}

gptq_status run_kv_read(const KvLayout& L, const HeadRows& K, const HeadRows& V, int dtype, const KvSeqs& q,
                        const void* pages, hipStream_t stream) {
  return by_shape(L, dtype, [&](auto d, auto g, auto t) {
    kv_read_kernel<d.value, g.value, decltype(t)><<<grid_of(L, q), kThreads, 0, stream>>>(
        L, K, V, q, static_cast<const uint8_t*>(pages));
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  });
}

}  // namespace gptq
