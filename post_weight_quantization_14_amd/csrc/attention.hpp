// Shared by the operators on the 4-bit key/value cache (kv_cache.hip,
// kv_attention.hip), the attention over whole prompts (prompt_attention.hip)
// and their entry points (abi_attention.hip): the cache's layout, the search
// of ragged batches, and the launchers' declarations.
#pragma once

#include <algorithm>

#include "gptq_internal.hpp"

namespace gptq {

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- cache layout
// A page holds page_size positions of every head as records of 16 positions of
// one head, [kv_heads][page_size / 16].  A record is
//   keys'   codes   [4 kg][16 t][D/32 ks]     32-bit words,
//   values' codes   [4 tg][16 i][4 t]         units of D/32 bytes,
//   keys'   params  [D/g][16 t]               words,
//   values' params  [D/g][16 t]               words,
// in the order in which the matrix cores take them: lane 16·kg + t of a wave
// reads its keys' operand (position t, channels 32·ks + 8·kg .. + 7) as one
// piece of D/8 bytes, lane 16·tg + i its values' (positions 4·tg .. + 3,
// channels 32·b + 2i, + 1 for b < D/32) as another, both D/8 bytes past its
// neighbour's, and four positions' params are 16 bytes.
// Every byte belongs to one position (a unit of values is D/32 bytes of one
// position), so a token is written without reading what is beside it.
//   A key word's nibble for channel c of its eight is 4·(c & 1) + c/2: w & 0xF000F
// is then the pair (0, 1), the pairs behind it follow by shifts of 4.
//   Byte b of a value unit holds channels 32·b + 2i (low nibble) and 32·b + 2i + 1.
//   A param word is bf16(s) << 16 | (uint16)z.
constexpr int kKvRec = 16;
constexpr int64_t kKvMost = int64_t(1) << 30;   // positions of a sequence: sums of two stay in 31 bits

struct KvLayout {
  int heads, dim, group, recs;   // recs: records of one head in a page (a power of two)
  int rec_shift;                 // log2(recs)
  int64_t rec_bytes, page_bytes;
};

constexpr __host__ __device__ int kv_code_bytes(int dim) { return kKvRec * dim / 2; }
constexpr __host__ __device__ int kv_param_bytes(int dim, int group) { return dim / group * kKvRec * 4; }
constexpr __host__ __device__ int kv_rec_bytes(int dim, int group) {
  return 2 * (kv_code_bytes(dim) + kv_param_bytes(dim, group));
}

inline KvLayout plan_kv(const gptq_kv_config& c) {
  KvLayout L{c.kv_heads, c.head_dim, c.group_size == -1 ? c.head_dim : c.group_size, c.page_size / kKvRec, 0, 0, 0};
  while ((1 << L.rec_shift) < L.recs) ++L.rec_shift;
  L.rec_bytes = kv_rec_bytes(L.dim, L.group);
  L.page_bytes = L.rec_bytes * L.recs * L.heads;
  return L;
}

// The sequences of a call: sequence b's n = cu[b + 1] - cu[b] tokens (one each
// if cu is NULL) are rows cu[b] .. of the token tensors and the last n of its
// lens[b] positions; position p is in page table[b·stride + p / page_size].
struct KvSeqs {
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* table;
  int64_t batch, tokens;
  int64_t width, stride;   // pages of a sequence that the table holds; its row stride
  int64_t pages;           // pages there are
  int32_t* status;         // or NULL
};

struct KvSeq {
  int64_t row;   // of its first token
  int n;         // tokens of this call
  int len;       // positions in the cache with them
  bool bad;      // something it gives is out of range: len is then n, and no page is read or written
};

// What the device data says of sequence b.  The rows are cut to those there are.
__device__ __forceinline__ KvSeq kv_seq(const KvSeqs& q, int64_t b, int64_t capacity) {
  KvSeq s;
  int64_t r0 = b, r1 = b + 1;
  if (q.cu) {
    r0 = q.cu[b];
    r1 = q.cu[b + 1];
  }
  const int64_t len = q.lens[b];
  s.bad = r0 < 0 || r1 < r0 || r1 > q.tokens || len < 0 || len > capacity;
  s.row = r0 < 0 ? 0 : r0 > q.tokens ? q.tokens : r0;
  const int64_t past = r1 > q.tokens ? q.tokens : r1;
  s.n = past > s.row ? (int)(past - s.row) : 0;
  s.len = s.bad ? s.n : (int)len;
  return s;
}

__device__ __forceinline__ void kv_bad(int32_t* status) {
  if (status) __hip_atomic_store(status, (int32_t)GPTQ_ERR_INVALID_ARG, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- ragged batches
// a value that all lanes hold, for the scalar unit
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}
__device__ __forceinline__ KvSeq uniform(const KvSeq& s) {
  return KvSeq{uniform(s.row), uniform(s.n), uniform(s.len), uniform((int)s.bad) != 0};
}

// sum over lanes 0 .. this one
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  auto add = [&](auto ctrl, auto rows) {   // lanes of `rows` add what DPP `ctrl` brings them
    constexpr int C = decltype(ctrl)::value, M = decltype(rows)::value;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, C, M, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), C, M, 0xf, false);
    v += (int64_t)((uint64_t)hi << 32 | lo);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});   // 1, 2, 4, 8 lanes before, in rows of 16
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});   // the row before's last lane, to rows 1 and 3
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});   // lane 31, to rows 2 and 3
  return v;
}
// a value of lane l, the same l in all
__device__ __forceinline__ int64_t lane_value(int64_t v, int l) {
  return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, l) | (int64_t)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32;
}

__device__ __forceinline__ KvSeq lane_value(const KvSeq& s, int l) {
  return KvSeq{lane_value(s.row, l), __builtin_amdgcn_readlane(s.n, l), __builtin_amdgcn_readlane(s.len, l),
               __builtin_amdgcn_readlane((int)s.bad, l) != 0};
}

// The sum of count(b) over the batch.  Called by whole waves.
template <class F>
__device__ __forceinline__ int64_t ragged_total(int64_t batch, const F& count) {
  int64_t v = 0;
  for (int64_t b = threadIdx.x & 63; b < batch; b += 64) v += count(b);
  return lane_value(wave_scan(v), 63);
}

// The sequence b in whose count(b) pieces the `index`-th piece of all lies, and
// which of them it is; false past the last.  Called by whole waves, which look at
// 64 sequences at a time: what count() kept of its last call in lane `l` is of b.
// `base` sequences before have `before` pieces: a search for a later piece goes on from there.
template <class F>
__device__ __forceinline__ bool ragged_find(int64_t index, int64_t batch, const F& count, int64_t* b, int64_t* at, int* l,
                                            int64_t* base, int64_t* before) {
  const int lane = threadIdx.x & 63;
  index = uniform(index) - *before;
  for (; *base < batch; *base += 64) {
    const int64_t c = *base + lane < batch ? count(*base + lane) : 0;
    const int64_t upto = wave_scan(c);
    const uint64_t past = __ballot(upto > index);   // wave-uniform
    if (past) {
      *l = __ffsll((unsigned long long)past) - 1;
      *b = *base + *l;
      *at = index - lane_value(upto - c, *l);
      return true;
    }
    const int64_t all = lane_value(upto, 63);
    index -= all;
    *before += all;
  }
  return false;
}
template <class F>
__device__ __forceinline__ bool ragged_find(int64_t index, int64_t batch, const F& count, int64_t* b, int64_t* at, int* l) {
  int64_t base = 0, before = 0;
  return ragged_find(index, batch, count, b, at, l, &base, &before);
}

// ---------------------------------------------------------------- softmax
// The running maximum of x·scale over raw logits x is kept as m + rest: m the rounded
// product, of which weights 2^(x·scale - m) by one fused step keep every bit while half
// a step of m is below 1.  From 2^23 on that half step would be their exponent (past 2^31
// the largest weight itself would be Inf or 0), so rest takes it: the product's exact
// remainder.  Below, rest is 0 and costs nothing.
constexpr float kFar = 0x1p23f;

// Raises the maximum to top·scale where that is more; the factor for what was summed before.
__device__ __forceinline__ float raise_to(float top, float scale, float* m, float* rest) {
  const float m0 = *m, rest0 = *rest;
  if (fmaf(top, scale, -m0) - rest0 > 0.f) {
    *m = top * scale;
    *rest = fabsf(*m) > kFar ? fmaf(top, scale, -*m) : 0.f;
  }
  return exp2f((m0 - *m) + (rest0 - *rest));
}

// A tensor [tokens][heads][D] with unit stride in D, strides in elements.
struct HeadRows {
  const void* p;
  int64_t ld, hs;
  int vec;   // rows may be read 16 bytes at a time
};

// ---------------------------------------------------------------- launchers
gptq_status run_kv_append(const KvLayout& L, const HeadRows& K, const HeadRows& V, int dtype, const KvSeqs& q,
                          void* pages, hipStream_t stream);
gptq_status run_kv_read(const KvLayout& L, const HeadRows& K, const HeadRows& V, int dtype, const KvSeqs& q,
                        const void* pages, hipStream_t stream);

struct KvAttentionPlan {
  int tile;           // rows of queries that a workgroup holds at once: 8, 16 or 32
  int parts;          // bf16 parts of a weight: 2, or 1 (of tiles of 32)
  bool whole;         // a workgroup for each unit (row tile and key head of a sequence), not an equal piece of all
  int wgs, waves;     // workgroups, and waves of each
  int rows;           // rows of a unit that should hold queries
  size_t partial, total;   // workspace bytes
};
// each: one token a sequence (no cu_seqlens); capacity: positions of a sequence that the page table can hold.
// Neither makes the workspace larger than {false, 0}.
KvAttentionPlan plan_kv_attention(const KvLayout& L, int heads, int64_t batch, int64_t tokens, int64_t max_queries,
                                  bool each, int64_t capacity);
gptq_status run_kv_attention(const KvLayout& L, int heads, const HeadRows& Q, const HeadRows& Y, float scale,
                             const KvSeqs& q, const void* pages, void* ws, const KvAttentionPlan& p, hipStream_t stream);

struct PromptCall {
  HeadRows Q, K, V, Y;
  const int32_t* cu;
  int64_t batch, tokens;
  int heads, kv_heads, dim;
  float scale;
};
gptq_status run_prompt_attention(const PromptCall& c, hipStream_t stream);

}  // namespace gptq
