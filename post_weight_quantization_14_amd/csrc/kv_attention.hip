// Attention of the last tokens of each sequence over its 4-bit cache.
//
// With k̂ = (c - z)·s per group of channels and the same for values,
//   logit[t] = scale·Σ_g s_g(t)·(Σ_{d in g} q_d·(128 + c_d(t)) - (128 + z_g(t))·Σ_{d in g} q_d),
//   y_d = Σ_t p'(t)·(128 + c_d(t)) - Σ_t p'(t)·(128 + z(t)),  p' = softmax(t)·s(t):
// 128 + c is a bf16 made from four bits by one AND-OR, so keys enter the matrix
// cores exactly; scales and zero points are taken off in fp32.
//
// What bounds it.  A step of 32 positions reads 4.35 KB (heads of 128, one scale
// each) and takes about 230 vector instructions for up to 8 rows, most of them to
// spread codes, then some 100 more for every further 16.  Decoding many sequences
// is near memory: 64 of up to 8192 tokens with 8 key heads (288 MB) take 80 us, 3.6
// TB/s; the vector unit is busy 67% of the time, the matrix cores 22%.
//   One sequence of 32768 tokens (38 MB) takes 18.5 us: 14 in pieces (a wave has four
// steps; before them three loads wait for each other: lengths, page numbers, codes)
// and 4 to 5 to join 32 of them.  One of 512 takes 7.6 us, most of it that chain.
//   A chunk of 512 tokens over 8192 takes 113 us, 0.59 PFLOP/s: here the vector
// unit spreads the codes again for every 32 rows, busy 77% of the time, the matrix cores 27%.
#include "attention.hpp"

namespace gptq {
namespace {

#define INLINE __attribute__((always_inline))
typedef __attribute__((address_space(4))) int32_t constant_int;

constexpr int kStep = 32;        // positions of a wave's step: two records
constexpr float kNone = -3e38f;  // a running maximum that has seen nothing
constexpr int kMaxWgs = 512;     // of a split call: two a CU (768: 1 x 32768 30 us instead of 20, 64 x 4096 57 instead of 53)

__device__ __forceinline__ float swap16(float x, float* y) {   // lane ^ 16
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  *y = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float swap32(float x, float* y) {   // lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  *y = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
// over the four lanes that hold one query
__device__ __forceinline__ float quad_max(float x) {
  float y;
  x = swap16(x, &y);
  x = fmaxf(x, y);
  x = swap32(x, &y);
  return fmaxf(x, y);
}
__device__ __forceinline__ float quad_sum(float x) {
  float y;
  x = swap16(x, &y);
  x += y;
  x = swap32(x, &y);
  return x + y;
}

// The constants of the AND-OR, hidden from folding (VOP3 takes no literals).
struct Consts {
  uint32_t m, c;
  __device__ __forceinline__ Consts() : m(0x000f000fu), c(0x43004300u) { asm volatile("" : "+v"(m), "+v"(c)); }
  __device__ __forceinline__ uint32_t pair(uint32_t w) const { return (w & m) | c; }   // (128 + nibble 0, 128 + nibble 4)
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {   // nearest even, one instruction
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2_t;
  return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}

template <int N, class F>
__device__ __forceinline__ void by_index(const F& f) {   // f(0) .. f(N - 1), each a constant
  if constexpr (N > 0) {
    by_index<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// The rest of the largest of several maxima m + rest: `each` gives them to its argument,
// `top` is the largest m (equal m's have a rest alike, or none).  They are looked at only
// where some lane's top may have one.
template <class F>
__device__ __forceinline__ float rest_of(float top, const F& each) {
  float rest = 0.f;
  if (__builtin_expect(__ballot(fabsf(top) > kFar) != 0, 0)) {
    rest = -INFINITY;
    each([&](float m, float r) INLINE { rest = m == top ? fmaxf(rest, r) : rest; });
  }
  return rest;
}

struct Split {
  int64_t token;      // of the unit's first row
  int head;           // key head
  uint32_t hq0;       // query head of the first row within the group
  int rows, slot;     // of the first part; part i > 0 is slot 2·(workgroup + i)
  int least;          // positions that its first row sees
  int parts;          // 0: no such unit
};

struct Work {
  KvLayout L;
  KvSeqs q;
  HeadRows Q, Y;
  float scale;           // times log2(e), positive: a masked logit times it stays -Inf
  uint32_t keep, flip;   // Q's bits and signs: a scale of 0 clears it, a negative one flips it
  int share;             // query heads of a key head
  uint32_t share_inv;    // above 2^32 / share: x / share = umulhi(x, share_inv) for x below 2^13 (not for share 1)
  const uint8_t* pages;
  float* partial;        // [2·wgs] of [rows][D] sums, [rows] maxima and their rests, [rows] sums of weights
  Split* meta;           // [wgs]: of a unit split over workgroups that begins in this one
};

// a / b of uniform numbers, by 32 bits where they do
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// A unit is one row tile (R query rows: tokens x the heads that share a key
// head) of one key head of one sequence; its steps are 32 positions each.  All
// units' steps lie one after the other, by sequence, head and tile (WHOLE: all
// units, of one step each here).  Lane i keeps what it read of sequence i: batches of
// up to 64 are read once.  Of larger ones a unit's index tells its sequence where each
// has as many (one token each, taken whole); else a workgroup searches on from its last.
template <int R, bool WHOLE>
struct Units {
  const Work& w;
  int64_t capacity, total;
  KvSeq mine;
  int64_t upto, own;   // steps of sequences 0 .. lane, and of this lane's
  int64_t base = 0, before = 0;   // of the search
  bool few;
  __device__ __forceinline__ explicit Units(const Work& w_) : w(w_) {
    capacity = min64(w.q.width * w.L.recs * kKvRec, kKvMost);
    few = w.q.batch <= 64;
    const int lane = threadIdx.x & 63;
    if (few) {
      mine = KvSeq{0, 0, 0, false};
      own = 0;
      if (lane < w.q.batch) {
        mine = kv_seq(w.q, lane, capacity);
        own = steps_of(mine);
      }
      upto = wave_scan(own);
      total = lane_value(upto, 63);
    } else if (WHOLE) {
      total = INT64_MAX;   // find() tells
    } else {
      total = ragged_total(w.q.batch, [&](int64_t b) { return steps_of(kv_seq(w.q, b, capacity)); });
    }
  }
  static __device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
  static __device__ __forceinline__ int64_t tiles(const KvSeq& s, int share) { return ((int64_t)s.n * share + R - 1) / R; }
  static __device__ __forceinline__ int steps(const KvSeq& s) { return s.len > kStep ? (int)(((int64_t)s.len + kStep - 1) / kStep) : 1; }
  __device__ __forceinline__ int64_t steps_of(const KvSeq& s) const { return tiles(s, w.share) * (WHOLE ? 1 : steps(s)) * w.L.heads; }
  // the sequence that step `pos` belongs to, and which of its steps it is; false past the last
  __device__ __forceinline__ bool find(int64_t pos, KvSeq* found, int64_t* b, int64_t* at) {
    KvSeq s = mine;
    int l;
    if (few) {
      l = __ffsll((unsigned long long)__ballot(upto > pos)) - 1;
      *b = l;
      *at = pos - lane_value(upto - own, l);
    } else if (WHOLE && w.q.cu == nullptr) {
      const int64_t each = (int64_t)((w.share + R - 1) / R) * w.L.heads;
      *b = divide(pos, each);
      *at = pos - *b * each;
      if (*b >= w.q.batch) return false;
      *found = uniform(kv_seq(w.q, *b, capacity));
      return true;
    } else {
      auto count = [&](int64_t i) {
        s = kv_seq(w.q, i, capacity);
        return steps_of(s);
      };
      if (!ragged_find(pos, w.q.batch, count, b, at, &l, &base, &before)) return false;
    }
    *found = lane_value(s, l);
    return true;
  }
};

// lane n of the row of 16 for SP 1, of the lane's own four for SP 2
template <int SP, int N>
__device__ __forceinline__ float lane_of(float x) {
  constexpr int kCtrl = SP == 1 ? 0x150 + N : (N & 3) * 0x55;
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), kCtrl, 0xf, 0xf, true));
}

// Params of the step's positions.  SP 1: lane 16·kg + 4·j + r has those of position
// 4·kg + r, j = 0, 1: keys of the two records, 2, 3: values.  SP 2: lane
// 16·kg + 8·u + 4·i + r has those of position 4·kg + r of record u, word 0 keys, word 1 values.
template <int D, int G, int SP>
struct Step {
  static constexpr int KS = D / 32, NG = D / G;
  uint32_t k[2][KS], v[2][KS];
  uint32_t pw[SP][NG];
  bool bad;          // a page that is none, of the lane's own record
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else {
    const u32x2_t x = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = x[0];
    w[1] = x[1];
  }
}

// values of tile 2·b + h (channels 32·b + 2i + h) at four positions, as two operand words
template <int D>
__device__ __forceinline__ void value_pairs(const uint32_t (&w)[D / 32], int b, int h, const Consts& kc, uint32_t* o) {
  if constexpr (D == 128) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t x = __builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], 0x0c000c00u | (uint32_t)(4 + b) << 16 | (uint32_t)b);
      o[e] = kc.pair(h ? x >> 4 : x);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) o[e] = kc.pair(w[e] >> (8 * b + 4 * h));
  }
}

// W waves share a unit's steps.  WHOLE: a workgroup takes one unit; otherwise each
// takes an equal piece of all units' steps, and units cut by a piece's end are
// joined by kv_join_kernel.
//   Rows are columns of the products.  With SP 2 (up to 8 rows) both halves of the 16
// columns hold the same rows; the left half keeps the logits of the step's first
// record, the right half those of the second, each with sums of its own, so that no
// lane works for rows that are not there: 64 x 4096 56.6 -> 53.1 us.  NT 2 holds 32
// rows: codes are spread once for both tiles, and with one scale a head a product sums
// the zero points as well.  PARTS is in how many bf16 parts weights enter: 2 leave 2^-16
// of each, 1 leaves 2^-8, as the result's own rounding does.
template <int D, int G, int NT, int SP, int PARTS, int W, bool WHOLE>
__global__ __launch_bounds__(64 * W, 2) void kv_attention_kernel(Work w) {
  constexpr int kThreads = 64 * W, R = 16 * NT / SP, NC = 16 / SP, E = 8 / SP, KS = D / 32, NG = D / G, MT = D / 16, PG = G / 32;   // PG: 32-channel steps of a group
  constexpr int kPitch = D + 4;
  __shared__ float so[W][16][kPitch];
  __shared__ float sm[W][16], sr[W][16], sl[W][16];
  // Maxima with a rest lie here while the wave has one: its logits are then taken relative
  // to them before their weights, and m is 0, by 1 (registers are short).
  __shared__ float far_m[W][NT * 16], far_rest[W][NT * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, kg = lane >> 4;
  const int nq = n16 % NC, half = n16 / NC;   // query row of the column, record of its logits
  Units<R, WHOLE> units(w);
  const Consts kc;

  // in steps, or in units where each is taken whole
  const int64_t even = divide(units.total + gridDim.x - 1, gridDim.x), piece = WHOLE ? 1 : even > W ? even : W;   // a step for each wave
  const int64_t begin = piece * blockIdx.x, end = begin + piece < units.total ? begin + piece : units.total;
  if (!WHOLE && tid == 0) w.meta[blockIdx.x].parts = 0;
  if (w.q.status)
    for (int64_t b = (int64_t)blockIdx.x * kThreads + tid; b < w.q.batch; b += (int64_t)gridDim.x * kThreads)
      if (kv_seq(w.q, b, units.capacity).bad) kv_bad(w.q.status);

  for (int64_t pos = begin; pos < end;) {
    int64_t b = 0, at = 0;
    KvSeq s;
    if (!units.find(pos, &s, &b, &at)) break;
    const int steps = units.steps(s);
    const int64_t unit = WHOLE ? at : divide(at, steps);          // head · tiles + tile
    const int s0 = WHOLE ? 0 : (int)(at - unit * steps);
    const int s1 = WHOLE || steps - s0 < end - pos ? steps : s0 + (int)(end - pos);
    const int64_t tiles = units.tiles(s, w.share);
    const int head = (int)divide(unit, tiles);
    const int64_t row0 = (unit - head * tiles) * R, tq0 = divide(row0, w.share);
    const uint32_t hq0 = (uint32_t)(row0 - tq0 * w.share);   // row0 is head hq0 of the group, token tq0
    const int rows = (int)units.min64(R, (int64_t)s.n * w.share - row0);

    // ---- queries: column n16 holds query row 16·nt + nq
    u32x4_t qx[NT][KS];
    int lim[NT];     // positions that the row sees
    const uint16_t* qp[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int i = nt * 16 + nq < rows ? nt * 16 + nq : 0;   // rows past the last: computed, not stored
      const uint32_t h = hq0 + i, t = w.share == 1 ? h : __umulhi(h, w.share_inv);
      lim[nt] = s.len - s.n + (int)tq0 + (int)t + 1;
      qp[nt] = static_cast<const uint16_t*>(w.Q.p) + (s.row + tq0 + t) * w.Q.ld + (head * w.share + (h - t * w.share)) * w.Q.hs + kg * 8;
    }
    if (w.Q.vec) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qx[nt][ks] = *reinterpret_cast<const u32x4_t*>(qp[nt] + ks * 32);
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 4; ++i) qx[nt][ks][i] = qp[nt][ks * 32 + 2 * i] | (uint32_t)qp[nt][ks * 32 + 2 * i + 1] << 16;
    }
    const int least = s.len - s.n + (int)tq0 + 1;   // positions that every row sees

    // ---- the wave's steps s0 + wave, + 4, ..
    const int last = uniform((s.len - 1) / kKvRec);   // record; pages past it may be none
    // page numbers go through the scalar unit a step ahead of the records in them
    const constant_int* table = (const constant_int*)uniform((int64_t)(s.bad ? w.q.lens + b : w.q.table + b * w.q.stride));
    const int page_shift = uniform(s.bad ? 31 : w.L.rec_shift);   // any number that can be read
    struct Pages {
      int id[2];
    };
    auto page_of = [&](int st) INLINE {
      Pages p;
#pragma unroll
      for (int u = 0; u < 2; ++u) p.id[u] = table[min(2 * st + u, last) >> page_shift];
      return p;
    };
    const uint32_t head_at = (uint32_t)head << w.L.rec_shift;
    const int param_at = 2 * kv_code_bytes(D) + (SP == 1 ? (n16 >> 3) * kv_param_bytes(D, G) : 0) + (kg * 4 + (n16 & 3)) * 4;
    auto load = [&](int st, const Pages& pg, Step<D, G, SP>& x) INLINE {
      const uint8_t* base[2];
      bool none[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int page = uniform(pg.id[u]);
        none[u] = s.bad || (uint32_t)page >= (uint32_t)w.q.pages;
        const int64_t id = none[u] ? 0 : page;
        const uint32_t rec = head_at + (min(2 * st + u, last) & (w.L.recs - 1));
        const uint8_t* p = w.pages + id * w.L.page_bytes + (int64_t)rec * kv_rec_bytes(D, G);
        load_words(p + lane * (D / 8), x.k[u]);
        load_words(p + (kv_code_bytes(D) + lane * (D / 8)), x.v[u]);
        base[u] = p;
      }
      const bool second = SP == 1 ? lane & 4 : half;
      x.bad = second ? none[1] : none[0];
      const uint8_t* p = (second ? base[1] : base[0]) + param_at;
#pragma unroll
      for (int i = 0; i < SP; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g) x.pw[i][g] = *reinterpret_cast<const uint32_t*>(p + i * kv_param_bytes(D, G) + g * 64);
    };
    Step<D, G, SP> cur, nxt;
    int st = s0 + wave;
    const bool some = st < s1 && s.len > 0;
    Pages ahead;
    bf16x8_t qf[NT][KS];
    float qs[NT][NG];   // sums of the query's channels, by group
    constexpr bool kMat = NT == 2 && NG == 1;   // sums of zero points by the matrix cores too
    f32x4_t zo[NT];
    uint32_t za[4] = {0, 0, 0, 0};
    // bytes that lane takes of its own word (4 .. 7) and its neighbour's (0 .. 3): even lanes both high halves, odd both low
    const uint32_t zsel = lane & 1 ? 0x05040100u : 0x03020706u;
    f32x4_t o[NT][MT];
    float m[NT], by = w.scale, l[NT], zs[NT][NG];   // weights are 2^(logit·by - m)
    uint64_t far = 0;   // lanes with a rest
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = kNone;
      l[nt] = 0.f;
      zo[nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < NG; ++g) zs[nt][g] = 0.f;
#pragma unroll
      for (int j = 0; j < MT; ++j) o[nt][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    auto compute = [&](int st, Step<D, G, SP>& x, auto next) INLINE {
      next();
      float sf[SP][NG], zf[SP][NG];   // scales and 128 + zero points, of the positions of `pw`
#pragma unroll
      for (int i = 0; i < SP; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          sf[i][g] = __uint_as_float(x.bad ? 0x7fc00000u : x.pw[i][g] & 0xffff0000u);
          zf[i][g] = (float)((int)(int16_t)(uint16_t)x.pw[i][g] + 128);
        }
      if (x.bad) kv_bad(w.q.status);
      // logits of positions at(i), i = 4·record + r (SP 1), r (SP 2)
      float sx[NT][E];
      auto at = [&](int i) { return st * kStep + (SP == 1 ? (i >> 2) * 16 : half * 16) + kg * 4 + (i & 3); };
      f32x4_t acc[NT][NG][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bf16x8_t a[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          u32x4_t t;
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = kc.pair(x.k[u][ks] >> (4 * i));
          a[ks] = __builtin_bit_cast(bf16x8_t, t);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][g][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = g * PG; ks < (g + 1) * PG; ++ks)
              acc[nt][g][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[ks], qf[nt][ks], acc[nt][g][u], 0, 0, 0);
            if constexpr (SP == 1)
              by_index<4>([&](auto r) INLINE {
                const float z = u ? lane_of<1, 4 + r.value>(zf[0][g]) : lane_of<1, r.value>(zf[0][g]);
                const float f = u ? lane_of<1, 4 + r.value>(sf[0][g]) : lane_of<1, r.value>(sf[0][g]);
                const float y = acc[nt][g][u][r.value] - z * qs[nt][g];
                float& o = sx[nt][u * 4 + r.value];
                o = g == 0 ? y * f : o + y * f;
              });
          }
      }
      if constexpr (SP == 2) {   // each half of the columns takes a record's
#pragma unroll
        for (int g = 0; g < NG; ++g)
          by_index<4>([&](auto r) INLINE {
            const float c = half ? acc[0][g][1][r.value] : acc[0][g][0][r.value];
            const float y = c - lane_of<2, r.value>(zf[0][g]) * qs[0][g], f = lane_of<2, r.value>(sf[0][g]);
            float& o = sx[0][r.value];
            o = g == 0 ? y * f : o + y * f;
          });
      }
      const bool edge = (st + 1) * kStep > least;
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (at(i) >= lim[nt]) sx[nt][i] = -INFINITY;
      }
      // running maximum of a column; its sums are scaled again only when that grows by more than 2^8
      bool grown = false;
      float top[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float t = sx[nt][0];
#pragma unroll
        for (int i = 1; i < E; ++i) t = fmaxf(t, sx[nt][i]);
        top[nt] = quad_max(t);
        grown |= fmaf(top[nt], w.scale, -m[nt]) > 8.f;
      }
      if (far | __ballot(grown)) {
        float rest[NT];
        bool rests = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          rest[nt] = 0.f;
          if (__builtin_expect(far != 0, 0)) m[nt] = far_m[wave][nt * 16 + n16], rest[nt] = far_rest[wave][nt * 16 + n16];
          const float f = raise_to(top[nt], w.scale, &m[nt], &rest[nt]);
          rests |= rest[nt] != 0.f;
          l[nt] *= f;
#pragma unroll
          for (int g = 0; g < NG; ++g) zs[nt][g] *= f;
          if (kMat) zo[nt] *= f;
#pragma unroll
          for (int j = 0; j < MT; ++j) o[nt][j] *= f;
        }
        far = __ballot(rests);
        by = w.scale;
        if (__builtin_expect(far != 0, 0)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            far_m[wave][nt * 16 + n16] = m[nt];   // the same in the four lanes of a column
            far_rest[wave][nt * 16 + n16] = rest[nt];
#pragma unroll
            for (int i = 0; i < E; ++i) sx[nt][i] = fmaf(sx[nt][i], w.scale, -m[nt]) - rest[nt];
            m[nt] = 0.f;
          }
          by = 1.f;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          float& p = sx[nt][i];
          p = __builtin_amdgcn_exp2f(fmaf(p, by, -m[nt]));
          l[nt] += p;
        }
      // values
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (kMat) {
          // 128 + z = hi + lo with 8 bits each; quad 2 of a row of lanes has record 0's, quad 3 record 1's
          const uint32_t zi = (uint32_t)((int)(int16_t)(uint16_t)x.pw[0][g] + 128);
          const float lo = (float)(zi & 255u), hi = zf[0][g] - lo;
          const uint32_t own = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
          const uint32_t other = __builtin_amdgcn_mov_dpp(own, 0xb1, 0xf, 0xf, true);
          const uint32_t both = __builtin_amdgcn_perm(own, other, zsel);
          za[0] = __builtin_amdgcn_update_dpp(za[0], both, 0x44, 0xf, 0x4, false);
          za[1] = __builtin_amdgcn_update_dpp(za[1], both, 0xee, 0xf, 0x4, false);
          za[2] = __builtin_amdgcn_update_dpp(za[2], both, 0x44, 0xf, 0x8, false);
          za[3] = __builtin_amdgcn_update_dpp(za[3], both, 0xee, 0xf, 0x8, false);
        }
        bf16x8_t ph[NT], pl[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pw[E];
          by_index<E>([&](auto i) INLINE { pw[i.value] = lane_of<SP, 8 + i.value>(sf[SP - 1][g]) * sx[nt][i.value]; });
          if (edge) {   // the scale there may be anything
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (at(i) >= lim[nt]) pw[i] = 0.f;
          }
          uint32_t hw[E / 2], lw[E / 2];
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            const uint32_t h = pack_bf16(pw[2 * i], pw[2 * i + 1]);
            if constexpr (PARTS == 1) {
              hw[i] = h;
              pw[2 * i] = __uint_as_float(h << 16);
              pw[2 * i + 1] = __uint_as_float(h & 0xffff0000u);
              continue;
            }
            const float h0 = __uint_as_float(h << 16), h1 = __uint_as_float(h & 0xffff0000u);
            const uint32_t lo = pack_bf16(pw[2 * i] - h0, pw[2 * i + 1] - h1);
            hw[i] = h;
            lw[i] = lo;
            pw[2 * i] = h0 + __uint_as_float(lo << 16);
            pw[2 * i + 1] = h1 + __uint_as_float(lo & 0xffff0000u);
          }
          if constexpr (!kMat) by_index<E>([&](auto i) INLINE { zs[nt][g] += lane_of<SP, 8 + i.value>(zf[SP - 1][g]) * pw[i.value]; });
          u32x4_t hx, lx;
          if constexpr (SP == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) hx[i] = hw[i], lx[i] = PARTS == 2 ? lw[i] : 0;
          } else {   // a column's weights stand at its record's positions, zeros at the other's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool mine = half == i >> 1;
              hx[i] = mine ? hw[i & 1] : 0;
              lx[i] = mine ? lw[i & 1] : 0;
            }
          }
          ph[nt] = __builtin_bit_cast(bf16x8_t, hx);
          pl[nt] = __builtin_bit_cast(bf16x8_t, lx);
          if constexpr (kMat) {
            const bf16x8_t z = __builtin_bit_cast(bf16x8_t, u32x4_t{za[0], za[1], za[2], za[3]});
            zo[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z, ph[nt], zo[nt], 0, 0, 0);
            if constexpr (PARTS == 2) zo[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z, pl[nt], zo[nt], 0, 0, 0);
          }
        }
#pragma unroll
        for (int j = g * PG * 2; j < (g + 1) * PG * 2; ++j) {
          u32x4_t t;
          uint32_t a0[2], a1[2];
          value_pairs<D>(x.v[0], j >> 1, j & 1, kc, a0);
          value_pairs<D>(x.v[1], j >> 1, j & 1, kc, a1);
          t[0] = a0[0], t[1] = a0[1], t[2] = a1[0], t[3] = a1[1];
          const bf16x8_t a = __builtin_bit_cast(bf16x8_t, t);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ph[nt], o[nt][j], 0, 0, 0);
            if constexpr (PARTS == 2) o[nt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, pl[nt], o[nt][j], 0, 0, 0);
          }
        }
      }
    };
    if (some) {
      load(st, page_of(st), cur);
      ahead = page_of(min(st + W, s1 - 1));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qx[nt][ks][i] = (qx[nt][ks][i] & w.keep) ^ w.flip;
          qf[nt][ks] = __builtin_bit_cast(bf16x8_t, qx[nt][ks]);
          float t = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) t += __uint_as_float(qx[nt][ks][i] << 16) + __uint_as_float(qx[nt][ks][i] & 0xffff0000u);
          t = quad_sum(t);
          qs[nt][ks / PG] = ks % PG == 0 ? t : qs[nt][ks / PG] + t;
        }
      for (;;) {
        compute(st, cur, [&]() INLINE {
          load(min(st + W, s1 - 1), ahead, nxt);
          ahead = page_of(min(st + 2 * W, s1 - 1));
        });
        if ((st += W) >= s1) break;
        compute(st, nxt, [&]() INLINE {
          load(min(st + W, s1 - 1), ahead, cur);
          ahead = page_of(min(st + 2 * W, s1 - 1));
        });
        if ((st += W) >= s1) break;
      }
    }

    // ---- the waves' sums together, and for SP 2 the halves of the columns: 16 columns at a time
    const bool whole = WHOLE || (s0 == 0 && s1 == steps);
    const int slot = pos == begin ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1;
    float* part = w.partial + (int64_t)slot * R * (D + 3);
    if (!whole && s0 == 0 && tid == 0)
      w.meta[blockIdx.x] = Split{s.row + tq0, head, hq0, rows, slot, least, (int)((pos + steps - 1) / piece) - (int)blockIdx.x + 1};
    auto top_of = [&](int row, float* rest) INLINE {   // of the waves' and halves' maxima of a row
      float up = kNone;
#pragma unroll
      for (int v = 0; v < W; ++v)
#pragma unroll
        for (int c = 0; c < SP; ++c) up = fmaxf(up, sm[v][c * NC + row]);
      *rest = rest_of(up, [&](auto take) INLINE {
        for (int v = 0; v < W; ++v)
          for (int c = 0; c < SP; ++c) take(sm[v][c * NC + row], sr[v][c * NC + row]);
      });
      return up;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float rest = 0.f;
      if (far) m[nt] = far_m[wave][nt * 16 + n16], rest = far_rest[wave][nt * 16 + n16];
      l[nt] = quad_sum(l[nt]);
      if (kMat) zs[nt][0] = kg >= 2 ? zo[nt][0] + zo[nt][1] : 0.f;   // rows 8, 9 and 12, 13
#pragma unroll
      for (int g = 0; g < NG; ++g) zs[nt][g] = quad_sum(zs[nt][g]);
      if (kg == 0) sm[wave][n16] = m[nt], sr[wave][n16] = rest;
      __syncthreads();
      float up_rest;
      const float up = top_of(nq, &up_rest), f = exp2f((m[nt] - up) + (rest - up_rest));
      if (kg == 0) sl[wave][n16] = l[nt] * f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          so[wave][n16][(j >> 1) * 32 + 2 * (kg * 4 + r) + (j & 1)] = (o[nt][j][r] - zs[nt][j / (2 * PG)]) * f;
      __syncthreads();
      for (int i = tid; i < NC * (D / 4); i += kThreads) {
        const int n = i / (D / 4), d = i % (D / 4) * 4;
        if (nt * 16 + n >= rows) continue;
        float ll = 0.f;
        f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < W; ++v)
#pragma unroll
          for (int c = 0; c < SP; ++c) {
            ll += sl[v][c * NC + n];
            y += *reinterpret_cast<const f32x4_t*>(&so[v][c * NC + n][d]);
          }
        if (whole) {
          const uint32_t i = hq0 + nt * 16 + n, t = w.share == 1 ? i : __umulhi(i, w.share_inv);
          const float inv = least + (int)t > 0 ? 1.f / ll : 0.f;   // a row that sees nothing gives zeros
          uint16_t* yp = const_cast<uint16_t*>(static_cast<const uint16_t*>(w.Y.p)) + (s.row + tq0 + t) * w.Y.ld +
                         (head * w.share + (i - t * w.share)) * w.Y.hs + d;
          uint16_t h[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) h[c] = __builtin_bit_cast(uint16_t, (__bf16)(y[c] * inv));
          if (w.Y.vec) {
            *reinterpret_cast<u32x2_t*>(yp) = u32x2_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) yp[c] = h[c];
          }
        } else {
          *reinterpret_cast<f32x4_t*>(part + (nt * 16 + n) * D + d) = y;
          if (d == 0) {
            float top_rest;
            part[R * D + nt * 16 + n] = top_of(n, &top_rest);
            part[R * D + R + nt * 16 + n] = top_rest;
            part[R * D + 2 * R + nt * 16 + n] = ll;
          }
        }
      }
      __syncthreads();
    }
    pos += WHOLE ? 1 : s1 - s0;
  }
}

// Joins the parts of units that were split: a wave takes a row of a unit at a time.
// The units are few and anywhere among `meta`, so each workgroup lists them first.
// What this costs is a chain of loads, not their bytes: a row's parts are all in
// flight at once, 64 at the most.  4 to 5 us after 1 x 32768 tokens and after a chunk.
constexpr int kJoinWgs = 512;
template <int D, int R>
__global__ __launch_bounds__(256) void kv_join_kernel(Work w, int wgs, int most_rows) {
  constexpr int64_t kSize = R * (D + 3);
  constexpr int L4 = D / 4, P = 64 / L4;   // lanes of a row, four channels each; parts side by side
  __shared__ int16_t list[kMaxWgs];
  __shared__ int count[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  constexpr int E = kMaxWgs / 256;
  int found = 0, parts_of[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    parts_of[e] = i < wgs ? w.meta[i].parts : 0;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) found += parts_of[e] > 0;
  const int before = (int)wave_scan(found);
  if (lane == 63) count[wave] = before;
  __syncthreads();
  int at = before - found, all = 0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (v < wave) at += count[v];
    all += count[v];
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (parts_of[e] > 0) list[at++] = (int16_t)(tid * E + e);
  __syncthreads();
  const int c4 = lane % L4 * 4, side = lane / L4;
  for (int pair = (int)blockIdx.x * 4 + wave; pair < uniform(all) * most_rows; pair += (int)gridDim.x * 4) {
    const int first = uniform((int)list[pair / most_rows]);
    const Split u = w.meta[first];
    const int parts = uniform(u.parts);
    const float* p0 = w.partial + uniform(u.slot) * kSize;
    const float* p1 = w.partial + 2 * (int64_t)first * kSize;
    for (int row = pair % most_rows; row < uniform(u.rows); row += most_rows) {
      float up = kNone, up_rest = 0.f, ll = 0.f;
      f32x4_t y = {0.f, 0.f, 0.f, 0.f};
      auto some = [&](auto n, int base) INLINE {   // parts base + P·j + side, j < N
        constexpr int N = decltype(n)::value;
        float m[N], l[N], rest[N];
        f32x4_t v[N];
        auto part = [&](int j) INLINE {
          const int i = min(base + P * j + side, parts - 1);
          return i == 0 ? p0 : p1 + 2 * i * kSize;
        };
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float* p = part(j);
          m[j] = p[R * D + row];
          rest[j] = 0.f;
          l[j] = p[R * D + 2 * R + row];
          v[j] = *reinterpret_cast<const f32x4_t*>(p + row * D + c4);
        }
        float top = up;
#pragma unroll
        for (int j = 0; j < N; ++j) top = fmaxf(top, m[j]);
#pragma unroll
        for (int d = L4; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        float top_rest = rest_of(top, [&](auto take) INLINE {
          take(up, up_rest);
#pragma unroll
          for (int j = 0; j < N; ++j) take(m[j], rest[j] = part(j)[R * D + R + row]);
        });
        if (__builtin_expect(__ballot(top_rest != 0.f) != 0, 0))
#pragma unroll
          for (int d = L4; d < 64; d <<= 1) top_rest = fmaxf(top_rest, __shfl_xor(top_rest, d));
        const float f = exp2f((up - top) + (up_rest - top_rest));
        up = top;
        up_rest = top_rest;
        ll *= f;
        y *= f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float g = exp2f((m[j] - up) + (rest[j] - up_rest));
          if (base + P * j + side < parts) {
            ll = fmaf(l[j], g, ll);
            y += v[j] * g;
          }
        }
      };
      if (parts <= 4 * P)
        some(std::integral_constant<int, 4>{}, 0);
      else
        for (int base = 0; base < parts; base += 16 * P) some(std::integral_constant<int, 16>{}, base);
#pragma unroll
      for (int d = L4; d < 64; d <<= 1) {
        ll += __shfl_xor(ll, d);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] += __shfl_xor(y[c], d);
      }
      if (side) continue;
      const uint32_t i = uniform((int)u.hq0) + row, t = w.share == 1 ? i : __umulhi(i, w.share_inv);
      const float inv = u.least + (int)t > 0 ? 1.f / ll : 0.f;   // a row that sees nothing gives zeros
      uint16_t* yp = const_cast<uint16_t*>(static_cast<const uint16_t*>(w.Y.p)) + (u.token + t) * w.Y.ld +
                     (u.head * w.share + (i - t * w.share)) * w.Y.hs + c4;
#pragma unroll
      for (int c = 0; c < 4; ++c) yp[c] = __builtin_bit_cast(uint16_t, (__bf16)(y[c] * inv));
    }
  }
}

template <int D, int G, int NT, int SP, int PARTS>
gptq_status launch(const Work& w, const KvAttentionPlan& p, hipStream_t stream) {
  if (p.whole) {
    if (p.waves == 8)
      kv_attention_kernel<D, G, NT, SP, PARTS, 8, true><<<p.wgs, 512, 0, stream>>>(w);
    else if (p.waves == 4)
      kv_attention_kernel<D, G, NT, SP, PARTS, 4, true><<<p.wgs, 256, 0, stream>>>(w);
    else if (p.waves == 2)
      kv_attention_kernel<D, G, NT, SP, PARTS, 2, true><<<p.wgs, 128, 0, stream>>>(w);
    else
      kv_attention_kernel<D, G, NT, SP, PARTS, 1, true><<<p.wgs, 64, 0, stream>>>(w);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
  }
  if (p.waves == 8)
    kv_attention_kernel<D, G, NT, SP, PARTS, 8, false><<<p.wgs, 512, 0, stream>>>(w);
  else
    kv_attention_kernel<D, G, NT, SP, PARTS, 4, false><<<p.wgs, 256, 0, stream>>>(w);
  GPTQ_LAUNCH_CHECK();
  kv_join_kernel<D, 16 * NT / SP><<<kJoinWgs, 256, 0, stream>>>(w, p.wgs, p.rows);
  GPTQ_LAUNCH_CHECK();
  return GPTQ_OK;
}

}  // namespace

// A unit is a workgroup's of its own, in one launch, where the page table holds no
// longer sequence than kWhole; otherwise a long one would be waited for, and
// workgroups get equal pieces of all units' steps.  Heads of 128, 8 key heads, us
// (whole / pieces): 1 x 512 tokens 7.5 / 10.7, 32 x 768 of 32 key heads 22.2 / 26.7, 64 x 1000
// 16.7 / 19.1, 128 x 250 of 32 heads 31 / 54, 1 x 1024 10.2 / 10.5, but 1 x 2048 15.0 / 10.9.
// Its waves are as many as leave a CU eight at the most: 64 x 100 of 32 heads, 2048
// units, 11.1 with one wave each, 14.7 with two, 17.6 with four; 64 x 512, 512 units,
// 17.7, 15.3 and 10.9; and have a step of the table each, eight of them three: 1 x 100
// 5.3 with four, 5.8 with eight, 1 x 250 6.1 and 6.9, 1 x 512 7.5 and 8.0, 1 x 900 10.5 and 10.3.
//   With cu_seqlens each such workgroup searches the batch for its unit, so larger ones go in
// pieces, which search once: sequences of 20 tokens, 32 heads on 8, us (whole / pieces):
// 1600 73 / 132, 4096 330 / 327, 16384 4222 / 1299.
constexpr int64_t kWhole = 1024, kMostUnits = 1 << 22;   // a grid's limit is 2^32 threads
constexpr int64_t kSearched = 4096;
// Weights are rounded once for chunks, where the matrix cores and the vector unit are the
// bound (512 tokens over 8192, 32 heads on 8: 112 us, 130 in two parts; groups of 64 147 and
// 182, of 32 236 and 319): from more tokens a sequence on than drafts have, whatever the heads.
constexpr int64_t kDrafts = 16;
// Two parts for 32 rows of more scales than one a head are short of registers: 16 sequences
// of 4096, 6 drafts of 4 heads a key head, groups of 64 39.5 us by tiles of 16 rows and 41.1
// of 32, groups of 32 51 and 106; with one scale a head 33.5 and 29.7.
// Smaller tiles of rows while there is a CU for each unit: 5 tokens x 4 heads a key
// head over 900 positions, us with tiles of 32, 16 and 8: 4 sequences 15.4, -, 10.4 (96 units
// of 8), 16 sequences 15.4, 11.9 (256 of 16) and 15.5 (384 of 8).
constexpr int64_t kUnits = 256;
// Pieces go to 256 workgroups of 8 waves where few units are cut into many parts, so
// that half of these are joined; to 512 of 4 otherwise.  us (8 waves / 4), one sequence: 1
// key head, 8192 positions 12.0 / 12.5, 32768 17.8 / 24.4; 8 heads, 8192 12.7 / 14.6, 32768
// 16.7 / 18.6, but 4096 12.0 / 11.1; 4 sequences of 2048 (32 units) 11.2 / 12.5, 8 of 4096 (64)
// 15.3 / 15.4, 64 of 4096 54 / 51; a chunk of 512 tokens (512 units) 117 / 112.
constexpr int64_t kWideUnits = 64, kWideFew = 16, kWidePositions = 8192;

KvAttentionPlan plan_kv_attention(const KvLayout& L, int heads, int64_t batch, int64_t tokens, int64_t max_queries,
                                  bool each, int64_t capacity) {
  KvAttentionPlan p;
  const int64_t share = heads / L.heads, some = std::min(batch, tokens);   // sequences that may have tokens
  const int64_t rows = (each ? 1 : std::min(std::max<int64_t>(max_queries, 1), std::max<int64_t>(tokens, 1))) * share;
  p.parts = rows / share > kDrafts ? 1 : 2;
  const int tile = rows <= 8 ? 8 : rows <= 16 || (p.parts == 2 && L.group != L.dim) ? 16 : 32;
  p.tile = tile;
  // Units at the most, for the grid: n rows take up to (n + tile - 1) / tile.  And as many as there should be, for the
  // choices: every sequence with the rows that max_queries says (the bound gives 64 sequences of 8 rows 120 a key head).
  auto most = [&](int tile) {
    return L.heads * (each ? batch * ceil_div(share, tile) : (tokens * share + (tile - 1) * some) / tile);
  };
  auto units = [&](int tile) { return std::min(most(tile), L.heads * some * ceil_div(rows, tile)); };
  p.whole = capacity <= kWhole && most(tile) <= kMostUnits && (each || batch <= kSearched);
  if (p.whole)
    while (p.tile > 8 && units(p.tile / 2) <= kUnits && most(p.tile / 2) <= kMostUnits) p.tile /= 2;
  p.rows = (int)std::min<int64_t>(rows, p.tile);
  if (p.whole) {
    p.wgs = (int)most(p.tile);
    p.waves = capacity >= 3 * 8 * kStep ? 8 : 4;
    while (p.waves > 1 && (units(p.tile) * p.waves > 2048 || p.waves * kStep > capacity)) p.waves /= 2;
  } else {
    const bool wide = units(tile) <= kWideUnits && (units(tile) >= kWideFew || capacity >= kWidePositions);
    p.wgs = wide ? kMaxWgs / 2 : kMaxWgs;
    p.waves = wide ? 8 : 4;
  }
  p.partial = (size_t)2 * kMaxWgs * tile * (L.dim + 3) * 4;   // whatever the capacity
  p.total = align256(p.partial) + (size_t)kMaxWgs * sizeof(Split);
  return p;
}

gptq_status run_kv_attention(const KvLayout& L, int heads, const HeadRows& Q, const HeadRows& Y, float scale,
                             const KvSeqs& q, const void* pages, void* ws, const KvAttentionPlan& p, hipStream_t stream) {
  const Work w{L, q, Q, Y, scale == 0.f ? 1.f : fabsf(scale) * 1.44269504088896340736f, scale == 0.f ? 0u : ~0u,
               scale < 0.f ? 0x80008000u : 0u, heads / L.heads, (uint32_t)((1ull << 32) / (heads / L.heads) + 1),
               static_cast<const uint8_t*>(pages),
               static_cast<float*>(ws), reinterpret_cast<Split*>(static_cast<uint8_t*>(ws) + align256(p.partial))};
  auto tiled = [&](auto d, auto g) {
    if (p.tile == 8) return launch<d.value, g.value, 1, 2, 2>(w, p, stream);
    if (p.tile == 16) return launch<d.value, g.value, 1, 1, 2>(w, p, stream);
    if constexpr (d.value == g.value)
      if (p.parts == 2) return launch<d.value, g.value, 2, 1, 2>(w, p, stream);
    return launch<d.value, g.value, 2, 1, 1>(w, p, stream);
  };
  using std::integral_constant;
  if (L.dim == 128 && L.group == 128) return tiled(integral_constant<int, 128>{}, integral_constant<int, 128>{});
  if (L.dim == 128 && L.group == 64) return tiled(integral_constant<int, 128>{}, integral_constant<int, 64>{});
  if (L.dim == 128) return tiled(integral_constant<int, 128>{}, integral_constant<int, 32>{});
  if (L.group == 64) return tiled(integral_constant<int, 64>{}, integral_constant<int, 64>{});
  return tiled(integral_constant<int, 64>{}, integral_constant<int, 32>{});
}

}  // namespace gptq
