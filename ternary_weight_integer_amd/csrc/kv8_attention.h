// Attention over the int8 K/V cache: the kernels, how a call is laid out, and
// its launches.
#pragma once

#include "kv8_device.h"

namespace {

// ---------------------------------------------------------------------------
// Attention.
//
// A wave owns one or two tiles of 16 rows (row = query token and head of the K/V
// head's group, so that a group shares what is read of the cache) and walks
// tiles of 64 tokens.  Everything stays in registers, operands are loaded
// straight into the order of the matrix instructions:
//   S^T = K Q^T   in one of two forms, in both of which a wide channel of a query
//     takes nothing from its other components (with 23 bits of the row's largest
//     magnitude F32 results were 60 times as far off as in F32 products where one
//     component was 1000 times the rest, with 15 BF16 results twice their rounding):
//     digits   int8 16x16x64.  The codes are exact, a query is four signed
//       base-256 digits of a fixed-point number (its row's largest magnitude
//       brought to 30 bits or more by a power of two), the int32 dots are exact.
//     direct   f16 16x16x32, sums in F32.  The codes are exact.  An F16 query is
//       its own operand, one of BF16 is exact when brought to 2^15 by a power of
//       two (to 2^-40 of the row's largest magnitude), one of F32 is then the sum
//       of two (22 bits).  The keys have to be turned into f16.
//   O^T = V^T P^T  f16 16x16x32.  V's codes are exact in f16; a weight is the sum
//     of two (22 bits), where many BF16 rows of plain scores are worked on one (11
//     bits: its rounding is an eighth of the result's own, and adds 0.5 to 0.8% to
//     its error; a second takes 18 to 20% of a prompt's time, and 1 to 4% where
//     rows are few).  Shaped scores have the second always: four capped BF16
//     prompts of 500 to 4000 tokens, 16 heads over 8 of 128, 184 us against 163.
// The rows of K's four 16-token operands are taken from the tile in the order
// 16 (m / 4) + 4 j + m % 4, which leaves lane (row, g) with the logits of the
// 16 consecutive tokens 16 g ..: those are its k indices of P^T, and one
// 16-byte load of a component's row in V is its part of V^T.  So probabilities
// never leave their lane, and a lane's tokens lie in one page: its scales are
// two scalars.
//
// The value scale is part of the weight: e = logit + log2(v_scale), running
// maximum M over e, weight exp2(e - M + 15) (f16 then resolves weights down to
// 2^-39 of the largest), and the denominator sums weight / v_scale.  A scale
// below kMinScale (0, say) counts as kMinScale there, so that the sum's terms,
// 2^15 / 1e-20, stay in range, and as 0 in the result: what such pages leave in
// it, at most kNothing, is far under the last bit of what an append's smallest
// scale, 7.9e-8, makes, and is taken as 0.

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kNoMax = -FLT_MAX; // running maximum of a row that has seen nothing
constexpr float kHeadroom = 15.0f; // weights are at most 2^15
constexpr float kSteady = 0x1p22f;  // of exponents: above, a product's rounding is 1/2 and more
constexpr float kMinScale = 1e-20f;
constexpr float kNothing = 127.5f * kMinScale;
constexpr int kTile = 64;          // tokens
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kMaxSplits = 256;
constexpr int kFewParts = 8;       // that 32 lanes join

struct Attend {
  Cache c;
  Batch s;
  const void *q;
  void *out;
  float *lse, *acc, *ml;  // acc [splits][rows * q_heads][dim], ml [splits][rows * q_heads][2]
  int64_t q_stride, out_stride;
  float scale;  // times log2 e
  int window;
  int q_heads, group, causal, splits;
  int least;  // token tiles of a part at least
  Divisor by_group, by_splits, by_round, by_each, by_heads, by_per_seq;  // by_each: workgroups of a sequence, starts NULL
  int blocks, round;  // workgroups along the rows of one head and part, and those that fill the compute units once
};

// A call whose scores have a shape of their own: capped (in units of log2: at
// `cap`, icap = 1 / cap; 0: not), with a bias by distance (slopes NULL: none),
// with a prefix that all rows see (prefix NULL: none).  Kernels are built for
// either argument: to those of plain scores the shape costs nothing.
struct Shaped : Attend {
  float cap, icap;
  const float *slopes;    // [q_heads]
  const int32_t *prefix;  // [seqs]
};

// v within F32's range; a NaN stays one.
__device__ inline float in_range(float v) { return fabsf(v) == INFINITY ? copysignf(FLT_MAX, v) : v; }

// A head's slope in units of log2.  One that log2 e takes out of F32's range is
// held at its end: an infinity would make distance 0 a NaN, and one token
// further on either's weight is 0.
__device__ inline float slope_of(const float *slopes, int head) { return slopes ? in_range(slopes[head] * kLog2e) : 0.0f; }

// Tokens in front of which rows of sequence b see all.
__device__ inline int prefix_of(const Attend &, int) { return 0; }
__device__ inline int prefix_of(const Shaped &a, int b) { return a.prefix ? a.prefix[b] : 0; }

// What rounding x0 and x1 to the pair left, as a pair of its own: differences
// that are exact, rounded once; one mixed-precision operation each (the compiler
// takes three for two).  It does not see what these write: settle() stands
// between them and a matrix instruction, which may read a register two wait
// states after another instruction wrote it.
__device__ inline f16x2 rest_of(float x0, float x1, f16x2 pair) {
  f16x2 r;
  asm("v_fma_mixlo_f16 %0, %1, -1.0, %2 op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(pair), "v"(x0));
  asm("v_fma_mixhi_f16 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(r) : "v"(pair), "v"(x1));
  return r;
}

__device__ inline void settle(f16x8 &a, f16x8 &b) { asm("s_nop 1" : "+v"(a), "+v"(b)); }

// What a tile of rows sees: tokens [begin, end), all of its rows [lo, hi), cut
// into `used` parts of `part` token tiles.
struct Range {
  int begin, end, lo, hi, part, used;
};

constexpr int kLeastFew = 8, kLeastMany = 4;  // token tiles of a part: shorter ones do not pay for joining

__device__ inline int clamp_int(int64_t v, int top) { return v < 0 ? 0 : v < top ? static_cast<int>(v) : top; }

// The end of what a row at position pos sees, at most top.
template <typename A>
__device__ inline int end_of(const A &a, int pos, int prefix, int top) {
  int64_t end = static_cast<int64_t>(pos) + 1;
  if constexpr (std::is_same<A, Shaped>::value) end = end > prefix ? end : prefix;
  return a.causal ? clamp_int(end, top) : top;
}

template <typename A>
__device__ inline Range range_of(const A &a, const Span &p, int first_row, int last_row) {
  const int ahead = p.len - p.n, p0 = ahead + a.by_group.of(first_row), p1 = ahead + a.by_group.of(last_row);
  const int held = a.s.blocks << a.c.lp, top = held < p.len ? held : p.len;
  Range r;
  const int prefix = prefix_of(a, p.b);
  r.hi = end_of(a, p0, prefix, top);
  r.end = end_of(a, p1, prefix, top);
  r.lo = a.window > 0 ? clamp_int(static_cast<int64_t>(p1) - a.window + 1, top) : 0;
  r.begin = (a.window > 0 ? clamp_int(static_cast<int64_t>(p0) - a.window + 1, top) : 0) & ~(kTile - 1);
  const int tiles = r.end > r.begin ? (r.end - r.begin + kTile - 1) / kTile : 0;
  r.part = a.by_splits.of(tiles + a.splits - 1);
  if (r.part < a.least) r.part = a.least;
  r.used = (tiles + r.part - 1) / r.part;
  return r;
}

// Max and sum over the four lanes that hold one row.
__device__ inline float over_lanes_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float over_lanes_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// a - b, held to the range of an int.
__device__ inline int sub_sat(int a, int b) { return __builtin_elementwise_sub_sat(a, b); }

// cap tanh(x / cap) of 16 scores, with icap = 1 / cap.  Up to kBend x / cap is
// a polynomial, which scores below 5/8 of the cap need no more of (a branch of
// the wave): tanh(y) = y + y z Q(z), z = y^2, Q fitted (least squares at Chebyshev
// nodes, reweighted to even it out) to a relative error of 2^-27.9, of 2^-26.5
// with its coefficients in F32 (at y = 0.604): x itself is only rounded once more.  Above: (1 - u) / (1 + u), u = exp(-2 |y|).
constexpr float kBend = 0.625f;

__device__ inline void capped(float (&x)[16], float cap, float icap) {
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(x[k]));
  const bool far = __any(most * icap > kBend);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float y = x[k] * icap, z = y * y;
    float q = fmaf(z, -0x1.72eedap-8f, 0x1.515cdep-6f);
    q = fmaf(q, z, -0x1.b8153ep-5f);
    q = fmaf(q, z, 0x1.110580p-3f);
    q = fmaf(q, z, -0x1.555524p-2f);
    const float near = fmaf(x[k], z * q, x[k]);
    if (far) {
      const float u = __builtin_amdgcn_exp2f(fabsf(y) * (-2.0f * kLog2e));
      const float wide = copysignf(cap * ((1.0f - u) * __builtin_amdgcn_rcpf(1.0f + u)), y);
      x[k] = fabsf(y) > kBend ? wide : near;
    } else {
      x[k] = near;
    }
  }
}

// Four codes as f16: 0x6400 + u is 1024 + u for a byte u = code + 128.
__device__ inline f16x4 codes_to_f16(int codes) {
  const uint32_t u = static_cast<uint32_t>(codes) ^ 0x80808080u;
  union {
    uint32_t w[2];
    f16x4 h;
  } r;
  r.w[0] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
  r.w[1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
  return r.h - static_cast<f16>(1152.0f);
}

// Four components of a result: o / l, with inv = 1 / l.
__device__ inline f32x4 result_of(f32x4 o, float inv) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] *= inv;
    o[i] = fabsf(o[i]) <= kNothing ? 0.0f : o[i];
  }
  return o;
}

template <typename T>
__device__ inline void store4(T *p, f32x4 v) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  T4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<T>(v[i]);
  *reinterpret_cast<T4 *>(p) = o;
}

// The sequence, rows, head and part of a workgroup.  Heads are dealt first:
// workgroups go to the 8 dies in turn, so that a die's cache holds few heads.
// Later rows see more (causal), so they are begun first, and every other round
// of workgroups over the compute units runs backwards: units that share one
// then have about the same to do between them.
struct Place {
  Span p;
  int rows, row0;  // rows of the sequence, first row of the workgroup
  int h, split;
};

__device__ inline bool place_of(const Attend &a, int block_rows, Place &w) {
  const int rest = a.c.by_heads.of(blockIdx.x), G = a.group;
  w.h = blockIdx.x - rest * a.c.heads;
  int x = a.by_splits.of(rest);
  w.split = rest - x * a.splits;
  const int turn = a.by_round.of(x);
  if ((turn & 1) && (turn + 1) * a.round <= a.blocks) x = (2 * turn + 1) * a.round - 1 - x;
  x = a.blocks - 1 - x;
  int rel;
  if (!a.s.starts) {
    const int b = a.by_each.of(x);
    rel = x - b * static_cast<int>(a.by_each.by);
    w.p = span_of(a.s, b);
  } else {
    auto key = [&](int i, int start) { return start * G / block_rows + i; };
    w.p = find(a.s, x, key);
    if (w.p.b < 0) return false;
    rel = x - key(w.p.b, w.p.first);
  }
  w.rows = w.p.n * G;
  w.row0 = rel * block_rows;
  return w.row0 < w.rows;
}

// Tokens [begin, end) of a part.
struct Part {
  int begin, end;
};

__device__ inline Part part_of(const Range &r, int split) {
  const int all = (r.end - r.begin + kTile - 1) / kTile, stop = (split + 1) * r.part;
  return {r.begin + split * r.part * kTile, stop < all ? r.begin + stop * kTile : r.end};
}

// Pages of a tile's tokens.  Loads are never conditional: the counters by
// which a wave waits for them could not tell how many are on their way.  Past
// the last tile its tokens are loaded again, holes load page 0 in their place
// (their weights are zero).
struct Pages {
  const int32_t *table;
  const int8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t bytes;  // of a page
  int heads, pages, lp, last;

  __device__ Pages(const Attend &a, int b, int h, int D, int end)
      : table(a.s.table + b * a.s.table_stride), heads(a.c.heads), pages(a.c.pages), lp(a.c.lp), last(end - 1) {
    const int64_t head = static_cast<int64_t>(D) << lp;
    bytes = heads * head;
    k = a.c.k + h * head;
    v = a.c.v + h * head;
    k_scale = a.c.k_scale + h;
    v_scale = a.c.v_scale + h;
  }
  __device__ int entry(int t) const { return table[(t < last ? t : last) >> lp]; }
  __device__ bool hole(int entry) const { return static_cast<unsigned>(entry) >= static_cast<unsigned>(pages); }
  __device__ int page(int entry) const { return hole(entry) ? 0 : entry; }
  __device__ int slot(int t) const { return t & ((1 << lp) - 1); }
};

// What a lane needs to know of its 16 tokens' scales.
struct Scales {
  float ks, vs;
  bool hole;

  __device__ void load(const Pages &p, int entry) {
    hole = p.hole(entry);
    const int64_t at = static_cast<int64_t>(p.page(entry)) * p.heads;
    ks = p.k_scale[at];
    vs = p.v_scale[at];
  }
};

// A wave's rows: queries, running statistics, results.  Lane (n, g) holds row
// n of each row tile; of a tile of tokens its logits are those of the 16
// tokens 16 g .., of a result the components 16 d + 4 g ...
template <typename A, typename T, int kChunks, bool kFull, int kRowTiles, bool kDirect, int kWeightParts>
struct Rows {
  static constexpr bool kShaped = std::is_same<A, Shaped>::value;
  static constexpr int kDigits = 4, kHalves = 2;
  static constexpr int kTerms = std::is_same<T, float>::value ? 2 : 1;    // f16 terms of a query's component
  static constexpr int kOperands = kDirect ? kHalves * kTerms : kDigits;  // of 64 components of the queries
  static constexpr int kKeys = kDirect ? kHalves : 1;                     // of 64 components of 16 keys
  static constexpr int kParts = kWeightParts;                             // f16 parts of a weight
  static constexpr int kOut = 4 * kChunks;               // 16-component tiles
  typedef typename Row<T>::Vec Vec;
  static constexpr int kVecs = 16 / Row<T>::kValues;
  union Weights {
    f16x2 pair[8];
    f16x8 half[2];
  };

  const A &a;
  const int n, g, D;
  f32x4 acc[kRowTiles][kOut];
  i32x4 q[kRowTiles][kChunks][kOperands];
  float qs[kRowTiles], m[kRowTiles], l[kRowTiles];  // m: the running maximum less kHeadroom
  int lo[kRowTiles], hi[kRowTiles];
  int row_of[kRowTiles], head_of[kRowTiles];        // row_of: -1 behind the last row
  Vec qv[kRowTiles][kChunks][kVecs];
  float slope[kShaped ? kRowTiles : 1];  // in units of log2
  int pos_of[kShaped ? kRowTiles : 1];

  __device__ Rows(const A &args)
      : a(args), n(threadIdx.x & 15), g((threadIdx.x & 63) >> 4), D(kFull ? 64 * kChunks : args.c.dim) {}

  __device__ void place(const Place &w, int row0, int end) {
    const int prefix = prefix_of(a, w.p.b);
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int row = row0 + 16 * t + n;
      const bool live = row < w.rows;
      const int i = live ? a.by_group.of(row) : 0;
      const int pos = w.p.len - w.p.n + i;
      row_of[t] = live ? w.p.first + i : -1;
      head_of[t] = w.h * a.group + (live ? row - i * a.group : 0);
      hi[t] = !live ? 0 : end_of(a, pos, prefix, end);
      if constexpr (kShaped) {
        slope[t] = slope_of(a.slopes, head_of[t]);
        pos_of[t] = pos;
      }
      lo[t] = a.window > 0 ? clamp_int(static_cast<int64_t>(pos) - a.window + 1, end) : 0;
      qs[t] = 0.0f;
      m[t] = kNoMax;
      l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < kOut; ++d) acc[t][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int z = 0; z < kOperands; ++z) q[t][c][z] = i32x4{0, 0, 0, 0};
      }
    }
  }

  __device__ void load_queries(const Place &w) {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const T *src = static_cast<const T *>(a.q) + (row_of[t] < 0 ? w.p.first : row_of[t]) * a.q_stride +
                     static_cast<int64_t>(head_of[t]) * D + 16 * g;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          qv[t][c][k] = Vec{};
          if (kFull || 64 * c + 16 * g < D) qv[t][c][k] = reinterpret_cast<const Vec *>(src + 64 * c)[k];
        }
      }
    }
  }

  // The loaded queries as operands.
  __device__ void set_queries() {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      float v[kChunks][16];
      float amax = 0.0f, nan = 0.0f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          v[c][k] = static_cast<float>(qv[t][c][k / Row<T>::kValues][k % Row<T>::kValues]);
          amax = fmaxf(amax, fabsf(v[c][k]));
          nan = fmaf(v[c][k], 0.0f, nan);  // NaN once a component is a NaN or an infinity
        }
      }
      if (nan != 0.0f) amax = INFINITY;
      amax = over_lanes_max(amax);
      // amax <= 127/128 2^over: the digits are at most 127, an f16 is below 2^15.
      const int over = __builtin_amdgcn_frexp_expf(amax * 0.504f) + 1;
      const int shift = !kDirect ? 8 * kDigits - 1 - over : std::is_same<T, f16>::value ? 0 : 15 - over;
      qs[t] = amax < INFINITY ? ldexpf(a.scale, -shift) : NAN;
      if constexpr (kShaped) qs[t] = in_range(qs[t]);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if constexpr (kDirect) {
#pragma unroll
          for (int z = 0; z < kHalves; ++z) {
            f16x8 term[kTerms];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float x = ldexpf(v[c][8 * z + k], shift);
              term[0][k] = static_cast<f16>(x);
              if constexpr (kTerms == 2) term[1][k] = static_cast<f16>(x - static_cast<float>(term[0][k]));
            }
#pragma unroll
            for (int i = 0; i < kTerms; ++i) q[t][c][z + kHalves * i] = __builtin_bit_cast(i32x4, term[i]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            // With 128 added to every digit the digits are the sum's bytes.
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = static_cast<uint32_t>(static_cast<int>(rintf(ldexpf(v[c][4 * w + k], shift)))) + 0x80808080u;
#pragma unroll
            for (int z = 0; z < kDigits; ++z) {
              const uint32_t byte = kDigits - 1 - z, pair = byte | (byte + 4) << 8 | 0x0c0c0000u;
              const uint32_t low = __builtin_amdgcn_perm(u[1], u[0], pair), high = __builtin_amdgcn_perm(u[3], u[2], pair);
              q[t][c][z][w] = static_cast<int>((low | high << 16) ^ 0x80808080u);
            }
          }
        }
      }
    }
  }

  // Dots of row tile t with 16 tokens, K's operands given.
  __device__ f32x4 dots(int t, const i32x4 (&k)[kChunks][kKeys]) const {
    if constexpr (kDirect) {
      f32x4 f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int z = 0; z < kOperands; ++z)
          f = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, k[c][z % kHalves]),
                                                     __builtin_bit_cast(f16x8, q[t][c][z]), f, 0, 0, 0);
      }
      return f;
    } else {
      i32x4 dot[kDigits];
#pragma unroll
      for (int z = 0; z < kDigits; ++z) {
        dot[z] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) dot[z] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k[c][0], q[t][c][z], dot[z], 0, 0, 0);
      }
      // Two digits' dots are an int32 together: at most 2^8 x 256 x 2^14 + 2^22.
      f32x4 f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = fmaf(static_cast<float>(dot[0][i] * 256 + dot[1][i]), 65536.0f, static_cast<float>(dot[2][i] * 256 + dot[3][i]));
      return f;
    }
  }

  // Weights of row tile t for the lane's tokens first .. first + 15, and the
  // running statistics.  edge: some row of the wave does not see them all, or
  // some are in a hole.
  __device__ void weigh(int t, const f32x4 (&f)[4], const Scales &s, int first, bool edge, Weights (&w)[kParts]) {
    if constexpr (kShaped) {
      float x[16];
      // Before a cap a score may be past F32's range.  Its factor is held to it,
      // so that a dot of 0 stays 0; the least other, 2^-24, is past every cap.
      const float factor = in_range(qs[t] * s.ks);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = f[k / 4][k % 4] * factor;
      if (a.cap > 0.0f) capped(x, a.cap, a.icap);
      if (a.slopes) {
        const float away = static_cast<float>(sub_sat(pos_of[t], first));
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = fmaf(-slope[t], fabsf(away - static_cast<float>(k)), x[k]);
      }
      f32x4 e[4];
#pragma unroll
      for (int k = 0; k < 16; ++k) e[k / 4][k % 4] = x[k];
      weigh_scaled(t, e, 1.0f, s, first, edge, w);
    } else {
      weigh_scaled(t, f, qs[t] * s.ks, s, first, edge, w);
    }
  }

  // The same for scores f * ck in units of log2.
  __device__ void weigh_scaled(int t, const f32x4 (&f)[4], float ck, const Scales &s, int first, bool edge, Weights (&w)[kParts]) {
    const float vs = s.hole ? 1.0f : fmaxf(s.vs, kMinScale);
    const float lvs = __builtin_amdgcn_logf(vs), rvs = __builtin_amdgcn_rcpf(vs);
    // Taken off the exponents: the running maximum, nothing while there is none.
    const bool unset = m[t] == kNoMax;
    const float off = unset ? 0.0f : m[t];
    float e[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) e[k] = fmaf(f[k / 4][k % 4], ck, lvs - off);
    if (edge) {
      const int under = lo[t] - first;
      const unsigned width = !s.hole && hi[t] > lo[t] ? hi[t] - lo[t] : 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        e[k] = static_cast<unsigned>(k - under) < width ? e[k] : -INFINITY;
        asm volatile("" : "+v"(e[k]));  // keeps this a branch: few tiles take it
      }
    }
    float top = e[0];
#pragma unroll
    for (int k = 1; k < 16; ++k) top = fmaxf(top, e[k]);
    if (__any(top > (unset ? -FLT_MAX : kHeadroom))) {
      top = over_lanes_max(top) + off - kHeadroom;
      const float now = fmaxf(m[t], top), shrink = __builtin_amdgcn_exp2f(m[t] - now);  // a row that has seen nothing stays unset
      m[t] = now;
      l[t] *= shrink;
#pragma unroll
      for (int d = 0; d < kOut; ++d) acc[t][d] *= shrink;
#pragma unroll
      for (int k = 0; k < 16; ++k) e[k] = e[k] == -INFINITY ? e[k] : fmaf(f[k / 4][k % 4], ck, lvs - now);
      // A maximum whose last bit is 1/2 or more misses the exponents that made it
      // by as much: the largest is set to weigh 2^15 all the same.
      const bool large = fabsf(now) > kSteady && now != kNoMax;
      if (__any(large)) {
        float most = e[0];
#pragma unroll
        for (int k = 1; k < 16; ++k) most = fmaxf(most, e[k]);
        most = over_lanes_max(most) - kHeadroom;
        most = large && (most > 0.0f || now == top) ? most : 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) e[k] -= most;
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float p0 = __builtin_amdgcn_exp2f(e[k]), p1 = __builtin_amdgcn_exp2f(e[k + 1]);
      sum += p0 + p1;
      const f16x2 near = {static_cast<f16>(p0), static_cast<f16>(p1)};
      w[0].pair[k / 2] = near;
      if constexpr (kParts == 2) w[1].pair[k / 2] = rest_of(p0, p1, near);
    }
    if constexpr (kParts == 2) settle(w[1].half[0], w[1].half[1]);
    l[t] = fmaf(sum, rvs, l[t]);
  }

  // acc += V^T P^T for 16 components and half of a tile's tokens.
  __device__ void add(int t, int d, int half, f16x8 v, const Weights (&w)[kParts]) {
#pragma unroll
    for (int z = 0; z < kParts; ++z) acc[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, w[z].half[half], acc[t][d], 0, 0, 0);
  }

  // Results of row tile t to the output, or (several parts) to the workspace:
  // value(i) gives the components of 16-component tile first + i * stride, for
  // kCount of them.
  template <int kCount, typename F>
  __device__ void store(int t, int used, int split, int first, int stride, F value) const {
    if (row_of[t] < 0) return;
    const int64_t at = static_cast<int64_t>(row_of[t]) * a.q_heads + head_of[t];
    const bool stats = first == 0 && g == 0;
    if (used > 1) {
      const int64_t row = static_cast<int64_t>(split) * a.s.rows * a.q_heads + at;
      float *to = a.acc + row * D + 4 * g;
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const int d = first + i * stride;
        if (kFull || 16 * d < D) *reinterpret_cast<f32x4 *>(to + 16 * d) = value(i);
      }
      if (stats) *reinterpret_cast<f32x2 *>(a.ml + 2 * row) = f32x2{m[t], l[t]};
    } else {
      const float inv = l[t] == 0.0f ? 0.0f : 1.0f / l[t];
      T *to = static_cast<T *>(a.out) + row_of[t] * a.out_stride + static_cast<int64_t>(head_of[t]) * D + 4 * g;
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const int d = first + i * stride;
        if (kFull || 16 * d < D) store4(to + 16 * d, result_of(value(i), inv));
      }
      if (stats && a.lse) a.lse[at] = l[t] == 0.0f ? -INFINITY : kLn2 * (m[t] + log2f(l[t]));
    }
  }
};

__device__ inline f16x8 codes_to_f16(int low, int high) {
  union {
    f16x4 part[2];
    f16x8 all;
  } v;
  v.part[0] = codes_to_f16(low);
  v.part[1] = codes_to_f16(high);
  return v.all;
}

// Few rows (a decode step): the workgroup's 4 waves share 16 rows, each takes
// every fourth tile of tokens straight into registers, and their results are
// joined through shared memory.  Bound by the cache's bytes: a tile's K is
// loaded while the tile before it is weighted and multiplied by V, its V while
// its own logits are formed, into the registers that the tile before has just
// left; the pages are looked up one tile further ahead.  64 sequences of 500 to
// 8000 tokens, 32 query heads over 8 of 128, BF16: 115 us for 559 MB (4.9 TB/s;
// a read alone reaches 5.4 to 6.4).  A single sequence of 777 tokens takes 11 us,
// latency and the fetch of instructions, one of 65536 tokens and 2 heads 12 us
// (2.9 TB/s).  Eight waves, or two tiles on their way, were slower.
// kChunks: 64-component chunks of a head, kFull: the head fills them.
template <typename A, typename T, int kChunks, bool kFull>
__global__ void __launch_bounds__(kThreads, kChunks > 2 ? 1 : 2) attention_few_kernel(A a) {
  typedef Rows<A, T, kChunks, kFull, 1, false, 2> R;
  constexpr int kOut = R::kOut, kWaves = kThreads / 64, kStep = kWaves * kTile;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  Place w;
  if (!place_of(a, 16, w)) return;
  const Range r = range_of(a, w.p, w.row0, (w.row0 + 16 < w.rows ? w.row0 + 16 : w.rows) - 1);
  if (w.split >= (r.used > 1 ? r.used : 1)) return;
  const Part part = part_of(r, w.split);
  R rows(a);
  rows.place(w, w.row0, r.end);
  const int n = rows.n, g = rows.g, D = rows.D, kgroup = 16 * (n >> 2), P = 1 << a.c.lp;

  int t0 = part.begin + wave * kTile;
  if (t0 < part.end) {
    const Pages pages(a, w.p.b, w.h, D, part.end);
    i32x4 kc[4][kChunks][1], vc[kOut];
    Scales next;
    auto load_k = [&](int t, int entry) {
      const int8_t *q = pages.k + pages.page(entry) * pages.bytes + (pages.slot(t + kgroup) + (n & 3)) * D + 16 * g;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (kFull || 64 * c + 16 * g < D) kc[j][c][0] = *reinterpret_cast<const i32x4 *>(q + 4 * j * D + 64 * c);
        }
      }
    };
    auto load_v = [&](int t, int entry) {
      const int8_t *q = pages.v + pages.page(entry) * pages.bytes + n * P + pages.slot(t + 16 * g);
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        if (kFull || 16 * d < D) vc[d] = *reinterpret_cast<const i32x4 *>(q + 16 * d * P);
      }
    };
    if (!kFull) {
#pragma unroll
      for (int d = 0; d < kOut; ++d) vc[d] = kc[d & 3][d >> 2][0] = i32x4{0, 0, 0, 0};
    }
    rows.load_queries(w);
    int kpage = pages.entry(t0 + kgroup), vpage = pages.entry(t0 + 16 * g);
    const int kthen = pages.entry(t0 + kStep + kgroup), vthen = pages.entry(t0 + kStep + 16 * g);
    load_k(t0, kpage);
    next.load(pages, vpage);
    load_v(t0, vpage);
    kpage = kthen;
    vpage = vthen;
    __builtin_amdgcn_sched_barrier(0);
    rows.set_queries();

    while (true) {
      const Scales now = next;
      f32x4 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = rows.dots(0, kc[j]);
      // The order of loads is that of their uses: what waits for one waits for
      // all before it.
      load_k(t0 + kStep, kpage);
      next.load(pages, vpage);
      kpage = pages.entry(t0 + 2 * kStep + kgroup);
      const int vthen = pages.entry(t0 + 2 * kStep + 16 * g);
      typename R::Weights weights[R::kParts];
      rows.weigh(0, f, now, t0 + 16 * g, t0 < r.lo || t0 + kTile > r.hi || __any(now.hole), weights);
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        if (!kFull && 16 * d >= D) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) rows.add(0, d, k, codes_to_f16(vc[d][2 * k], vc[d][2 * k + 1]), weights);
      }
      t0 += kStep;
      if (t0 >= part.end) break;
      load_v(t0, vpage);
      vpage = vthen;
    }
  }

  __shared__ f32x4 parts[kWaves][kOut][64];
  __shared__ float stats[kWaves][16][2];
  rows.l[0] = over_lanes_sum(rows.l[0]);
  if (g == 0) {
    stats[wave][n][0] = rows.m[0];
    stats[wave][n][1] = rows.l[0];
  }
#pragma unroll
  for (int d = 0; d < kOut; ++d) parts[wave][d][lane] = rows.acc[0][d];
  __syncthreads();
  float wm[kWaves], top = kNoMax;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    wm[k] = stats[k][n][0];
    top = fmaxf(top, wm[k]);
  }
  rows.l[0] = 0.0f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) {
    wm[k] = __builtin_amdgcn_exp2f(wm[k] - top);
    rows.l[0] = fmaf(wm[k], stats[k][n][1], rows.l[0]);
  }
  rows.m[0] = top;
  rows.template store<kOut / kWaves>(0, r.used, w.split, wave, kWaves, [&](int i) {
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k) o += wm[k] * parts[k][wave + i * kWaves][lane];
    return o;
  });
}

// Many rows (prompts, drafted tokens): each of the workgroup's 4 waves has
// kRowTiles x 16 rows of its own, and all walk the same tiles.  A wave loads a
// quarter of the next tile's operands while the present one is worked on,
// turns its part into f16 (once for the workgroup), and lays both down
// in shared memory in the order in which lanes take them: 64 lanes x 16
// bytes, free of bank conflicts.  Bound by issuing vector instructions (a
// weight's exponent, sum and f16 parts, the joining of digits) and the matrix
// products, which a wave does by turns.  A causal prompt of 4096 F32 rows, 12
// query heads over 2 of 128: 115 to 120 us, 0.44 PFLOP/s of the formula's
// operations; vector instructions are active in 58% of the SIMDs' cycles, the
// matrix units in 35%.  Six BF16 prompts of 150 to 5000 tokens, 16 query heads
// over 4 of 64, a window of 1024: 139 us, 0.48 PFLOP/s; 76% and 19%.
//
// F32 rows by digits where 48 KB of codes and V leave room for a third
// workgroup and f16 keys (64 KB) do not: one prompt of 4096 rows, 12 heads over
// 2 of 128, 118 against 120 us, chunks of 300 to 400 rows 85 against 87; with
// two row tiles (two workgroups in either form) directly: six prompts of 500 to
// 3000 rows, 16 heads over 4 of 128, 289 against 313 us.
template <typename T, int kChunks, int kRowTiles>
struct Many {
  static constexpr bool kDirect = !(std::is_same<T, float>::value && kRowTiles == 1 && kChunks > 1);
  static constexpr int kGroups = kChunks > 2 ? 1 : kDirect ? 2 : 3;  // workgroups on a unit, at least
};

// f16 parts of a weight where rows are many.
template <typename A, typename T>
constexpr int kManyParts = std::is_same<T, bf16>::value && !std::is_same<A, Shaped>::value ? 1 : 2;

template <typename A, typename T, int kChunks, bool kFull, int kRowTiles>
__global__ void __launch_bounds__(kThreads, (Many<T, kChunks, kRowTiles>::kGroups)) attention_many_kernel(A a) {
  constexpr bool kDirect = Many<T, kChunks, kRowTiles>::kDirect;
  typedef Rows<A, T, kChunks, kFull, kRowTiles, kDirect, kManyParts<A, T>> R;
  constexpr int kOut = R::kOut, kRows = 16 * kRowTiles, kBlock = 4 * kRows;
  __shared__ i32x4 lk[2][4][kChunks][R::kKeys][64];
  __shared__ f16x8 lv[2][kOut][2][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  Place w;
  if (!place_of(a, kBlock, w)) return;
  const int last = (w.row0 + kBlock < w.rows ? w.row0 + kBlock : w.rows) - 1;
  const Range r = range_of(a, w.p, w.row0, last);
  if (w.split >= (r.used > 1 ? r.used : 1)) return;
  const Part part = part_of(r, w.split);
  R rows(a);
  const int row0 = w.row0 + wave * kRows;
  rows.place(w, row0, r.end);
  const int n = rows.n, g = rows.g, D = rows.D, kgroup = 16 * (n >> 2), P = 1 << a.c.lp;

  if (part.begin < part.end) {
    // Every row of this wave sees tokens own.lo .. own.hi - 1.
    const Range own = range_of(a, w.p, row0 <= last ? row0 : last, row0 + kRows - 1 < last ? row0 + kRows - 1 : last);
    const Pages pages(a, w.p.b, w.h, D, part.end);
    i32x4 kc[kChunks], vc[kChunks];  // K's operand `wave`, V's components wave, wave + 4, ...
    const bool whole = P >= kTile;  // a tile lies in one page
    const int kplace = ((whole ? kgroup : 0) + (n & 3) + 4 * wave) * D + 16 * g, vplace = (n + 16 * wave) * P + (whole ? 16 * g : 0);
    auto load = [&](int t, int kentry, int ventry) {
      const int8_t *k, *v;
      if (whole) {  // its address is the workgroup's
        const int64_t at = pages.page(__builtin_amdgcn_readfirstlane(kentry)) * pages.bytes;
        k = pages.k + at + pages.slot(t) * D + kplace;
        v = pages.v + at + pages.slot(t) + vplace;
      } else {
        k = pages.k + pages.page(kentry) * pages.bytes + pages.slot(t + kgroup) * D + kplace;
        v = pages.v + pages.page(ventry) * pages.bytes + pages.slot(t + 16 * g) + vplace;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (kFull || 64 * c + 16 * g < D) kc[c] = *reinterpret_cast<const i32x4 *>(k + 64 * c);
        if (kFull || 16 * (4 * c + wave) < D) vc[c] = *reinterpret_cast<const i32x4 *>(v + 64 * c * P);
      }
    };
    auto lay_down = [&](int to) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if constexpr (kDirect) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            lk[to][wave][c][k][lane] = __builtin_bit_cast(i32x4, codes_to_f16(kc[c][2 * k], kc[c][2 * k + 1]));
        } else {
          lk[to][wave][c][0][lane] = kc[c];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) lv[to][4 * c + wave][k][lane] = codes_to_f16(vc[c][2 * k], vc[c][2 * k + 1]);
      }
    };
    if (!kFull) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) kc[c] = vc[c] = i32x4{0, 0, 0, 0};
    }
    rows.load_queries(w);
    int t0 = part.begin;
    Scales now, next;
    int kpage = pages.entry(t0 + kgroup), vpage = pages.entry(t0 + 16 * g);
    int vnext = pages.entry(t0 + kTile + 16 * g);
    const int knext = pages.entry(t0 + kTile + kgroup);
    load(t0, kpage, vpage);
    now.load(pages, vpage);
    __builtin_amdgcn_sched_barrier(0);
    rows.set_queries();
    lay_down(0);
    load(t0 + kTile, knext, vnext);
    kpage = pages.entry(t0 + 2 * kTile + kgroup);
    vpage = pages.entry(t0 + 2 * kTile + 16 * g);
    __syncthreads();

    // What is carried on to the next round in other registers is loaded at a
    // round's begin: the copies at its end then wait for nothing.
    int kthen, vthen;
    auto begin_round = [&]() {
      next.load(pages, vnext);
      kthen = pages.entry(t0 + 3 * kTile + kgroup);
      vthen = pages.entry(t0 + 3 * kTile + 16 * g);
    };
    auto pass_on = [&](int to) {
      lay_down(to);
      load(t0 + 2 * kTile, kpage, vpage);
    };
    auto end_round = [&]() {
      vnext = vpage;
      kpage = kthen;
      vpage = vthen;
      now = next;
      __syncthreads();
    };
    if (row0 > last) {  // no rows: this wave only fetches for the others
      for (int from = 0; t0 < part.end; t0 += kTile, from ^= 1) {
        begin_round();
        pass_on(from ^ 1);
        end_round();
      }
      return;
    }
    for (int from = 0; t0 < part.end; t0 += kTile, from ^= 1) {
      begin_round();
      typename R::Weights weights[kRowTiles][R::kParts];
      const bool edge = t0 < own.lo || t0 + kTile > own.hi || __any(now.hole);
      f32x4 f[kRowTiles][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        i32x4 k[kChunks][R::kKeys];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int z = 0; z < R::kKeys; ++z) k[c][z] = lk[from][j][c][z][lane];
        }
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t) f[t][j] = rows.dots(t, k);
      }
#pragma unroll
      for (int t = 0; t < kRowTiles; ++t) rows.weigh(t, f[t], now, t0 + 16 * g, edge, weights[t]);
      pass_on(from ^ 1);
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        if (!kFull && 16 * d >= D) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f16x8 v = lv[from][d][h][lane];
#pragma unroll
          for (int t = 0; t < kRowTiles; ++t) rows.add(t, d, h, v, weights[t]);
        }
      }
      end_round();
    }
  }
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) {
    rows.l[t] = over_lanes_sum(rows.l[t]);
    rows.template store<kOut>(t, r.used, w.split, 0, 1, [&](int d) { return rows.acc[t][d]; });
  }
}

// Joins the parts of rows that were split.

// The parts that the row and head at place `at` was cut into.
template <typename A>
__device__ inline int parts_of(const A &a, const Span &p, int row, int hq, int block_rows) {
  const int h = a.by_group.of(hq), in_group = (row - p.first) * a.group + hq - h * a.group;
  const int row0 = in_group & -block_rows;  // a power of two
  const int rows = p.n * a.group;
  return range_of(a, p, row0, (row0 + block_rows < rows ? row0 + block_rows : rows) - 1).used;
}

// Few parts (at most kFewParts): 32 lanes a row and head, four components each.
// block_rows: rows of the attention's workgroups.
template <typename A, typename T>
__global__ void __launch_bounds__(kThreads) join_few_kernel(A a, int block_rows) {
  const int each = a.s.rows * a.q_heads, item = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int row = a.by_heads.of(item < each ? item : each - 1), hq = item - row * a.q_heads, D = a.c.dim;
  // A wave's two items may lie in neighbouring rows, and these in two sequences
  // or the first in front of all: then each row's sequence is looked for.
  Span p;
  if (!a.s.starts) {
    p = span_of(a.s, a.by_per_seq.of(row));
  } else {
    auto key = [](int, int start) { return start; };
    const int first = __builtin_amdgcn_readlane(row, 0), second = __builtin_amdgcn_readlane(row, 32);
    p = find(a.s, first, key);
    if (second != first) {
      const Span other = find(a.s, second, key);
      if (row == second) p = other;
    }
  }
  const bool live = item < each && p.b >= 0 && row >= p.first && row < p.first + p.n;
  const int used = live ? parts_of(a, p, row, hq, block_rows) : 0;
  if (used <= 1) return;
  const float *ml = a.ml + 2 * static_cast<int64_t>(item), *acc = a.acc + static_cast<int64_t>(item) * D;
  f32x2 v[kFewParts];
  float now = kNoMax, l = 0.0f;
#pragma unroll
  for (int k = 0; k < kFewParts; ++k) {
    v[k] = f32x2{kNoMax, 0.0f};
    if (k < used) v[k] = *reinterpret_cast<const f32x2 *>(ml + 2 * k * static_cast<int64_t>(each));
    now = fmaxf(now, v[k][0]);
  }
#pragma unroll
  for (int k = 0; k < kFewParts; ++k) {
    v[k][0] = __builtin_amdgcn_exp2f(v[k][0] - now);
    l = fmaf(v[k][0], v[k][1], l);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  T *out = static_cast<T *>(a.out) + row * a.out_stride + static_cast<int64_t>(hq) * D;
  for (int c = lane; c < D / 4; c += 32) {
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kFewParts; ++k)
      if (k < used) o += v[k][0] * *reinterpret_cast<const f32x4 *>(acc + k * static_cast<int64_t>(each) * D + 4 * c);
    store4(out + 4 * c, result_of(o, inv));
  }
  if (a.lse && lane == 0) a.lse[item] = l == 0.0f ? -INFINITY : kLn2 * (now + log2f(l));
}

// Many parts: a workgroup a row and head; its threads hold the parts' weights,
// and eight groups of 32 lanes each sum every eighth part.
template <typename A, typename T>
__global__ void __launch_bounds__(kThreads) join_many_kernel(A a, int block_rows) {
  static_assert(kMaxSplits == kThreads, "a thread holds one part's weight");
  __shared__ f32x4 sums[8][KV8_MAX_DIM / 4];
  __shared__ float weight[kMaxSplits], red[4], sl[4];
  const int row = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x, D = a.c.dim;
  const Span p = a.s.starts ? find(a.s, row, [](int, int start) { return start; }) : span_of(a.s, a.by_per_seq.of(row));
  if (p.b < 0 || row >= p.first + p.n) return;
  const int used = parts_of(a, p, row, hq, block_rows);
  if (used <= 1) return;
  const int64_t each = static_cast<int64_t>(a.s.rows) * a.q_heads, at = static_cast<int64_t>(row) * a.q_heads + hq;
  const f32x2 v = tid < used ? *reinterpret_cast<const f32x2 *>(a.ml + 2 * (tid * each + at)) : f32x2{kNoMax, 0.0f};
  float now = wave_max(v[0]);
  if ((tid & 63) == 0) red[tid >> 6] = now;
  __syncthreads();
  now = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  weight[tid] = __builtin_amdgcn_exp2f(v[0] - now);
  float l = weight[tid] * v[1];
#pragma unroll
  for (int k = 1; k < 64; k *= 2) l += __shfl_xor(l, k);
  if ((tid & 63) == 0) sl[tid >> 6] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const int team = tid >> 5;
  for (int c = tid & 31; c < D / 4; c += 32) {
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k = team; k < used; k += 8) o += weight[k] * *reinterpret_cast<const f32x4 *>(a.acc + (k * each + at) * D + 4 * c);
    sums[team][c] = o;
  }
  __syncthreads();
  if (tid < D / 4) {
    f32x4 o = sums[0][tid];
#pragma unroll
    for (int k = 1; k < 8; ++k) o += sums[k][tid];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    store4(static_cast<T *>(a.out) + row * a.out_stride + static_cast<int64_t>(hq) * D + 4 * tid, result_of(o, inv));
  }
  if (a.lse && tid == 0) a.lse[at] = l == 0.0f ? -INFINITY : kLn2 * (now + log2f(l));
}
// How an attention call is laid out: 16-row tiles of a wave (0: four waves
// share one), rows of a workgroup, and into how many parts tokens are cut.
struct Plan {
  int row_tiles, block_rows, splits, least;
  int64_t blocks;  // workgroups along the rows
  double us;       // what it is thought to take
};

// The plan with row_tiles given.  Microseconds, as measured for 128 F32
// components: a wave's walk over a tile of 64 tokens takes 1.9 alone (64 rows
// of a workgroup), 1.2 where four waves take every fourth tile; a full card
// does one of 16 rows in 1.15e-3, or 1.6e-3 where each wave turns V for itself
// and 1.05e-3 for two at a time; joining takes 5 and writing and reading a
// part of all rows at 4 TB/s.
inline Plan plan_for(int row_tiles, const Cache &c, const Batch &s, int64_t len, int64_t q_heads) {
  const int64_t group = q_heads / c.heads;
  Plan p;
  p.row_tiles = row_tiles;
  p.block_rows = row_tiles ? 64 * row_tiles : 16;
  p.blocks = s.starts ? s.rows * group / p.block_rows + s.seqs
                      : (s.per_seq * group + p.block_rows - 1) / p.block_rows * s.seqs;
  // Up to two least parts are not worth a second launch (777 tokens: 11.0 us
  // whole, 8.7 + 4.5 us in two parts).
  p.least = row_tiles ? kLeastMany : kLeastFew;
  int64_t splits = (row_tiles ? 4 : 8) * kUnits / (p.blocks * c.heads);
  const int64_t most = len <= 2 * kTile * p.least ? 1 : (len + kTile * p.least - 1) / (kTile * p.least);
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  const double tiles = static_cast<double>(len) / kTile, walk = tiles * (row_tiles ? 1.9 : 0.3);
  const double part = 8e-6 * s.rows * q_heads * c.dim / 4;
  if (splits > 1) {  // many rows are many partial results
    const int64_t best = static_cast<int64_t>(sqrt(walk / part));
    if (splits > best) splits = best;
    if (splits <= 1 || walk / splits + 5.0 + part * splits >= walk) splits = 1;
  }
  p.splits = static_cast<int>(splits);
  const double full = tiles * s.rows * q_heads / 16 * (c.dim + 64) / 192 *
                      (row_tiles == 0 ? 1.6e-3 : row_tiles == 1 ? 1.15e-3 : 1.05e-3);
  p.us = (walk / splits > full ? walk / splits : full) + (splits > 1 ? 5.0 + part * splits : 0.0);
  return p;
}

// Positions are below kMaxRows: a window of that many tokens or more is none.
inline int64_t window_of(int64_t window) { return window < kMaxRows ? window : 0; }

// The workspace is sized without a window, which only takes parts away.
inline Plan plan_of(const Cache &c, const Batch &s, int64_t max_len, int64_t q_heads, int64_t window, bool causal) {
  const int64_t group = q_heads / c.heads, rows = s.rows * group / s.seqs;  // of a sequence, on average
  const int64_t held = static_cast<int64_t>(s.blocks) << c.lp;
  if (max_len <= 0 || max_len > held) max_len = held;
  // Over 26 calls each of 48 to 128, to 512 and of more rows a sequence, lengths
  // drawn up to 4096 and beyond, the kernel for few rows took 1.38, 1.27 and 1.97
  // times (floor + 8 us) in the mean, that for many 1.37, 1.42 and 1.91, the
  // one of the lower estimate 1.34, 1.26 and 1.69.
  Plan best = plan_for(0, c, s, max_len, q_heads);
  if (rows > 16) {
    // Two tiles of rows a wave read and turn V half as often, one leaves more
    // workgroups to balance: 16 heads of width 64, prompts of 150 to 5000
    // tokens in BF16, 139 against 152 us; 12 heads of width 128, one prompt of
    // 4096 tokens in F32 (386 workgroups of two tiles), 129 against 116 us.
    Plan many = plan_for(2, c, s, max_len, q_heads);
    if (c.dim > 128 || rows <= 64 || many.blocks * c.heads < 4 * kUnits) many = plan_for(1, c, s, max_len, q_heads);
    if (many.us < best.us) best = many;
  }
  if (window > 0 && best.splits > 1) {  // fewer tokens to walk
    const int64_t seen = window + kTile + (causal ? best.block_rows / group + 1 : s.rows);
    if (seen < max_len) {
      const int splits = plan_for(best.row_tiles, c, s, seen, q_heads).splits;
      if (splits < best.splits) best.splits = splits;
    }
  }
  return best;
}

// Checks shared by kv8_attention and its workspace's size.
inline int check_attention(const kv8_cache *cache, const kv8_batch *batch, int type, int64_t q_heads, int64_t rows, Cache &c,
                    Batch &s) {
  if (const int st = check_batch(cache, batch, type, rows, c, s)) return st;
  if (q_heads < 1 || q_heads % c.heads) return I2S_EINVAL;
  if (q_heads > 65535 || rows * (q_heads / c.heads) > kMaxRows - 4 * KV8_MAX_PAGE ||
      (static_cast<int64_t>(s.blocks) << c.lp) > kMaxRows - 4 * KV8_MAX_PAGE)
    return I2S_ERANGE;
  return I2S_OK;
}

inline size_t workspace_of(const Plan &p, const Cache &c, const Batch &s, int64_t q_heads) {
  return p.splits > 1 ? static_cast<size_t>(p.splits) * s.rows * q_heads * (c.dim + 2) * sizeof(float) : 0;
}

template <typename T, int kChunks, bool kFull, typename A>
int launch_attention(const Plan &p, const A &a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.blocks * a.c.heads * p.splits);
  if (p.row_tiles == 0) {
    attention_few_kernel<A, T, kChunks, kFull><<<grid, kThreads, 0, stream>>>(a);
  } else if (p.row_tiles == 1) {
    attention_many_kernel<A, T, kChunks, kFull, 1><<<grid, kThreads, 0, stream>>>(a);
  } else if constexpr (kChunks <= 2) {  // two row tiles fit the registers, see plan_of
    attention_many_kernel<A, T, kChunks, kFull, 2><<<grid, kThreads, 0, stream>>>(a);
  }
  return hip_status();
}

// Rows, outputs and workspace of a call.
struct Rowset {
  const void *q;
  int64_t q_stride, q_heads, rows;
  void *out;
  int64_t out_stride;
  float *lse;
  void *workspace;
  size_t workspace_bytes;
};

// The call itself: what is left to check, the plan and the launches.
template <typename A>
int attend(A &a, const kv8_batch *batch, int type, const Rowset &r, float scale, int causal, int64_t window, void *stream) {
  if (window < 0 || !(fabsf(scale) < INFINITY)) return I2S_EINVAL;
  if (r.rows == 0 || a.s.seqs == 0) return I2S_OK;
  const int64_t width = r.q_heads * a.c.dim;
  if (const int st = check_rows(r.q, r.q_stride, width, value_bytes(type))) return st;
  if (const int st = check_rows(r.out, r.out_stride, width, value_bytes(type))) return st;
  if (!aligned(r.lse, 4)) return I2S_EINVAL;
  const Plan p = plan_of(a.c, a.s, batch->max_len, r.q_heads, window_of(window), causal != 0);
  if (p.blocks * a.c.heads * p.splits > 0x7fffffff || r.rows * r.q_heads > 0x7fffffff) return I2S_ERANGE;
  const size_t need = workspace_of(p, a.c, a.s, r.q_heads);
  if (need > 0 && (!r.workspace || r.workspace_bytes < need || !aligned(r.workspace, 256))) return I2S_EWORKSPACE;
  a.q = r.q;
  a.out = r.out;
  a.lse = r.lse;
  a.acc = static_cast<float *>(r.workspace);
  a.ml = need ? a.acc + static_cast<int64_t>(p.splits) * r.rows * r.q_heads * a.c.dim : nullptr;
  a.q_stride = r.q_stride;
  a.out_stride = r.out_stride;
  a.window = static_cast<int>(window_of(window));
  a.scale = scale * kLog2e;
  a.q_heads = static_cast<int>(r.q_heads);
  a.group = static_cast<int>(r.q_heads / a.c.heads);
  a.causal = causal != 0;
  a.by_group = Divisor(a.group);
  a.by_splits = Divisor(p.splits);
  a.by_heads = Divisor(a.q_heads);
  a.by_per_seq = Divisor(a.s.per_seq > 0 ? a.s.per_seq : 1);
  const int64_t each = (a.s.per_seq * static_cast<int64_t>(a.group) + p.block_rows - 1) / p.block_rows;
  a.by_each = Divisor(each > 0 ? static_cast<int>(each) : 1);
  a.splits = p.splits;
  a.least = p.least;
  a.blocks = static_cast<int>(p.blocks);
  a.round = kUnits / (a.c.heads * p.splits) > 1 ? kUnits / (a.c.heads * p.splits) : 1;
  a.by_round = Divisor(a.round);
  const hipStream_t on = static_cast<hipStream_t>(stream);
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    const int st = a.c.dim == 128  ? launch_attention<T, 2, true>(p, a, on)
                   : a.c.dim == 64 ? launch_attention<T, 1, true>(p, a, on)
                   : a.c.dim < 64  ? launch_attention<T, 1, false>(p, a, on)
                   : a.c.dim < 128 ? launch_attention<T, 2, false>(p, a, on)
                                   : launch_attention<T, 4, false>(p, a, on);
    if (st || p.splits == 1) return st;
    if (p.splits > kFewParts) {
      join_many_kernel<A, T><<<dim3(static_cast<unsigned>(r.rows), a.q_heads), kThreads, 0, on>>>(a, p.block_rows);
    } else {
      join_few_kernel<A, T><<<static_cast<unsigned>((r.rows * r.q_heads + 7) / 8), kThreads, 0, on>>>(a, p.block_rows);
    }
    return hip_status();
  });
}

}  // namespace
