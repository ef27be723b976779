// gfx950 (MI355X) kernels and C ABI of attention over an int8 K/V cache:
// rotation with per-head norms, the quantizing cache write, its read-back and
// the attention itself.  The ABI is declared, with its contract, in
// include/kv8.h.
//
// Every float operation that decides a code (the scale's division, x / s,
// q * ratio) is one IEEE operation: the library is built without fast-math and
// without FP contraction, and '/' is the correctly rounded division, so the
// cache's bytes match the definition bit for bit.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "kv8.h"

namespace {

constexpr int kThreads = 256;  // 4 wave64s
constexpr float kAmaxFloor = 1e-5f;
constexpr int64_t kMaxSeqs = 1 << 20;
constexpr int64_t kMaxRows = 0x7fffffff;

typedef _Float16 f16;
typedef __bf16 bf16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Row {  // 16 bytes of a row
  static constexpr int kValues = 16 / sizeof(T);
  typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
};

// 16 / sizeof(T) consecutive values, 16-byte aligned, as F32.
template <typename T>
__device__ inline void load16(const T *p, float *out) {
  const typename Row<T>::Vec v = *reinterpret_cast<const typename Row<T>::Vec *>(p);
#pragma unroll
  for (int i = 0; i < Row<T>::kValues; ++i) out[i] = static_cast<float>(v[i]);
}

// The same number of values, rounded to nearest even, to 16 aligned bytes.
template <typename T>
__device__ inline void store16(T *p, const float *in) {
  typename Row<T>::Vec v;
#pragma unroll
  for (int i = 0; i < Row<T>::kValues; ++i) v[i] = static_cast<T>(in[i]);
  *reinterpret_cast<typename Row<T>::Vec *>(p) = v;
}

template <int CTRL>
__device__ inline float dpp_move(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}

// Max over the wave, in every lane (the order of a maximum's terms is free).
__device__ inline float wave_max(float v) {
  v = fmaxf(v, dpp_move<0xB1>(v));   // quad_perm(1,0,3,2)
  v = fmaxf(v, dpp_move<0x4E>(v));   // quad_perm(2,3,0,1)
  v = fmaxf(v, dpp_move<0x141>(v));  // row_half_mirror
  v = fmaxf(v, dpp_move<0x140>(v));  // row_mirror
  const int b = __float_as_int(v);
  return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               fmaxf(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
}

__device__ inline float block_max(float v, float *red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// x rounded half away from zero, as a code.
__device__ inline int code_of(float x) {
  return static_cast<int>(fminf(fmaxf(roundf(x), -127.0f), 127.0f));
}

// ---------------------------------------------------------------------------
// The batch on the device.

struct Batch {
  const int32_t *table, *lens, *starts;
  int64_t table_stride;
  int blocks, seqs, rows, per_seq;  // per_seq: rows of each sequence where starts is NULL
};

struct Span {
  int b, first, n, len;  // sequence, its first row, its rows, its tokens
};

__device__ inline int start_of(const Batch &s, int b) {
  if (!s.starts) return b * s.per_seq;
  const int v = s.starts[b];
  return v < 0 ? 0 : v < s.rows ? v : s.rows;
}

__device__ inline Span span_of(const Batch &s, int b) {
  Span p;
  p.b = b;
  p.first = start_of(s, b);
  const int end = start_of(s, b + 1);
  p.n = end > p.first ? end - p.first : 0;
  const int len = s.lens[b];
  p.len = len > 0 ? len : 0;
  return p;
}

// The last sequence whose key(b) is at most x (-1: none), for a rising key,
// found 64 candidates at a time by the wave; every lane gets it.
template <typename Key>
__device__ inline int last_at_most(int seqs, int x, Key key) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = seqs;
  while (true) {
    const int step = (hi - lo + 63) >> 6;
    const int64_t i = lo + static_cast<int64_t>(lane) * step;
    const int count = __popcll(__ballot(i < hi && key(static_cast<int>(i < hi ? i : lo)) <= x));
    if (count == 0) return -1;
    lo += (count - 1) * step;
    hi = hi < lo + step ? hi : lo + step;
    if (step == 1) return lo;
  }
}

// Page of block j of sequence b, or -1 for a hole.
__device__ inline int page_of(const Batch &s, int b, int64_t j, int pages) {
  if (j >= s.blocks) return -1;
  const int p = s.table[b * s.table_stride + j];
  return p >= 0 && p < pages ? p : -1;
}

// A grid of page slots: sequence b has the slots from key(b) = start(b) / P +
// 2 b on.  n rows lie in at most n / P + 2 pages, so the slots of different
// sequences are distinct and rows / P + 2 seqs of them suffice, whatever the
// device's starts say.
__device__ inline bool slot_of(const Batch &s, int lp, int x, Span &p, int64_t &j) {
  int b, rel;
  if (!s.starts) {
    const int per = ((s.per_seq + (1 << lp) - 2) >> lp) + 1;
    b = x / per;
    rel = x - b * per;
    if (b >= s.seqs) return false;
  } else {
    b = last_at_most(s.seqs, x, [&](int i) { return (start_of(s, i) >> lp) + 2 * i; });
    if (b < 0) return false;
    rel = x - ((start_of(s, b) >> lp) + 2 * b);
  }
  p = span_of(s, b);
  const int done = p.len - p.n;
  j = static_cast<int64_t>((done > 0 ? done : 0) >> lp) + rel;
  return true;
}

struct Cache {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int pages, heads, dim, lp;
};

// ---------------------------------------------------------------------------
// Append.  One workgroup per (page slot, head) and K or V: the maximum of the
// page's new values, the page's scale, then the codes.

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(Cache c, Batch s, const T *__restrict__ kx, int64_t k_stride,
                                                          const T *__restrict__ vx, int64_t v_stride) {
  extern __shared__ int8_t tile[];  // V: [new tokens][dim] codes
  __shared__ float red[4];
  Span p;
  int64_t j;
  if (!slot_of(s, c.lp, blockIdx.x, p, j)) return;
  const int P = 1 << c.lp, D = c.dim, h = blockIdx.y;
  const int64_t done = static_cast<int64_t>(p.len) - p.n, begin = j << c.lp;
  int64_t t0 = done > begin ? done : begin, t1 = begin + P;
  if (t0 < 0) t0 = 0;
  if (t1 > p.len) t1 = p.len;
  if (t0 >= t1) return;
  const int page = page_of(s, p.b, j, c.pages);
  if (page < 0) return;
  const bool value = blockIdx.z != 0;
  const int64_t stride = value ? v_stride : k_stride;
  const T *src = (value ? vx : kx) + (p.first + (t0 - done)) * stride + static_cast<int64_t>(h) * D;
  const int64_t at = static_cast<int64_t>(page) * c.heads + h;
  float *scale = (value ? c.v_scale : c.k_scale) + at;
  int8_t *codes = (value ? c.v : c.k) + at * P * D;
  const int n = static_cast<int>(t1 - t0), lo = static_cast<int>(t0 - begin), per = D / 16, units = n * per;

  float amax = 0.0f;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    const T *q = src + (u / per) * stride + (u % per) * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; i += Row<T>::kValues) load16(q + i, x + i);
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
  }
  amax = block_max(amax, red);
  float now = fmaxf(amax, kAmaxFloor) / 127.0f, ratio = 1.0f;
  bool grown = false;
  if (lo > 0) {
    const float before = *scale;
    if (now > before) {
      grown = true;
      ratio = before / now;
    } else if (before >= now) {  // a scale that is no number counts for nothing
      now = before;
    }
  }
  __syncthreads();  // the old scale is read before it is written
  if (threadIdx.x == 0) *scale = now;

  for (int u = threadIdx.x; u < units; u += kThreads) {
    const int t = u / per, d = (u % per) * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; i += Row<T>::kValues) load16(src + t * stride + d + i, x + i);
    union {
      int8_t b[16];
      i32x4 v;
    } q;
#pragma unroll
    for (int i = 0; i < 16; ++i) q.b[i] = static_cast<int8_t>(code_of(x[i] / now));
    int8_t *to = value ? tile + t * D + d : codes + (lo + t) * D + d;
    *reinterpret_cast<i32x4 *>(to) = q.v;
  }
  if (!value) {
    if (grown) {
      for (int u = threadIdx.x; u < lo * per; u += kThreads) {
        union {
          int8_t b[16];
          i32x4 v;
        } q;
        q.v = reinterpret_cast<i32x4 *>(codes)[u];
#pragma unroll
        for (int i = 0; i < 16; ++i) q.b[i] = static_cast<int8_t>(roundf(static_cast<float>(q.b[i]) * ratio));
        reinterpret_cast<i32x4 *>(codes)[u] = q.v;
      }
    }
    return;
  }
  __syncthreads();
  const int chunks = P / 16;  // of a component's row, 16 tokens each
  for (int u = threadIdx.x; u < D * chunks; u += kThreads) {
    const int d = u / chunks, s0 = (u % chunks) * 16;
    const bool has_new = s0 < lo + n && s0 + 16 > lo, has_old = s0 < lo;
    if (!has_new && !(grown && has_old)) continue;
    union {
      int8_t b[16];
      i32x4 v;
    } q;
    i32x4 *to = reinterpret_cast<i32x4 *>(codes + d * P + s0);
    q.v = *to;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int slot = s0 + i;
      if (slot < lo) {
        if (grown) q.b[i] = static_cast<int8_t>(roundf(static_cast<float>(q.b[i]) * ratio));
      } else if (slot < lo + n) {
        q.b[i] = tile[(slot - lo) * D + d];
      }
    }
    *to = q.v;
  }
}

// ---------------------------------------------------------------------------
// Read back.  One workgroup per (page slot, head); V's codes are turned
// through shared memory.

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(Cache c, Batch s, T *__restrict__ ko, int64_t k_stride,
                                                        T *__restrict__ vo, int64_t v_stride) {
  extern __shared__ int8_t tile[];  // [P][dim]
  Span p;
  int64_t j;
  if (!slot_of(s, c.lp, blockIdx.x, p, j)) return;
  const int P = 1 << c.lp, D = c.dim, h = blockIdx.y, per = D / 16;
  const int64_t done = static_cast<int64_t>(p.len) - p.n, begin = j << c.lp;
  ko += static_cast<int64_t>(h) * D;
  vo += static_cast<int64_t>(h) * D;
  float zero[16] = {};
  if (done < 0 && begin == 0) {  // rows in front of position 0
    const int64_t ahead = -done < p.n ? -done : p.n;
    for (int64_t u = threadIdx.x; u < ahead * per; u += kThreads) {
      const int64_t row = p.first + u / per, d = (u % per) * 16;
#pragma unroll
      for (int i = 0; i < 16; i += Row<T>::kValues) {
        store16(ko + row * k_stride + d + i, zero);
        store16(vo + row * v_stride + d + i, zero);
      }
    }
  }
  int64_t t0 = done > begin ? done : begin, t1 = begin + P;
  if (t0 < 0) t0 = 0;
  if (t1 > p.len) t1 = p.len;
  if (t0 >= t1) return;
  const int page = page_of(s, p.b, j, c.pages);
  const int n = static_cast<int>(t1 - t0), lo = static_cast<int>(t0 - begin);
  const int64_t row0 = p.first + (t0 - done), at = static_cast<int64_t>(page) * c.heads + h;
  float ks = 0.0f, vs = 0.0f;
  if (page >= 0) {
    ks = c.k_scale[at];
    vs = c.v_scale[at];
    const int chunks = P / 16;
    for (int u = threadIdx.x; u < D * chunks; u += kThreads) {
      const int d = u / chunks, s0 = (u % chunks) * 16;
      union {
        int8_t b[16];
        i32x4 v;
      } q;
      q.v = *reinterpret_cast<const i32x4 *>(c.v + at * P * D + d * P + s0);
#pragma unroll
      for (int i = 0; i < 16; ++i) tile[(s0 + i) * D + d] = q.b[i];
    }
    __syncthreads();
  }
  for (int u = threadIdx.x; u < n * per; u += kThreads) {
    const int t = u / per, d = (u % per) * 16;
    union {
      int8_t b[16];
      i32x4 v;
    } qk, qv;
    qk.v = qv.v = i32x4{0, 0, 0, 0};
    if (page >= 0) {
      qk.v = *reinterpret_cast<const i32x4 *>(c.k + at * P * D + (lo + t) * D + d);
      qv.v = *reinterpret_cast<const i32x4 *>(tile + (lo + t) * D + d);
    }
    float xk[16], xv[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      xk[i] = static_cast<float>(qk.b[i]) * ks;
      xv[i] = static_cast<float>(qv.b[i]) * vs;
    }
#pragma unroll
    for (int i = 0; i < 16; i += Row<T>::kValues) {
      store16(ko + (row0 + t) * k_stride + d + i, xk + i);
      store16(vo + (row0 + t) * v_stride + d + i, xv + i);
    }
  }
}

// ---------------------------------------------------------------------------
// Attention.
//
// A wave owns kRowTiles x 16 rows (row = query token and head of the K/V
// head's group, so that a group shares what is read of the cache) and walks
// tiles of 64 tokens.  Everything stays in registers, operands are loaded
// straight into the order of the matrix instructions:
//   S^T = K Q^T   int8 16x16x64.  The codes are exact, a query is held as
//     kDigits signed base-256 digits of its row's largest magnitude (3 for
//     F32 rows: 23 bits; 2 for 16-bit rows: 15 bits, of which their own
//     mantissas fill 8 or 11), and the int32 dots are exact.
//   O^T = V^T P^T  f16 16x16x32.  V's codes are exact in f16; a weight is one
//     f16 (16-bit rows) or a sum of two (F32 rows: 22 bits).
// The rows of K's four 16-token operands are taken from the tile in the order
// 16 (m / 4) + 4 j + m % 4, which leaves lane (row, g) with the logits of the
// 16 consecutive tokens 16 g ..: those are its k indices of P^T, and one
// 16-byte load of a component's row in V is its part of V^T.  So probabilities
// never leave their lane, and a lane's tokens lie in one page: its scales are
// two scalars.
//
// The value scale is part of the weight: e = logit + log2(v_scale), running
// maximum M over e, weight exp2(e - M + 15) (f16 then resolves weights down to
// 2^-39 of the largest), and the denominator sums weight / v_scale.

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kNoMax = -1e30f;   // running maximum of a row that has seen nothing
constexpr float kHeadroom = 15.0f; // weights are at most 2^15
constexpr float kMinScale = 1e-30f;
constexpr int kTile = 64;          // tokens

struct Attend {
  Cache c;
  Batch s;
  const void *q;
  void *out;
  float *lse, *acc, *ml;  // acc [splits][rows * q_heads][dim], ml [splits][rows * q_heads][2]
  int64_t q_stride, out_stride, window;
  float scale;  // times log2 e
  int q_heads, group, causal, splits;
};

// What a tile of rows sees: tokens [begin, end), all of its rows [lo, hi), cut
// into `used` parts of `part` token tiles.
struct Range {
  int begin, end, lo, hi, part, used;
};

constexpr int kMinPart = 4;  // token tiles of a part: shorter ones do not pay for joining

__device__ inline int clamp_int(int64_t v, int top) { return v < 0 ? 0 : v < top ? static_cast<int>(v) : top; }

__device__ inline Range range_of(const Attend &a, const Span &p, int first_row, int last_row) {
  const int64_t ahead = static_cast<int64_t>(p.len) - p.n;
  const int64_t p0 = ahead + first_row / a.group, p1 = ahead + last_row / a.group;
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len;
  Range r;
  r.hi = a.causal ? clamp_int(p0 + 1, top) : top;
  r.end = a.causal ? clamp_int(p1 + 1, top) : top;
  r.lo = a.window > 0 ? clamp_int(p1 - a.window + 1, top) : 0;
  r.begin = (a.window > 0 ? clamp_int(p0 - a.window + 1, top) : 0) & ~(kTile - 1);
  const int tiles = r.end > r.begin ? (r.end - r.begin + kTile - 1) / kTile : 0;
  r.part = (tiles + a.splits - 1) / a.splits;
  if (r.part < kMinPart) r.part = kMinPart;
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

template <typename T>
__device__ inline void store4(T *p, f32x4 v) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  T4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<T>(v[i]);
  *reinterpret_cast<T4 *>(p) = o;
}

// kChunks: 64-component chunks of a head (the head may end inside the last);
// kTeam: the workgroup's 4 waves share the rows and take every fourth tile,
// joined through shared memory; otherwise each has rows of its own.
template <typename T, int kChunks, int kRowTiles, bool kTeam>
__global__ void __launch_bounds__(kThreads) attention_kernel(Attend a) {
  constexpr int kDigits = sizeof(T) == 4 ? 3 : 2;
  constexpr int kParts = sizeof(T) == 4 ? 2 : 1;  // f16 parts of a weight
  constexpr int kOut = 4 * kChunks;               // 16-component tiles
  constexpr int kRows = 16 * kRowTiles;
  constexpr int kBlockRows = kTeam ? kRows : 4 * kRows;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n = lane & 15, g = lane >> 4;
  const int h = blockIdx.y, split = blockIdx.z, G = a.group, D = a.c.dim, P = 1 << a.c.lp;

  // Later rows see more: they are begun first.
  const int x = gridDim.x - 1 - blockIdx.x;
  int b, rel;
  if (!a.s.starts) {
    const int per = (a.s.per_seq * G + kBlockRows - 1) / kBlockRows;
    b = x / per;
    rel = x - b * per;
  } else {
    auto key = [&](int i) { return start_of(a.s, i) * G / kBlockRows + i; };
    b = last_at_most(a.s.seqs, x, key);
    if (b < 0) return;
    rel = x - key(b);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  rel = __builtin_amdgcn_readfirstlane(rel);
  const Span p = span_of(a.s, b);
  const int rows = p.n * G, row0 = rel * kBlockRows + (kTeam ? 0 : wave * kRows);
  if (row0 >= rows) return;
  const int last = (row0 + kRows < rows ? row0 + kRows : rows) - 1;
  const Range r = range_of(a, p, row0, last);
  if (split >= (r.used > 1 ? r.used : 1)) return;
  const int all = (r.end - r.begin + kTile - 1) / kTile, stop = (split + 1) * r.part;
  const int end = stop < all ? r.begin + stop * kTile : r.end;

  // Queries, as digits.
  i32x4 q[kRowTiles][kChunks][kDigits];
  float qs[kRowTiles];
  int lo[kRowTiles], hi[kRowTiles];
  int64_t at[kRowTiles];  // row * q_heads + head, or -1
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) {
    const int row = row0 + 16 * t + n;
    const bool live = row < rows;
    const int i = live ? row / G : 0, hq = h * G + (live ? row - i * G : 0);
    const int64_t pos = static_cast<int64_t>(p.len) - p.n + i;
    at[t] = live ? static_cast<int64_t>(p.first + i) * a.q_heads + hq : -1;
    hi[t] = !live ? 0 : a.causal ? clamp_int(pos + 1, r.end) : r.end;
    lo[t] = a.window > 0 ? clamp_int(pos - a.window + 1, r.end) : 0;
    const T *src = static_cast<const T *>(a.q) + (p.first + i) * a.q_stride + static_cast<int64_t>(hq) * D;
    float v[kChunks][16];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int d = 64 * c + 16 * g;
#pragma unroll
      for (int k = 0; k < 16; ++k) v[c][k] = 0.0f;
      if (live && d < D) {
#pragma unroll
        for (int k = 0; k < 16; k += Row<T>::kValues) load16(src + d + k, &v[c][k]);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = fabsf(v[c][k]) < INFINITY ? fmaxf(amax, fabsf(v[c][k])) : INFINITY;
    }
    amax = over_lanes_max(amax);
    constexpr float kTop = kDigits == 3 ? 127.0f * 65536.0f : 127.0f * 256.0f;
    const float inv = amax > kMinScale && amax < INFINITY ? kTop / amax : 0.0f;
    qs[t] = amax < INFINITY ? (amax > kMinScale ? amax / kTop * a.scale : 0.0f) : NAN;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t word[3] = {0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          int rest = static_cast<int>(rintf(v[c][4 * w + k] * inv));
#pragma unroll
          for (int z = kDigits - 1; z >= 0; --z) {
            const int digit = static_cast<int8_t>(rest);
            word[z] |= (static_cast<uint32_t>(digit) & 0xffu) << (8 * k);
            rest = (rest - digit) >> 8;
          }
        }
#pragma unroll
        for (int z = 0; z < kDigits; ++z) q[t][c][z][w] = static_cast<int>(word[z]);
      }
    }
  }

  f32x4 acc[kRowTiles][kOut] = {};
  float m[kRowTiles], l[kRowTiles];  // m: the running maximum less kHeadroom
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) {
    m[t] = kNoMax;
    l[t] = 0.0f;
  }

  const int64_t page_bytes = static_cast<int64_t>(a.c.heads) * P * D;
  const int8_t *kbase = a.c.k + static_cast<int64_t>(h) * P * D, *vbase = a.c.v + static_cast<int64_t>(h) * P * D;
  const int step = kTeam ? 4 * kTile : kTile;
  auto page_at = [&](int t) { return t < r.end ? page_of(a.s, b, t >> a.c.lp, a.c.pages) : -1; };
  int t0 = r.begin + split * r.part * kTile + (kTeam ? wave * kTile : 0);
  int kpage = -1, vpage = -1;
  if (t0 < end) {
    kpage = page_at(t0 + 16 * (n >> 2));
    vpage = page_at(t0 + 16 * g);
  }
  for (; t0 < end; t0 += step) {
    // Holes load page 0 in their place; their weights are zero.
    const bool hole = vpage < 0;
    const int64_t kp = kpage < 0 ? 0 : kpage, vp = hole ? 0 : vpage;
    const float ks = hole ? 0.0f : a.c.k_scale[vp * a.c.heads + h];
    const float vs = hole ? 1.0f : fmaxf(a.c.v_scale[vp * a.c.heads + h], kMinScale);
    const int kslot = ((t0 + 16 * (n >> 2)) & (P - 1)) + (n & 3);
    const int8_t *kptr = kbase + kp * page_bytes + kslot * D + 16 * g;
    const int8_t *vptr = vbase + vp * page_bytes + n * P + ((t0 + 16 * g) & (P - 1));
    i32x4 kc[4][kChunks], vc[kOut];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        kc[j][c] = i32x4{0, 0, 0, 0};
        if (64 * c + 16 * g < D) kc[j][c] = *reinterpret_cast<const i32x4 *>(kptr + 4 * j * D + 64 * c);
      }
    }
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
      vc[d] = i32x4{0, 0, 0, 0};
      if (16 * d < D) vc[d] = *reinterpret_cast<const i32x4 *>(vptr + 16 * d * P);
    }
    if (t0 + step < end) {
      kpage = page_at(t0 + step + 16 * (n >> 2));
      vpage = page_at(t0 + step + 16 * g);
    }
    const float lvs = hole ? -INFINITY : __log2f(vs), rvs = 1.0f / vs;
    const bool edge = t0 < r.lo || t0 + kTile > r.hi;

    union Weights {
      f16x2 pair[8];
      f16x8 half[2];
    } w[kRowTiles][kParts];
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      float f[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        i32x4 dot[kDigits];
#pragma unroll
        for (int z = 0; z < kDigits; ++z) {
          dot[z] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            dot[z] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kc[j][c], q[t][c][z], dot[z], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kDigits == 3) {
            f[4 * j + i] = fmaf(static_cast<float>(dot[0][i]), 65536.0f, static_cast<float>(dot[1][i] * 256 + dot[2][i]));
          } else {
            f[4 * j + i] = static_cast<float>(dot[0][i] * 256 + dot[1][i]);
          }
        }
      }
      const float ck = qs[t] * ks;
      float e[16];
      auto exponents = [&](float base) {
#pragma unroll
        for (int k = 0; k < 16; ++k) e[k] = fmaf(f[k], ck, base);
        if (edge) {
          const int under = lo[t] - (t0 + 16 * g), over = hi[t] - (t0 + 16 * g);
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] = k >= under && k < over ? e[k] : -INFINITY;
        }
        float top = e[0];
#pragma unroll
        for (int k = 1; k < 16; ++k) top = fmaxf(top, e[k]);
        return top;
      };
      float top = exponents(lvs - m[t]);
      if (__any(top > kHeadroom)) {
        top = over_lanes_max(exponents(lvs)) - kHeadroom;
        const float now = fmaxf(m[t], top), shrink = __builtin_amdgcn_exp2f(m[t] - now);
        m[t] = now;
        l[t] *= shrink;
#pragma unroll
        for (int d = 0; d < kOut; ++d) acc[t][d] *= shrink;
        exponents(lvs - now);
      }
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float p0 = __builtin_amdgcn_exp2f(e[k]), p1 = __builtin_amdgcn_exp2f(e[k + 1]);
        sum += p0 + p1;
        const f16x2 near = {static_cast<f16>(p0), static_cast<f16>(p1)};
        w[t][0].pair[k / 2] = near;
        if (kParts == 2)
          w[t][kParts - 1].pair[k / 2] = f16x2{static_cast<f16>(p0 - static_cast<float>(near[0])),
                                               static_cast<f16>(p1 - static_cast<float>(near[1]))};
      }
      l[t] = fmaf(sum, rvs, l[t]);
    }
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
      if (16 * d >= D) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        union {
          f16x4 part[2];
          f16x8 all;
        } v;
        v.part[0] = codes_to_f16(vc[d][2 * k]);
        v.part[1] = codes_to_f16(vc[d][2 * k + 1]);
#pragma unroll
        for (int t = 0; t < kRowTiles; ++t) {
#pragma unroll
          for (int z = 0; z < kParts; ++z)
            acc[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v.all, w[t][z].half[k], acc[t][d], 0, 0, 0);
        }
      }
    }
  }

  // The lanes' sums, then (a team) the waves' results.
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) l[t] = over_lanes_sum(l[t]);
  auto finish = [&](int t, int d, f32x4 o) {
    if (at[t] < 0 || 16 * d >= D) return;
    const int c = 16 * d + 4 * g;
    if (r.used > 1) {
      const int64_t row = static_cast<int64_t>(split) * a.s.rows * a.q_heads + at[t];
      *reinterpret_cast<f32x4 *>(a.acc + row * D + c) = o;
      if (d == 0 && g == 0) {
        a.ml[2 * row] = m[t];
        a.ml[2 * row + 1] = l[t];
      }
    } else {
      const float inv = l[t] == 0.0f ? 0.0f : 1.0f / l[t];
      const int64_t row = at[t] / a.q_heads, hq = at[t] - row * a.q_heads;
      store4(static_cast<T *>(a.out) + row * a.out_stride + hq * D + c, o * inv);
      if (d == 0 && g == 0 && a.lse) a.lse[at[t]] = l[t] == 0.0f ? -INFINITY : 0.69314718055994531f * (m[t] + log2f(l[t]));
    }
  };
  if constexpr (kTeam) {
    __shared__ f32x4 parts[4][kOut][64];
    __shared__ float stats[4][16][2];
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      if (t > 0) __syncthreads();
      if (g == 0) {
        stats[wave][n][0] = m[t];
        stats[wave][n][1] = l[t];
      }
#pragma unroll
      for (int d = 0; d < kOut; ++d) parts[wave][d][lane] = acc[t][d];
      __syncthreads();
      float wm[4], wl[4], now = kNoMax;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wm[k] = stats[k][n][0];
        wl[k] = stats[k][n][1];
        now = fmaxf(now, wm[k]);
      }
      l[t] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wm[k] = __builtin_amdgcn_exp2f(wm[k] - now);
        l[t] = fmaf(wm[k], wl[k], l[t]);
      }
      m[t] = now;
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        if ((d & 3) != wave) continue;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k) o += wm[k] * parts[k][d][lane];
        finish(t, d, o);
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
#pragma unroll
      for (int d = 0; d < kOut; ++d) finish(t, d, acc[t][d]);
    }
  }
}

// Joins the parts of rows that were split: one workgroup per row and head,
// waves over parts, lanes over components.  unit: rows of the attention's tile.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(Attend a, int unit) {
  __shared__ float sums[4][KV8_MAX_DIM], sl[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row = blockIdx.x, hq = blockIdx.y, D = a.c.dim;
  int b;
  if (a.s.starts) {
    b = last_at_most(a.s.seqs, row, [&](int i) { return start_of(a.s, i); });
    if (b < 0) return;
  } else {
    b = row / a.s.per_seq;
  }
  const Span p = span_of(a.s, b);
  if (row >= p.first + p.n) return;
  const int in_group = (row - p.first) * a.group + hq % a.group, row0 = in_group / unit * unit;
  const int rows = p.n * a.group;
  const Range r = range_of(a, p, row0, (row0 + unit < rows ? row0 + unit : rows) - 1);
  if (r.used <= 1) return;
  const int64_t each = static_cast<int64_t>(a.s.rows) * a.q_heads, at = static_cast<int64_t>(row) * a.q_heads + hq;
  float now = kNoMax;
  for (int k = lane; k < r.used; k += 64) now = fmaxf(now, a.ml[2 * (k * each + at)]);
  now = wave_max(now);
  float l = 0.0f, o[KV8_MAX_DIM / 64] = {};
  for (int k = wave; k < r.used; k += 4) {
    const int64_t from = k * each + at;
    const float w = __builtin_amdgcn_exp2f(a.ml[2 * from] - now);
    l = fmaf(w, a.ml[2 * from + 1], l);
#pragma unroll
    for (int i = 0; i < KV8_MAX_DIM / 64; ++i)
      if (lane + 64 * i < D) o[i] = fmaf(w, a.acc[from * D + lane + 64 * i], o[i]);
  }
#pragma unroll
  for (int i = 0; i < KV8_MAX_DIM / 64; ++i) sums[wave][lane + 64 * i] = o[i];
  if (lane == 0) sl[wave] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  for (int d = threadIdx.x; d < D; d += kThreads)
    static_cast<T *>(a.out)[row * a.out_stride + static_cast<int64_t>(hq) * D + d] =
        static_cast<T>(((sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d])) * inv);
  if (a.lse && threadIdx.x == 0) a.lse[at] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (now + log2f(l));
}

// ---------------------------------------------------------------------------
// Norm and rotation.  A wave takes one row and a share of its heads.  A lane
// holds 32 bytes of a head: the two halves of its pairs (16 bytes at i and 16
// at i + pairs), or 32 neighbouring bytes, so a rotation never leaves its
// lane; only the norm's sum crosses lanes.

template <typename T, bool kNeighbours>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const T *__restrict__ q, int64_t q_stride, int q_heads, const T *__restrict__ k, int64_t k_stride,
                int k_heads, const int32_t *__restrict__ pos, const float *__restrict__ inv_freq, int pairs,
                const float *__restrict__ q_weight, const float *__restrict__ k_weight, float eps, T *q_out,
                int64_t q_out_stride, T *k_out, int64_t k_out_stride, int rows, int dim, int lanes_log, int split) {
  constexpr int V = Row<T>::kValues;
  __shared__ float2 turn[kThreads / 64][KV8_MAX_DIM / 2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + wave;
  const int64_t row = item / split;
  if (row < rows) {
    for (int i = lane; i < pairs; i += 64) {
      // The angle in turns, 64 bits: positions far along a context keep their
      // fraction; what is left of the fraction's rounding is 2^-26 of a turn.
      double t = static_cast<double>(pos[row]) * static_cast<double>(inv_freq[i]) * 0.15915494309189533577;
      t -= rint(t);
      float sn, cs;
      sincospif(static_cast<float>(t) * 2.0f, &sn, &cs);
      turn[wave][i] = make_float2(cs, sn);
    }
  }
  __syncthreads();
  if (row >= rows) return;
  const int per = 64 >> lanes_log, c = lane & ((1 << lanes_log) - 1), sub = lane >> lanes_log;
  const int q_groups = (q_heads + per - 1) / per, groups = q_groups + (k_heads + per - 1) / per;
  const bool rotated = c < pairs / V;
  int a0, a1;
  if (!rotated) {
    a0 = 2 * c * V;
    a1 = a0 + V;
  } else if (kNeighbours) {
    a0 = 2 * c * V;
    a1 = a0 + V;
  } else {
    a0 = c * V;
    a1 = pairs + c * V;
  }
  float cs[V], sn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 r = rotated ? turn[wave][c * V + i] : make_float2(1.0f, 0.0f);
    cs[i] = r.x;
    sn[i] = r.y;
  }
  for (int g = static_cast<int>(item - row * split); g < groups; g += split) {
    const bool key = g >= q_groups;
    const int head = (key ? g - q_groups : g) * per + sub;
    const bool live = head < (key ? k_heads : q_heads) && 2 * c * V < dim;
    const float *weight = key ? k_weight : q_weight;
    float x[2 * V] = {};
    if (live) {
      const T *p = (key ? k + row * k_stride : q + row * q_stride) + static_cast<int64_t>(head) * dim;
      load16(p + a0, x);
      load16(p + a1, x + V);
    }
    if (weight) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) ss += x[i] * x[i];
      if (lanes_log > 0) ss += dpp_move<0xB1>(ss);
      if (lanes_log > 1) ss += dpp_move<0x4E>(ss);
      if (lanes_log > 2) ss += dpp_move<0x141>(ss);
      if (lanes_log > 3) ss += dpp_move<0x140>(ss);
      if (lanes_log > 4) ss += __shfl_xor(ss, 16);
      const float r = 1.0f / sqrtf(ss / static_cast<float>(dim) + eps);
      if (live) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[i] = x[i] * r * weight[a0 + i];
          x[V + i] = x[V + i] * r * weight[a1 + i];
        }
      }
    }
    if (!live) continue;
    float y[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int iu = kNeighbours ? 2 * i : i, iv = kNeighbours ? 2 * i + 1 : V + i;
      const float u = x[iu], v = x[iv];
      y[iu] = rotated ? u * cs[i] - v * sn[i] : u;
      y[iv] = rotated ? v * cs[i] + u * sn[i] : v;
    }
    T *o = (key ? k_out + row * k_out_stride : q_out + row * q_out_stride) + static_cast<int64_t>(head) * dim;
    store16(o + a0, y);
    store16(o + a1, y + V);
  }
}

// ---------------------------------------------------------------------------
// Host side.

inline int hip_status() { return hipGetLastError() == hipSuccess ? I2S_OK : I2S_EHIP; }
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int value_bytes(int type) { return type == KV8_F32 ? 4 : type == KV8_F16 || type == KV8_BF16 ? 2 : 0; }

inline bool bad_rows(const void *p, int64_t stride, int64_t width, int size) {
  return !p || !aligned(p, 16) || stride < width || (stride * size) % 16 != 0;
}

int check_batch(const kv8_cache *c, const kv8_batch *b, int type, int64_t rows, Cache &dc, Batch &db) {
  if (!c || !b || !value_bytes(type) || rows < 0) return I2S_EINVAL;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !aligned(c->k, 16) || !aligned(c->v, 16) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || c->pages < 1 || c->heads < 1)
    return I2S_EINVAL;
  if (c->dim < 16 || c->dim > KV8_MAX_DIM || c->dim % 16 || c->page_tokens < 16 || c->page_tokens > KV8_MAX_PAGE ||
      (c->page_tokens & (c->page_tokens - 1)))
    return I2S_EALIGN;
  if (b->seqs < 0 || b->blocks < 0 || b->table_stride < b->blocks || b->max_len < 0) return I2S_EINVAL;
  if (c->pages > 0x7fffffff || c->heads > 1024 || b->seqs > kMaxSeqs || b->blocks > 0x7fffffff || rows > kMaxRows ||
      b->table_stride > (INT64_C(1) << 40))
    return I2S_ERANGE;
  if (b->seqs > 0 && (!b->lens || !aligned(b->lens, 4) || (b->blocks > 0 && !b->table) || !aligned(b->table, 4) ||
                      !aligned(b->starts, 4)))
    return I2S_EINVAL;
  if (b->seqs > 0 && !b->starts && rows % b->seqs) return I2S_EINVAL;
  dc.k = c->k;
  dc.v = c->v;
  dc.k_scale = c->k_scale;
  dc.v_scale = c->v_scale;
  dc.pages = static_cast<int>(c->pages);
  dc.heads = c->heads;
  dc.dim = c->dim;
  dc.lp = __builtin_ctz(c->page_tokens);
  db.table = b->table;
  db.lens = b->lens;
  db.starts = b->starts;
  db.table_stride = b->table_stride;
  db.blocks = static_cast<int>(b->blocks);
  db.seqs = static_cast<int>(b->seqs);
  db.rows = static_cast<int>(rows);
  db.per_seq = b->seqs > 0 ? static_cast<int>(rows / b->seqs) : 0;
  return I2S_OK;
}

// Page slots of a batch: see slot_of.
inline int64_t slots(const Batch &s, int lp) {
  if (s.starts) return (s.rows >> lp) + 2 * static_cast<int64_t>(s.seqs);
  return static_cast<int64_t>(s.seqs) * (((s.per_seq + (INT64_C(1) << lp) - 2) >> lp) + 1);
}

// How an attention call is laid out: rows of a wave, whether a workgroup's
// waves share them, and into how many parts the tokens are cut.
struct Plan {
  int row_tiles, splits;
  bool team;
  int64_t blocks;  // workgroups along the rows
};

Plan plan_of(const Cache &c, const Batch &s, int64_t max_len, int64_t q_heads) {
  const int64_t group = q_heads / c.heads, rows = s.rows * group / s.seqs;  // of a sequence, on average
  Plan p;
  p.team = rows <= 64;
  p.row_tiles = rows <= 16 || c.dim > 128 ? 1 : 2;
  const int64_t unit = 16 * p.row_tiles * (p.team ? 1 : 4);
  p.blocks = s.starts ? s.rows * group / unit + s.seqs : (s.per_seq * group + unit - 1) / unit * s.seqs;
  const int64_t held = static_cast<int64_t>(s.blocks) << c.lp;
  if (max_len <= 0 || max_len > held) max_len = held;
  const int64_t most = (max_len + kTile * kMinPart - 1) / (kTile * kMinPart);
  int64_t splits = 1024 / (p.blocks * c.heads);
  if (splits > most) splits = most;
  if (splits > 1024) splits = 1024;
  p.splits = splits < 1 ? 1 : static_cast<int>(splits);
  return p;
}

// Checks shared by kv8_attention and its workspace's size.
int check_attention(const kv8_cache *cache, const kv8_batch *batch, int type, int64_t q_heads, int64_t rows, Cache &c,
                    Batch &s) {
  if (const int st = check_batch(cache, batch, type, rows, c, s)) return st;
  if (q_heads < 1 || q_heads % c.heads) return I2S_EINVAL;
  if (q_heads > 65535 || rows * (q_heads / c.heads) > kMaxRows ||
      (static_cast<int64_t>(s.blocks) << c.lp) > kMaxRows - 4 * KV8_MAX_PAGE)
    return I2S_ERANGE;
  return I2S_OK;
}

inline size_t workspace_of(const Plan &p, const Cache &c, const Batch &s, int64_t q_heads) {
  return p.splits > 1 ? static_cast<size_t>(p.splits) * s.rows * q_heads * (c.dim + 2) * sizeof(float) : 0;
}

template <typename T, int kChunks>
int launch_attention(const Plan &p, const Attend &a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.blocks), a.c.heads, p.splits);
  constexpr int kMost = kChunks > 2 ? 1 : 2;  // row tiles that fit the registers
  if (p.team && p.row_tiles == 1) {
    attention_kernel<T, kChunks, 1, true><<<grid, kThreads, 0, stream>>>(a);
  } else if (p.team) {
    attention_kernel<T, kChunks, kMost, true><<<grid, kThreads, 0, stream>>>(a);
  } else {
    attention_kernel<T, kChunks, kMost, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return hip_status();
}

template <typename F>
int by_type(int type, F f) {
  if (type == KV8_F32) return f(float());
  if (type == KV8_F16) return f(f16());
  return f(bf16());
}

}  // namespace

extern "C" int kv8_append(const kv8_cache *cache, const kv8_batch *batch, int type, const void *k, int64_t k_stride,
                          const void *v, int64_t v_stride, int64_t rows, void *stream) {
  Cache c;
  Batch s;
  if (const int st = check_batch(cache, batch, type, rows, c, s)) return st;
  if (rows == 0 || s.seqs == 0) return I2S_OK;
  const int64_t width = static_cast<int64_t>(c.heads) * c.dim;
  if (bad_rows(k, k_stride, width, value_bytes(type)) || bad_rows(v, v_stride, width, value_bytes(type))) return I2S_EINVAL;
  const int64_t n = slots(s, c.lp);
  if (n > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    append_kernel<T><<<dim3(static_cast<unsigned>(n), c.heads, 2), kThreads, static_cast<size_t>(c.dim) << c.lp,
                       static_cast<hipStream_t>(stream)>>>(c, s, static_cast<const T *>(k), k_stride,
                                                           static_cast<const T *>(v), v_stride);
    return hip_status();
  });
}

extern "C" int kv8_read(const kv8_cache *cache, const kv8_batch *batch, int type, void *k, int64_t k_stride, void *v,
                        int64_t v_stride, int64_t rows, void *stream) {
  Cache c;
  Batch s;
  if (const int st = check_batch(cache, batch, type, rows, c, s)) return st;
  if (rows == 0 || s.seqs == 0) return I2S_OK;
  const int64_t width = static_cast<int64_t>(c.heads) * c.dim;
  if (bad_rows(k, k_stride, width, value_bytes(type)) || bad_rows(v, v_stride, width, value_bytes(type))) return I2S_EINVAL;
  const int64_t n = slots(s, c.lp);
  if (n > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    read_kernel<T><<<dim3(static_cast<unsigned>(n), c.heads), kThreads, static_cast<size_t>(c.dim) << c.lp,
                     static_cast<hipStream_t>(stream)>>>(c, s, static_cast<T *>(k), k_stride, static_cast<T *>(v), v_stride);
    return hip_status();
  });
}

extern "C" size_t kv8_attention_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch, int64_t q_heads,
                                                int64_t rows) {
  Cache c;
  Batch s;
  if (check_attention(cache, batch, KV8_F32, q_heads, rows, c, s) || rows == 0 || s.seqs == 0) return 0;
  return workspace_of(plan_of(c, s, batch->max_len, q_heads), c, s, q_heads);
}

extern "C" int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, int type, const void *q, int64_t q_stride,
                             int64_t q_heads, int64_t rows, float scale, int causal, int64_t window, void *out,
                             int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  Attend a;
  if (const int st = check_attention(cache, batch, type, q_heads, rows, a.c, a.s)) return st;
  if (window < 0 || !(fabsf(scale) < INFINITY)) return I2S_EINVAL;
  if (rows == 0 || a.s.seqs == 0) return I2S_OK;
  const int64_t width = q_heads * a.c.dim;
  if (bad_rows(q, q_stride, width, value_bytes(type)) || bad_rows(out, out_stride, width, value_bytes(type)) ||
      !aligned(lse, 4))
    return I2S_EINVAL;
  const Plan p = plan_of(a.c, a.s, batch->max_len, q_heads);
  if (p.blocks > 0x7fffffff) return I2S_ERANGE;
  const size_t need = workspace_of(p, a.c, a.s, q_heads);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I2S_EWORKSPACE;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.acc = static_cast<float *>(workspace);
  a.ml = need ? a.acc + static_cast<int64_t>(p.splits) * rows * q_heads * a.c.dim : nullptr;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.window = window;
  a.scale = scale * 1.44269504088896341f;
  a.q_heads = static_cast<int>(q_heads);
  a.group = static_cast<int>(q_heads / a.c.heads);
  a.causal = causal != 0;
  a.splits = p.splits;
  const hipStream_t on = static_cast<hipStream_t>(stream);
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    const int st = a.c.dim <= 64    ? launch_attention<T, 1>(p, a, on)
                   : a.c.dim <= 128 ? launch_attention<T, 2>(p, a, on)
                                    : launch_attention<T, 4>(p, a, on);
    if (st || p.splits == 1) return st;
    join_kernel<T><<<dim3(static_cast<unsigned>(rows), a.q_heads), kThreads, 0, on>>>(a, 16 * p.row_tiles);
    return hip_status();
  });
}

extern "C" int kv8_qk_norm_rope(int type, int64_t rows, int64_t dim, const void *q, int64_t q_stride, int64_t q_heads,
                                const void *k, int64_t k_stride, int64_t k_heads, const int32_t *pos,
                                const float *inv_freq, int64_t pairs, int neighbours, const float *q_weight,
                                const float *k_weight, float eps, void *q_out, int64_t q_out_stride, void *k_out,
                                int64_t k_out_stride, void *stream) {
  const int size = value_bytes(type);
  if (!size || rows < 0 || q_heads < 0 || k_heads < 0 || pairs < 0 || !(eps >= 0.0f)) return I2S_EINVAL;
  if (dim < 16 || dim > KV8_MAX_DIM || dim % 16 || pairs % 8 || 2 * pairs > dim) return I2S_EALIGN;
  if (rows > kMaxRows || q_heads > 65535 || k_heads > 65535) return I2S_ERANGE;
  if (rows == 0 || q_heads + k_heads == 0) return I2S_OK;
  if (q_heads > 0 && (bad_rows(q, q_stride, q_heads * dim, size) || bad_rows(q_out, q_out_stride, q_heads * dim, size)))
    return I2S_EINVAL;
  if (k_heads > 0 && (bad_rows(k, k_stride, k_heads * dim, size) || bad_rows(k_out, k_out_stride, k_heads * dim, size)))
    return I2S_EINVAL;
  if (!pos || !aligned(pos, 4) || (pairs > 0 && !inv_freq) || !aligned(inv_freq, 4) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4))
    return I2S_EINVAL;
  const int chunks = static_cast<int>(dim) * size / 32;
  int lanes_log = 0;
  while ((1 << lanes_log) < chunks) ++lanes_log;
  const int64_t per = 64 >> lanes_log, groups = (q_heads + per - 1) / per + (k_heads + per - 1) / per;
  // Few rows: a wave for each group of heads that fit it; many: a wave per
  // row, which then turns its angles once.
  int64_t split = (2048 + rows - 1) / rows;
  if (split > groups) split = groups;
  const int64_t blocks = (rows * split + kThreads / 64 - 1) / (kThreads / 64);
  if (blocks > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    auto launch = [&](auto kernel) {
      kernel<<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(
          static_cast<const T *>(q), q_stride, static_cast<int>(q_heads), static_cast<const T *>(k), k_stride,
          static_cast<int>(k_heads), pos, inv_freq, static_cast<int>(pairs), q_weight, k_weight, eps,
          static_cast<T *>(q_out), q_out_stride, static_cast<T *>(k_out), k_out_stride, static_cast<int>(rows),
          static_cast<int>(dim), lanes_log, static_cast<int>(split));
    };
    if (neighbours) {
      launch(rope_kernel<T, true>);
    } else {
      launch(rope_kernel<T, false>);
    }
    return hip_status();
  });
}
