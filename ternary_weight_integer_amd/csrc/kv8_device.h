// What the gfx950 kernels over the int8 K/V cache share: rows, codes, the batch
// and the cache on the device, and the host's checks of them.
#pragma once

#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kv8.h"

namespace {

constexpr int kThreads = 256;  // 4 wave64s
constexpr int kUnits = 256;        // compute units
constexpr int kFillWaves = 8 * kUnits;
constexpr float kAmaxFloor = 1e-5f;
constexpr int64_t kMaxSeqs = 1 << 20;
constexpr int64_t kMaxRows = 0x7fffffff;

typedef _Float16 f16;
typedef __bf16 bf16;
typedef float f32x2 __attribute__((ext_vector_type(2)));
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

// x rounded half away from zero, as a code.
__device__ inline int code_of(float x) {
  return static_cast<int>(fminf(fmaxf(roundf(x), -127.0f), 127.0f));
}

// ---------------------------------------------------------------------------
// Division of non-negative ints by a divisor that the host knows: its
// reciprocal to 32 bits past the divisor's own, rounded up (exact for 31-bit
// dividends), a multiplication where the hardware has none for '/'.
struct Divisor {
  uint32_t by, mul, shift;

  Divisor() = default;
  explicit Divisor(int d) : by(static_cast<uint32_t>(d)), mul(0), shift(0) {
    while ((uint64_t{1} << shift) < by) ++shift;
    // ceil(2^(31 + shift) / by) < 2^32: by > 2^(shift - 1)
    mul = static_cast<uint32_t>(((uint64_t{1} << (31 + shift)) + by - 1) / by);
  }
  __device__ int of(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> 31 >> shift);
  }
};

// The batch on the device.

struct Batch {
  const int32_t *table, *lens, *starts;
  int64_t table_stride;
  int blocks, seqs, rows, per_seq;  // per_seq: rows of each sequence where starts is NULL
  Divisor slots_each;               // page slots of a sequence then
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

// The sequence that holds place x of a grid: the last whose key(b, start(b))
// is at most x, for a rising key (b = -1: none).  Up to 63 sequences are
// looked at in one load of starts and lengths, whose latency is all that a
// workgroup then waits for; more are searched 64 candidates at a time.
template <typename Key>
__device__ inline Span find(const Batch &s, int x, Key key) {
  const int lane = threadIdx.x & 63;
  if (s.seqs < 64) {
    const int v = start_of(s, lane < s.seqs ? lane : s.seqs);
    const int len = s.lens[lane < s.seqs ? lane : 0];
    const int count = __popcll(__ballot(lane < s.seqs && key(lane, v) <= x));
    Span p;
    p.b = count - 1;
    const int b = count > 0 ? count - 1 : 0;
    p.first = __builtin_amdgcn_readlane(v, b);
    const int n = __builtin_amdgcn_readlane(v, b + 1) - p.first, l = __builtin_amdgcn_readlane(len, b);
    p.n = n > 0 ? n : 0;
    p.len = l > 0 ? l : 0;
    return p;
  }
  int lo = 0, hi = s.seqs;
  while (true) {
    const int step = (hi - lo + 63) >> 6;
    const int64_t i = lo + static_cast<int64_t>(lane) * step;
    const int at = static_cast<int>(i < hi ? i : lo);
    const int count = __popcll(__ballot(i < hi && key(at, start_of(s, at)) <= x));
    if (count == 0) {
      Span p = {-1, 0, 0, 0};
      return p;
    }
    lo += (count - 1) * step;
    hi = hi < lo + step ? hi : lo + step;
    if (step == 1) break;
  }
  return span_of(s, __builtin_amdgcn_readfirstlane(lo));
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
  int rel;
  if (!s.starts) {
    const int b = s.slots_each.of(x);
    rel = x - b * static_cast<int>(s.slots_each.by);
    if (b >= s.seqs) return false;
    p = span_of(s, b);
  } else {
    auto key = [&](int i, int start) { return (start >> lp) + 2 * i; };
    p = find(s, x, key);
    if (p.b < 0) return false;
    rel = x - key(p.b, p.first);
  }
  const int done = p.len - p.n;
  j = static_cast<int64_t>((done > 0 ? done : 0) >> lp) + rel;
  return true;
}

struct Cache {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int pages, heads, dim, lp;
  Divisor by_heads;
};
// ---------------------------------------------------------------------------
// Codes.

template <typename T>
struct Four {
  typedef T Vec __attribute__((ext_vector_type(4)));
};

// Transposes 4 x 4 bytes: byte j of row i becomes byte i of row j.
__device__ inline void transpose4(uint32_t (&r)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
  r[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  r[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  r[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  r[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

__device__ inline uint32_t pack_bytes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  const uint32_t lo = __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(b3, b2, 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Four codes round_half_away(x / s), |x| <= 127 s.  The division is replaced by
// a product with inv = 1 / s wherever that gives the same code: x * inv and
// x / s, each rounded, lie within 2^-18 + 1.6e-5 of the quotient, so where the
// product's fraction is more than 2^-14 from 1/2 both round to its nearest
// integer.  Adding 1.5 * 2^23 rounds to that integer and leaves its byte lowest.
__device__ inline uint32_t codes_of(const float (&x)[4], float s, float inv) {
  float r[4];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = x[j] * inv;
    near |= fabsf(__builtin_amdgcn_fractf(fabsf(r[j])) - 0.5f) <= 0x1p-14f;
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = static_cast<float>(code_of(x[j] / s));
  }
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(r[j] + 0x1.8p23f);
  return pack_bytes(b[0], b[1], b[2], b[3]);
}

// Four codes round_half_away(q * ratio) of codes q.
__device__ inline uint32_t rescaled(uint32_t q, float ratio) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    b[j] = static_cast<uint32_t>(static_cast<int>(roundf(static_cast<float>(static_cast<int8_t>(q >> (8 * j))) * ratio)));
  return pack_bytes(b[0], b[1], b[2], b[3]);
}
// A page's scale after new values of maximum amax; ratio: of its earlier codes.
struct Scaling {
  float now, ratio;
  bool grown;

  __device__ Scaling(float amax, float before, bool begun) : now(fmaxf(amax, kAmaxFloor) / 127.0f), ratio(1.0f), grown(false) {
    if (!begun) return;
    if (now > before) {
      grown = true;
      ratio = before / now;
    } else if (before >= now) {  // a scale that is no number counts for nothing
      now = before;
    }
  }
};
// ---------------------------------------------------------------------------
// Host side.

inline int hip_status() { return hipGetLastError() == hipSuccess ? I2S_OK : I2S_EHIP; }
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int value_bytes(int type) { return type == KV8_F32 ? 4 : type == KV8_F16 || type == KV8_BF16 ? 2 : 0; }

constexpr int64_t kMaxStride = INT64_C(1) << 40;

// I2S_OK, or what is wrong with rows of `width` values of `size` bytes.
inline int check_rows(const void *p, int64_t stride, int64_t width, int size) {
  if (!p || !aligned(p, 16) || stride < width || stride % (16 / size) != 0) return I2S_EINVAL;
  return stride > kMaxStride ? I2S_ERANGE : I2S_OK;
}

inline int check_batch(const kv8_cache *c, const kv8_batch *b, int type, int64_t rows, Cache &dc, Batch &db) {
  if (!c || !b || !value_bytes(type) || rows < 0) return I2S_EINVAL;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !aligned(c->k, 16) || !aligned(c->v, 16) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || c->pages < 1 || c->heads < 1)
    return I2S_EINVAL;
  if (c->dim < 16 || c->dim > KV8_MAX_DIM || c->dim % 16 || c->page_tokens < 16 || c->page_tokens > KV8_MAX_PAGE ||
      (c->page_tokens & (c->page_tokens - 1)))
    return I2S_EALIGN;
  if (b->seqs < 0 || b->blocks < 0 || b->table_stride < b->blocks || b->max_len < 0) return I2S_EINVAL;
  if (c->pages > 0x7fffffff || c->heads > 1024 || b->seqs > kMaxSeqs || b->blocks > 0x7fffffff || rows > kMaxRows ||
      b->table_stride > kMaxStride)
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
  dc.by_heads = Divisor(c->heads);
  db.table = b->table;
  db.lens = b->lens;
  db.starts = b->starts;
  db.table_stride = b->table_stride;
  db.blocks = static_cast<int>(b->blocks);
  db.seqs = static_cast<int>(b->seqs);
  db.rows = static_cast<int>(rows);
  db.per_seq = b->seqs > 0 ? static_cast<int>(rows / b->seqs) : 0;
  db.slots_each = Divisor(((db.per_seq + c->page_tokens - 2) >> dc.lp) + 1);
  return I2S_OK;
}

// Page slots of a batch: see slot_of.
inline int64_t slots(const Batch &s, int lp) {
  if (s.starts) return (s.rows >> lp) + 2 * static_cast<int64_t>(s.seqs);
  return static_cast<int64_t>(s.seqs) * (((s.per_seq + (INT64_C(1) << lp) - 2) >> lp) + 1);
}
template <typename F>
int by_type(int type, F f) {
  if (type == KV8_F32) return f(float());
  if (type == KV8_F16) return f(f16());
  return f(bf16());
}

}  // namespace
