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

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kv8.h"

namespace {

constexpr int kThreads = 256;  // 4 wave64s
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
// Append and read-back.
//
// One item is a page slot, a head, and K or V.  A lane works on units of
// kTokens (8 or 16) tokens x 4 components: 32 neighbouring lanes cover a row of
// 128 components, so rows are read and written in whole lines, and V's turning (tokens
// innermost in the page) is 4 x 4 byte transposes within the lane.  A wave has
// 64 units at a time; an item has as many waves as its units fill, up to the
// workgroup's 4.

constexpr int kUnitDims = 4, kAppendTokens = 8, kFewTokens = 4;

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

// An item: the tokens [t0, t1) that it holds of the call's rows, in slots
// lo .. lo + n - 1 of its page.
struct Item {
  int b, h, lo, n;
  bool value;
  int page;     // -1: a hole
  int64_t row;  // of token t0
  int ahead, first;  // rows in front of position 0 (at the sequence's first slot), and the first of them
};

__device__ inline bool item_of(const Cache &c, const Batch &s, int64_t index, Item &it) {
  it.n = it.ahead = 0;
  it.page = -1;
  it.value = index & 1;
  const int place = static_cast<int>(index >> 1), slot = c.by_heads.of(place);
  it.h = place - slot * c.heads;
  Span p;
  int64_t j;
  if (!slot_of(s, c.lp, slot, p, j)) return false;
  const int64_t done = static_cast<int64_t>(p.len) - p.n, begin = j << c.lp;
  it.b = p.b;
  it.first = p.first;
  if (done < 0 && begin == 0) it.ahead = static_cast<int>(-done < p.n ? -done : p.n);
  int64_t t0 = done > begin ? done : begin, t1 = begin + (1 << c.lp);
  if (t0 < 0) t0 = 0;
  if (t1 > p.len) t1 = p.len;
  if (t0 < t1) {
    it.n = static_cast<int>(t1 - t0);
    it.lo = static_cast<int>(t0 - begin);
    it.row = p.first + (t0 - done);
    it.page = page_of(s, p.b, j, c.pages);
  }
  return true;
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

// Few new tokens (a decode step): one wave, a lane four components of each
// token.  Nothing is read back unless the scale grew, V's new codes are single
// bytes: for 48 sequences of one token 8 heads took 17.6 us by whole units.
template <typename T>
__device__ inline void append_few(const T *src, int64_t stride, int8_t *codes, float *scale, int P, int D, int lo, int n, bool value) {
  typedef typename Four<T>::Vec Vec;
  const int lane = threadIdx.x & 63, d = kUnitDims * lane;
  Vec x[kFewTokens];
  float before = 0.0f, amax = 0.0f;
  if (lo > 0) before = *scale;
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    x[i] = Vec{};
    if (i < n && d < D) x[i] = *reinterpret_cast<const Vec *>(src + i * stride + d);
  }
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fabsf(static_cast<float>(x[i][k])));
  }
  const Scaling s(wave_max(amax), before, lo > 0);
  if (lane == 0 && s.now != before) *scale = s.now;
  if (s.grown) {
    const int row = value ? P : D, count = value ? D * P / 16 : lo * D / 16;
    for (int u = lane; u < count; u += 64) {
      const int slot = value ? 16 * u % row : 0;
      if (slot >= lo && value) continue;
      i32x4 *at = reinterpret_cast<i32x4 *>(codes) + u;
      i32x4 q = *at;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // Codes behind the earlier tokens keep their bytes.
        const int left = value ? lo - slot - 4 * w : 4;
        const uint32_t mask = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1;
        const uint32_t old = static_cast<uint32_t>(q[w]);
        q[w] = static_cast<int>((old & ~mask) | (rescaled(old, s.ratio) & mask));
      }
      *at = q;
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);  // before single bytes of the same 16 are written
  }
  if (d >= D) return;
  const float inv = 1.0f / s.now;
#pragma unroll
  for (int i = 0; i < kFewTokens; ++i) {
    if (i >= n) continue;
    const float v[4] = {static_cast<float>(x[i][0]), static_cast<float>(x[i][1]), static_cast<float>(x[i][2]),
                        static_cast<float>(x[i][3])};
    const uint32_t code = codes_of(v, s.now, inv);
    if (!value) {
      *reinterpret_cast<uint32_t *>(codes + (lo + i) * D + d) = code;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) codes[(d + k) * P + lo + i] = static_cast<int8_t>(code >> (8 * k));
    }
  }
}

// Append: the maximum of the item's new values, the page's scale, then the
// codes.  Bound by the chain of lookup, values, maximum and stores: 7 prompts
// (12163 rows of 2 heads of 128 F32 values, 31 MB) in 15 us, with units of 4, 8
// or 16 tokens and with V's units dealt to lanes along tokens alike.  kOnce:
// the item's units fill its waves once, and the values stay in registers
// between the two; else they are read again (from the cache).
template <typename T, bool kOnce>
__global__ void __launch_bounds__(kThreads) append_kernel(Cache c, Batch s, const T *__restrict__ kx, int64_t k_stride,
                                                          const T *__restrict__ vx, int64_t v_stride, int waves,
                                                          int64_t items) {
  constexpr int kTokens = kAppendTokens;
  __shared__ float red[kThreads / 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t index = static_cast<int64_t>(blockIdx.x) * (4 / waves) + wave / waves;
  Item it;
  const bool live = index < items && item_of(c, s, index, it) && it.n > 0 && it.page >= 0;
  const bool few = live && it.n <= kFewTokens;
  const int P = 1 << c.lp, D = c.dim, per = D / kUnitDims, units = live && !few ? P / kTokens * per : 0;
  const int64_t stride = live && it.value ? v_stride : k_stride;
  const T *src = (live && it.value ? vx : kx) + (live ? it.row * stride + static_cast<int64_t>(it.h) * D : 0);
  const int64_t at = live ? static_cast<int64_t>(it.page) * c.heads + it.h : 0;
  float *scale = (live && it.value ? c.v_scale : c.k_scale) + at;
  int8_t *codes = (live && it.value ? c.v : c.k) + at * P * D;
  const int lo = live ? it.lo : 0, end = live ? it.lo + it.n : 0;
  const int first = (wave % waves) * 64 + lane, step = waves * 64;
  if (few && wave % waves == 0) append_few(src, stride, codes, scale, P, D, lo, it.n, it.value);
  typedef typename Four<T>::Vec Vec;
  typedef int Tokens __attribute__((ext_vector_type(kTokens / 4)));  // a component's codes in a unit
  Vec x[kTokens];
  auto load = [&](int u) {
    const int d = u % per * kUnitDims, s0 = u / per * kTokens;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      x[i] = Vec{};
      if (s0 + i >= lo && s0 + i < end) x[i] = *reinterpret_cast<const Vec *>(src + (s0 + i - lo) * stride + d);
    }
  };
  const float before = units > 0 && lo > 0 ? *scale : 0.0f;
  float amax = 0.0f;
  for (int u = first; u < units; u += step) {
    load(u);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fabsf(static_cast<float>(x[i][k])));
    }
  }
  amax = wave_max(amax);
  if (lane == 0) red[wave] = amax;
  __syncthreads();  // the old scale has been read, too
  if (units == 0) return;
  for (int k = 0; k < waves; ++k) amax = fmaxf(amax, red[wave / waves * waves + k]);
  const Scaling scaling(amax, before, lo > 0);
  const float now = scaling.now, ratio = scaling.ratio, inv = 1.0f / now;
  const bool grown = scaling.grown;
  if (first == 0) *scale = now;
  for (int u = first; u < units; u += step) {
    const int d = u % per * kUnitDims, s0 = u / per * kTokens;
    const bool has_new = s0 < end && s0 + kTokens > lo, has_old = grown && s0 < lo;
    if (!has_new && !has_old) continue;
    if (!kOnce) load(u);
    uint32_t code[kTokens];  // a token's four components
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = static_cast<float>(x[i][k]);
      code[i] = codes_of(v, now, inv);  // 0 outside the new tokens
    }
    if (!it.value) {
      uint32_t *to = reinterpret_cast<uint32_t *>(codes + s0 * D + d);
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        if (s0 + i >= lo && s0 + i < end) {
          to[i * per] = code[i];
        } else if (grown && s0 + i < lo) {
          to[i * per] = rescaled(to[i * per], ratio);
        }
      }
    } else {
      const bool whole = s0 >= lo && s0 + kTokens <= end;
      Tokens row[4];  // of a component
#pragma unroll
      for (int i = 0; i < kTokens / 4; ++i) {
        uint32_t r[4] = {code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]};
        transpose4(r);
#pragma unroll
        for (int k = 0; k < 4; ++k) row[k][i] = static_cast<int>(r[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        Tokens *to = reinterpret_cast<Tokens *>(codes + (d + k) * P + s0);
        if (!whole) {
          const Tokens old = *to;
#pragma unroll
          for (int i = 0; i < kTokens / 4; ++i) {
            uint32_t kept = static_cast<uint32_t>(old[i]), mask = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int slot = s0 + 4 * i + j;
              if (slot >= lo && slot < end) mask |= 0xffu << (8 * j);
            }
            if (grown && s0 + 4 * i < lo) {
              const uint32_t moved = rescaled(kept, ratio);
              uint32_t gone = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (s0 + 4 * i + j < lo) gone |= 0xffu << (8 * j);
              kept = (kept & ~gone) | (moved & gone);
            }
            row[k][i] = static_cast<int>((kept & ~mask) | (static_cast<uint32_t>(row[k][i]) & mask));
          }
        }
        *to = row[k];
      }
    }
  }
}

// Read-back, the inverse.  Bound by memory: 405 MB of codes and BF16 values in
// 78 to 85 us (4.8 to 5.2 TB/s).
template <typename T, int kTokens>
__global__ void __launch_bounds__(kThreads) read_kernel(Cache c, Batch s, T *__restrict__ ko, int64_t k_stride,
                                                        T *__restrict__ vo, int64_t v_stride, int waves, int64_t items) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t index = static_cast<int64_t>(blockIdx.x) * (4 / waves) + wave / waves;
  Item it;
  if (index >= items || !item_of(c, s, index, it)) return;
  const int P = 1 << c.lp, D = c.dim, per = D / kUnitDims, first = (wave % waves) * 64 + lane, step = waves * 64;
  const int64_t stride = it.value ? v_stride : k_stride;
  T *out = (it.value ? vo : ko) + static_cast<int64_t>(it.h) * D;
  typedef typename Four<T>::Vec Vec;
  typedef int Tokens __attribute__((ext_vector_type(kTokens / 4)));  // a component's codes in a unit
  for (int64_t u = first; u < static_cast<int64_t>(it.ahead) * per; u += step)
    *reinterpret_cast<Vec *>(out + (it.first + u / per) * stride + u % per * kUnitDims) = Vec{};
  if (it.n == 0) return;
  const int units = P / kTokens * per, end = it.lo + it.n;
  const int64_t at = static_cast<int64_t>(it.page < 0 ? 0 : it.page) * c.heads + it.h;
  const float scale = it.page < 0 ? 0.0f : (it.value ? c.v_scale : c.k_scale)[at];
  const int8_t *codes = (it.value ? c.v : c.k) + at * P * D;
  out += it.row * stride;
  for (int u = first; u < units; u += step) {
    const int d = u % per * kUnitDims, s0 = u / per * kTokens;
    if (s0 >= end || s0 + kTokens <= it.lo) continue;
    uint32_t code[kTokens];
    if (!it.value) {
#pragma unroll
      for (int i = 0; i < kTokens; ++i) code[i] = *reinterpret_cast<const uint32_t *>(codes + (s0 + i) * D + d);
    } else {
      Tokens row[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) row[k] = *reinterpret_cast<const Tokens *>(codes + (d + k) * P + s0);
#pragma unroll
      for (int i = 0; i < kTokens / 4; ++i) {
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = static_cast<uint32_t>(row[k][i]);
        transpose4(r);
#pragma unroll
        for (int k = 0; k < 4; ++k) code[4 * i + k] = r[k];
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (s0 + i < it.lo || s0 + i >= end) continue;
      Vec v;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float q = static_cast<float>(static_cast<int8_t>(code[i] >> (8 * k)));
        v[k] = static_cast<T>(it.page < 0 ? 0.0f : q * scale);
      }
      *reinterpret_cast<Vec *>(out + (s0 + i - it.lo) * stride + d) = v;
    }
  }
}

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
//     of two (22 bits), where many BF16 rows are worked on one (11 bits: its
//     rounding is an eighth of the result's own, and adds 0.5 to 0.8% to its
//     error; a second takes 18 to 20% of a prompt's time, and 1 to 4% where rows
//     are few).
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
constexpr int kMaxSplits = 256;
constexpr int kFewParts = 8;       // that 32 lanes join
constexpr int kUnits = 256;        // compute units
constexpr int kFillWaves = 8 * kUnits;

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

__device__ inline Range range_of(const Attend &a, const Span &p, int first_row, int last_row) {
  const int ahead = p.len - p.n, p0 = ahead + a.by_group.of(first_row), p1 = ahead + a.by_group.of(last_row);
  const int held = a.s.blocks << a.c.lp, top = held < p.len ? held : p.len;
  Range r;
  r.hi = a.causal ? clamp_int(static_cast<int64_t>(p0) + 1, top) : top;
  r.end = a.causal ? clamp_int(static_cast<int64_t>(p1) + 1, top) : top;
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
template <typename T, int kChunks, bool kFull, int kRowTiles, bool kDirect, int kWeightParts>
struct Rows {
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

  const Attend &a;
  const int n, g, D;
  f32x4 acc[kRowTiles][kOut];
  i32x4 q[kRowTiles][kChunks][kOperands];
  float qs[kRowTiles], m[kRowTiles], l[kRowTiles];  // m: the running maximum less kHeadroom
  int lo[kRowTiles], hi[kRowTiles];
  int row_of[kRowTiles], head_of[kRowTiles];        // row_of: -1 behind the last row
  Vec qv[kRowTiles][kChunks][kVecs];

  __device__ Rows(const Attend &args)
      : a(args), n(threadIdx.x & 15), g((threadIdx.x & 63) >> 4), D(kFull ? 64 * kChunks : args.c.dim) {}

  __device__ void place(const Place &w, int row0, int end) {
#pragma unroll
    for (int t = 0; t < kRowTiles; ++t) {
      const int row = row0 + 16 * t + n;
      const bool live = row < w.rows;
      const int i = live ? a.by_group.of(row) : 0;
      const int pos = w.p.len - w.p.n + i;
      row_of[t] = live ? w.p.first + i : -1;
      head_of[t] = w.h * a.group + (live ? row - i * a.group : 0);
      hi[t] = !live ? 0 : a.causal ? clamp_int(static_cast<int64_t>(pos) + 1, end) : end;
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
    const float vs = s.hole ? 1.0f : fmaxf(s.vs, kMinScale);
    const float lvs = __builtin_amdgcn_logf(vs), rvs = __builtin_amdgcn_rcpf(vs);
    const float ck = qs[t] * s.ks;
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
template <typename T, int kChunks, bool kFull>
__global__ void __launch_bounds__(kThreads, kChunks > 2 ? 1 : 2) attention_few_kernel(Attend a) {
  typedef Rows<T, kChunks, kFull, 1, false, 2> R;
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

template <typename T, int kChunks, bool kFull, int kRowTiles>
__global__ void __launch_bounds__(kThreads, (Many<T, kChunks, kRowTiles>::kGroups)) attention_many_kernel(Attend a) {
  constexpr bool kDirect = Many<T, kChunks, kRowTiles>::kDirect;
  typedef Rows<T, kChunks, kFull, kRowTiles, kDirect, std::is_same<T, bf16>::value ? 1 : 2> R;
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
__device__ inline int parts_of(const Attend &a, const Span &p, int row, int hq, int block_rows) {
  const int h = a.by_group.of(hq), in_group = (row - p.first) * a.group + hq - h * a.group;
  const int row0 = in_group & -block_rows;  // a power of two
  const int rows = p.n * a.group;
  return range_of(a, p, row0, (row0 + block_rows < rows ? row0 + block_rows : rows) - 1).used;
}

// Few parts (at most kFewParts): 32 lanes a row and head, four components each.
// block_rows: rows of the attention's workgroups.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_few_kernel(Attend a, int block_rows) {
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
template <typename T>
__global__ void __launch_bounds__(kThreads) join_many_kernel(Attend a, int block_rows) {
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

// ---------------------------------------------------------------------------
// Norm and rotation.  A wave takes one row and a share of its heads, or (few
// heads) several rows.  A lane holds 32 bytes of a head: the two halves of its
// pairs (16 bytes at i and 16 at i + pairs), or 32 neighbouring bytes, so a
// rotation never leaves its lane (and may be in place); only the norm's sum
// crosses lanes.  Bound by memory: 8192 rows of 40 heads of 128 BF16 values in
// 34 to 37 us (4.6 TB/s).

constexpr int kMaxTurns = 512;  // angles of a wave

template <typename T, bool kNeighbours>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const T *q, int64_t q_stride, int q_heads, const T *k, int64_t k_stride,
                int k_heads, const int32_t *__restrict__ pos, const float *__restrict__ inv_freq, int pairs,
                const float *__restrict__ q_weight, const float *__restrict__ k_weight, float eps, T *q_out,
                int64_t q_out_stride, T *k_out, int64_t k_out_stride, int rows, int dim, int lanes_log, int rows_log,
                int split) {
  constexpr int V = Row<T>::kValues;
  __shared__ float2 turn[kThreads / 64][kMaxTurns];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + wave;
  const int64_t row0 = (item / split) << rows_log;
  for (int i = lane; i < pairs << rows_log; i += 64) {
    const int r = i / pairs;
    if (row0 + r >= rows) break;
    // The angle in turns, 64 bits: positions far along a context keep their
    // fraction; what is left of the fraction's rounding is 2^-26 of a turn.
    double t = static_cast<double>(pos[row0 + r]) * static_cast<double>(inv_freq[i - r * pairs]) * 0.15915494309189533577;
    t -= rint(t);
    float sn, cs;
    sincospif(static_cast<float>(t) * 2.0f, &sn, &cs);
    turn[wave][i] = make_float2(cs, sn);
  }
  __syncthreads();
  // Lanes of a head, heads of a row, rows.
  const int heads_log = 6 - lanes_log - rows_log, per = 1 << heads_log;
  const int c = lane & ((1 << lanes_log) - 1), sub = (lane >> lanes_log) & (per - 1), r = lane >> (lanes_log + heads_log);
  const int64_t row = row0 + r;
  if (row0 >= rows) return;
  const int q_groups = (q_heads + per - 1) >> heads_log, groups = q_groups + ((k_heads + per - 1) >> heads_log);
  const bool rotated = c < pairs / V;
  const int a0 = rotated && !kNeighbours ? c * V : 2 * c * V, a1 = rotated && !kNeighbours ? pairs + c * V : a0 + V;
  float cs[V], sn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 a = rotated ? turn[wave][r * pairs + c * V + i] : make_float2(1.0f, 0.0f);
    cs[i] = a.x;
    sn[i] = a.y;
  }
  for (int g = static_cast<int>(item % split); g < groups; g += split) {
    const bool key = g >= q_groups;
    const int head = (key ? g - q_groups : g) * per + sub;
    const bool live = row < rows && head < (key ? k_heads : q_heads) && 2 * c * V < dim;
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
      const float scale = 1.0f / sqrtf(ss / static_cast<float>(dim) + eps);
      if (live) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[i] = x[i] * scale * weight[a0 + i];
          x[V + i] = x[V + i] * scale * weight[a1 + i];
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

constexpr int64_t kMaxStride = INT64_C(1) << 40;

// I2S_OK, or what is wrong with rows of `width` values of `size` bytes.
inline int check_rows(const void *p, int64_t stride, int64_t width, int size) {
  if (!p || !aligned(p, 16) || stride < width || stride % (16 / size) != 0) return I2S_EINVAL;
  return stride > kMaxStride ? I2S_ERANGE : I2S_OK;
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

// How an append or a read-back is laid out: tokens of a unit, units and waves
// of an item, all items and the workgroups that hold them.
struct Items {
  int tokens, units, waves;
  int64_t items, blocks;

  Items(const Cache &c, const Batch &s, bool append) {
    items = slots(s, c.lp) * c.heads * 2;
    // Reading back, units of 16 tokens move whole 16-byte pieces of V's rows
    // (84 against 91 us for 65536 x 8 x 128 values, BF16), units of 8 make more
    // waves where there are few (5.6 against 6.5 us for 1100 x 2 x 128, F32).
    // Appending holds a unit's values in registers: 8.
    tokens = append ? kAppendTokens : items << c.lp < (INT64_C(1) << 19) ? 8 : 16;
    units = (1 << c.lp) / tokens * (c.dim / kUnitDims);
    waves = units <= 64 ? 1 : units <= 128 ? 2 : 4;
    // A decode step's items are one wave's work.
    if (append && s.rows <= kFewTokens * s.seqs) waves = 1;
    blocks = (items * waves + 3) / 4;
  }
};

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
Plan plan_for(int row_tiles, const Cache &c, const Batch &s, int64_t len, int64_t q_heads) {
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
Plan plan_of(const Cache &c, const Batch &s, int64_t max_len, int64_t q_heads, int64_t window, bool causal) {
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
int check_attention(const kv8_cache *cache, const kv8_batch *batch, int type, int64_t q_heads, int64_t rows, Cache &c,
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

template <typename T, int kChunks, bool kFull>
int launch_attention(const Plan &p, const Attend &a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.blocks * a.c.heads * p.splits);
  if (p.row_tiles == 0) {
    attention_few_kernel<T, kChunks, kFull><<<grid, kThreads, 0, stream>>>(a);
  } else if (p.row_tiles == 1) {
    attention_many_kernel<T, kChunks, kFull, 1><<<grid, kThreads, 0, stream>>>(a);
  } else if constexpr (kChunks <= 2) {  // two row tiles fit the registers, see plan_of
    attention_many_kernel<T, kChunks, kFull, 2><<<grid, kThreads, 0, stream>>>(a);
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
  if (const int st = check_rows(k, k_stride, width, value_bytes(type))) return st;
  if (const int st = check_rows(v, v_stride, width, value_bytes(type))) return st;
  const Items n(c, s, true);
  if (n.blocks > 0x7fffffff || n.items / 2 > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    auto launch = [&](auto kernel) {
      kernel<<<static_cast<unsigned>(n.blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(
          c, s, static_cast<const T *>(k), k_stride, static_cast<const T *>(v), v_stride, n.waves, n.items);
    };
    if (n.units <= 64 * n.waves) {
      launch(append_kernel<T, true>);
    } else {
      launch(append_kernel<T, false>);
    }
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
  if (const int st = check_rows(k, k_stride, width, value_bytes(type))) return st;
  if (const int st = check_rows(v, v_stride, width, value_bytes(type))) return st;
  const Items n(c, s, false);
  if (n.blocks > 0x7fffffff || n.items / 2 > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    auto launch = [&](auto kernel) {
      kernel<<<static_cast<unsigned>(n.blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(
          c, s, static_cast<T *>(k), k_stride, static_cast<T *>(v), v_stride, n.waves, n.items);
    };
    if (n.tokens == 16) {
      launch(read_kernel<T, 16>);
    } else {
      launch(read_kernel<T, 8>);
    }
    return hip_status();
  });
}

extern "C" size_t kv8_attention_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch, int64_t q_heads,
                                                int64_t rows) {
  Cache c;
  Batch s;
  if (check_attention(cache, batch, KV8_F32, q_heads, rows, c, s) || rows == 0 || s.seqs == 0) return 0;
  return workspace_of(plan_of(c, s, batch->max_len, q_heads, 0, true), c, s, q_heads);
}

// What a kv8_attention call with these sizes runs: row_tiles of a wave of the
// kernel for many rows (0: the kernel for few) and the parts that tokens are
// cut into.  No part of the ABI: tests learn from it which kernel they test.
extern "C" int kv8_attention_choice(const kv8_cache *cache, const kv8_batch *batch, int64_t q_heads, int64_t rows,
                                    int causal, int64_t window, int *row_tiles, int *parts) {
  Cache c;
  Batch s;
  if (const int st = check_attention(cache, batch, KV8_F32, q_heads, rows, c, s)) return st;
  if (rows == 0 || s.seqs == 0 || window < 0) return I2S_EINVAL;
  const Plan p = plan_of(c, s, batch->max_len, q_heads, window_of(window), causal != 0);
  *row_tiles = p.row_tiles;
  *parts = p.splits;
  return I2S_OK;
}

extern "C" int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, int type, const void *q, int64_t q_stride,
                             int64_t q_heads, int64_t rows, float scale, int causal, int64_t window, void *out,
                             int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  Attend a;
  if (const int st = check_attention(cache, batch, type, q_heads, rows, a.c, a.s)) return st;
  if (window < 0 || !(fabsf(scale) < INFINITY)) return I2S_EINVAL;
  if (rows == 0 || a.s.seqs == 0) return I2S_OK;
  const int64_t width = q_heads * a.c.dim;
  if (const int st = check_rows(q, q_stride, width, value_bytes(type))) return st;
  if (const int st = check_rows(out, out_stride, width, value_bytes(type))) return st;
  if (!aligned(lse, 4)) return I2S_EINVAL;
  const Plan p = plan_of(a.c, a.s, batch->max_len, q_heads, window_of(window), causal != 0);
  if (p.blocks * a.c.heads * p.splits > 0x7fffffff || rows * q_heads > 0x7fffffff) return I2S_ERANGE;
  const size_t need = workspace_of(p, a.c, a.s, q_heads);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I2S_EWORKSPACE;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.acc = static_cast<float *>(workspace);
  a.ml = need ? a.acc + static_cast<int64_t>(p.splits) * rows * q_heads * a.c.dim : nullptr;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.window = static_cast<int>(window_of(window));
  a.scale = scale * 1.44269504088896341f;
  a.q_heads = static_cast<int>(q_heads);
  a.group = static_cast<int>(q_heads / a.c.heads);
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
      join_many_kernel<T><<<dim3(static_cast<unsigned>(rows), a.q_heads), kThreads, 0, on>>>(a, p.block_rows);
    } else {
      join_few_kernel<T><<<static_cast<unsigned>((rows * q_heads + 7) / 8), kThreads, 0, on>>>(a, p.block_rows);
    }
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
  if (q_heads > 0) {
    if (const int st = check_rows(q, q_stride, q_heads * dim, size)) return st;
    if (const int st = check_rows(q_out, q_out_stride, q_heads * dim, size)) return st;
  }
  if (k_heads > 0) {
    if (const int st = check_rows(k, k_stride, k_heads * dim, size)) return st;
    if (const int st = check_rows(k_out, k_out_stride, k_heads * dim, size)) return st;
  }
  if (!pos || !aligned(pos, 4) || (pairs > 0 && !inv_freq) || !aligned(inv_freq, 4) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4))
    return I2S_EINVAL;
  const int chunks = static_cast<int>(dim) * size / 32;
  int lanes_log = 0;
  while ((1 << lanes_log) < chunks) ++lanes_log;
  // Few heads and enough rows to fill the card's waves: several rows a wave
  // (40000 rows of 3 heads of 64 BF16 values: 12 against 38 us).
  int rows_log = 0;
  while (rows_log < 6 - lanes_log && (q_heads > k_heads ? q_heads : k_heads) <= (64 >> lanes_log >> (rows_log + 1)) &&
         pairs << (rows_log + 1) <= kMaxTurns && rows >> (rows_log + 1) >= kFillWaves)
    ++rows_log;
  const int64_t per = 64 >> lanes_log >> rows_log, groups = (q_heads + per - 1) / per + (k_heads + per - 1) / per;
  // Few rows: a wave for each group of heads that fit it; many: a wave per
  // row, which then turns its angles once.
  const int64_t units = ((rows - 1) >> rows_log) + 1;
  int64_t split = rows_log ? 1 : (kFillWaves + rows - 1) / rows;
  if (split > groups) split = groups;
  const int64_t blocks = (units * split + kThreads / 64 - 1) / (kThreads / 64);
  if (blocks > 0x7fffffff) return I2S_ERANGE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    auto launch = [&](auto kernel) {
      kernel<<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(
          static_cast<const T *>(q), q_stride, static_cast<int>(q_heads), static_cast<const T *>(k), k_stride,
          static_cast<int>(k_heads), pos, inv_freq, static_cast<int>(pairs), q_weight, k_weight, eps,
          static_cast<T *>(q_out), q_out_stride, static_cast<T *>(k_out), k_out_stride, static_cast<int>(rows),
          static_cast<int>(dim), lanes_log, rows_log, static_cast<int>(split));
    };
    if (neighbours) {
      launch(rope_kernel<T, true>);
    } else {
      launch(rope_kernel<T, false>);
    }
    return hip_status();
  });
}
