// gfx950 (MI355X) kernels and C ABI of attention over an int8 K/V cache:
// rotation with per-head norms, the quantizing cache write, its read-back and
// the attention itself.  The ABI is declared, with its contract, in
// include/kv8.h.
//
// Every float operation that decides a code (the scale's division, x / s,
// q * ratio) is one IEEE operation: the library is built without fast-math and
// without FP contraction, and '/' is the correctly rounded division, so the
// cache's bytes match the definition bit for bit.

#include "kv8_attention.h"

namespace {

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
  const Rowset r = {q, q_stride, q_heads, rows, out, out_stride, lse, workspace, workspace_bytes};
  return attend(a, batch, type, r, scale, causal, window, stream);
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
