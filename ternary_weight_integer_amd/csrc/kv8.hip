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
// Attention, the plain way: one wave per (row, query head), 64 tokens at a
// time, sums in 64 bits.

template <typename T>
__global__ void __launch_bounds__(64) attention_kernel(Cache c, Batch s, const T *__restrict__ q, int64_t q_stride,
                                                       int q_heads, float scale, int causal, int64_t window,
                                                       T *__restrict__ out, int64_t out_stride, float *__restrict__ lse) {
  __shared__ double x[KV8_MAX_DIM], w[64];
  const int row = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x;
  int b;
  if (s.starts) {
    b = last_at_most(s.seqs, row, [&](int i) { return start_of(s, i); });
    if (b < 0) return;
  } else {
    b = row / s.per_seq;
  }
  const Span p = span_of(s, b);
  if (row >= p.first + p.n) return;
  const int D = c.dim, P = 1 << c.lp, h = hq / (q_heads / c.heads);
  const int64_t pos = static_cast<int64_t>(p.len) - p.n + (row - p.first);
  for (int d = lane; d < D; d += 64) x[d] = static_cast<float>(q[row * q_stride + hq * D + d]);
  __syncthreads();
  int64_t t1 = p.len, t0 = 0;
  if (causal && pos + 1 < t1) t1 = pos + 1;
  if (window > 0 && pos - window + 1 > 0) t0 = pos - window + 1;
  double m = -HUGE_VAL, l = 0.0, acc[KV8_MAX_DIM / 64] = {};
  for (int64_t base = t0; base < t1; base += 64) {
    const int64_t t = base + lane;
    double e = -HUGE_VAL, vs = 0.0;
    if (t < t1) {
      const int page = page_of(s, b, t >> c.lp, c.pages);
      if (page >= 0) {
        const int64_t at = static_cast<int64_t>(page) * c.heads + h;
        const int8_t *k = c.k + at * P * D + (t & (P - 1)) * D;
        double dot = 0.0;
        for (int d = 0; d < D; ++d) dot += x[d] * k[d];
        e = dot * c.k_scale[at] * scale;
        vs = c.v_scale[at];
      }
    }
    double top = e;
    for (int k = 1; k < 64; k *= 2) top = fmax(top, __shfl_xor(top, k));
    if (e != e) top = e;
    top = fmax(top, m);
    const double ref = top == -HUGE_VAL ? 0.0 : top, alpha = exp(m - ref), pr = exp(e - ref);
    double sum = pr;
    for (int k = 1; k < 64; k *= 2) sum += __shfl_xor(sum, k);
    l = l * alpha + sum;
    m = top;
    w[lane] = pr * vs;
    __syncthreads();
    for (int i = 0, d = lane; d < D; d += 64, ++i) acc[i] *= alpha;
    for (int k = 0; k < 64 && base + k < t1; ++k) {
      const int page = page_of(s, b, (base + k) >> c.lp, c.pages);
      if (page < 0) continue;
      const int8_t *v = c.v + (static_cast<int64_t>(page) * c.heads + h) * P * D + ((base + k) & (P - 1));
      for (int i = 0, d = lane; d < D; d += 64, ++i) acc[i] += w[k] * v[d * P];
    }
    __syncthreads();
  }
  for (int i = 0, d = lane; d < D; d += 64, ++i)
    out[row * out_stride + hq * D + d] = static_cast<T>(static_cast<float>(l == 0.0 ? 0.0 : acc[i] / l));
  if (lse && lane == 0) lse[static_cast<int64_t>(row) * q_heads + hq] = static_cast<float>(l == 0.0 ? -HUGE_VAL : m + log(l));
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
  if (check_batch(cache, batch, KV8_F32, rows, c, s) || q_heads < 1 || q_heads % c.heads) return 0;
  return 0;
}

extern "C" int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, int type, const void *q, int64_t q_stride,
                             int64_t q_heads, int64_t rows, float scale, int causal, int64_t window, void *out,
                             int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  Cache c;
  Batch s;
  if (const int st = check_batch(cache, batch, type, rows, c, s)) return st;
  if (q_heads < 1 || q_heads % c.heads || window < 0 || !(fabsf(scale) < INFINITY)) return I2S_EINVAL;
  if (q_heads > 65535) return I2S_ERANGE;
  if (rows == 0 || s.seqs == 0) return I2S_OK;
  const int64_t width = q_heads * c.dim;
  if (bad_rows(q, q_stride, width, value_bytes(type)) || bad_rows(out, out_stride, width, value_bytes(type)) ||
      !aligned(lse, 4))
    return I2S_EINVAL;
  const size_t need = kv8_attention_workspace_bytes(cache, batch, q_heads, rows);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I2S_EWORKSPACE;
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    attention_kernel<T><<<dim3(static_cast<unsigned>(rows), static_cast<unsigned>(q_heads)), 64, 0,
                          static_cast<hipStream_t>(stream)>>>(c, s, static_cast<const T *>(q), q_stride,
                                                              static_cast<int>(q_heads), scale, causal, window,
                                                              static_cast<T *>(out), out_stride, lse);
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
