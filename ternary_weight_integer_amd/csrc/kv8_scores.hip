// gfx950 (MI355X) kernels and C ABI of scores, weights and eviction over the
// int8 K/V cache: attention with shaped scores (the kernels of
// kv8_attention.h), the weight that each cached token gets, the choice of those
// that stay and their move to fresh pages.  The ABI is declared, with its
// contract, in include/kv8_scores.h.

#include "kv8_scores.h"

#include "kv8_attention.h"

namespace {

// ---------------------------------------------------------------------------
// The weight that rows give the cached tokens.

struct Weigh {
  Cache c;
  Batch s;
  const void *q;
  const float *lse, *slopes;
  const int32_t *prefix;
  float *mass;
  int64_t q_stride;
  float scale, cap, icap;  // in units of log2
  int window, q_heads, group, causal, blocks;  // workgroups along a sequence's tokens
};

// A workgroup has 256 tokens of a sequence and head, a thread one of them.
template <typename T>
__global__ void __launch_bounds__(kThreads) weigh_kernel(Weigh a) {
  __shared__ float qrow[KV8_MAX_DIM];
  const int h = blockIdx.x % a.c.heads, rest = blockIdx.x / a.c.heads, b = rest / a.blocks;
  const Span p = span_of(a.s, b);
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len, D = a.c.dim, own = p.len - p.n;
  const int prefix = a.prefix ? a.prefix[b] : 0;
  if (p.n == 0) return;
  for (int64_t t0 = static_cast<int64_t>(rest % a.blocks) * kThreads; t0 < top; t0 += static_cast<int64_t>(a.blocks) * kThreads) {
    const int64_t t = t0 + threadIdx.x;
    const int page = t < top ? page_of(a.s, b, t >> a.c.lp, a.c.pages) : -1;
    const int64_t at = static_cast<int64_t>(page < 0 ? 0 : page) * a.c.heads + h, slot = t & ((1 << a.c.lp) - 1);
    const int8_t *k = a.c.k + ((at << a.c.lp) + slot) * D;
    const float ks = a.c.k_scale[at];
    float sum = 0.0f;
    for (int i = 0; i < p.n; ++i) {
      const int64_t pos = static_cast<int64_t>(own) + i;
      const bool seen = page >= 0 && (!a.causal || t <= pos || t < prefix) && (a.window == 0 || t > pos - a.window);
      for (int g = 0; g < a.group; ++g) {
        const int hq = h * a.group + g;
        const float lse = a.lse[static_cast<int64_t>(p.first + i) * a.q_heads + hq];
        if (!(fabsf(lse) < INFINITY)) continue;
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < D)
          qrow[threadIdx.x] = static_cast<float>(static_cast<const T *>(a.q)[(p.first + i) * a.q_stride + static_cast<int64_t>(hq) * D + threadIdx.x]);
        __syncthreads();
        if (!seen) continue;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot = fmaf(static_cast<float>(k[d]), qrow[d], dot);
        float x = a.scale * (ks * dot);
        if (a.cap > 0.0f) {
          float all[16] = {x};
          capped(all, a.cap, a.icap);
          x = all[0];
        }
        if (a.slopes) x = fmaf(-a.slopes[hq] * kLog2e, static_cast<float>(llabs(pos - t)), x);
        sum += __builtin_amdgcn_exp2f(fmaf(-lse, kLog2e, x));
      }
    }
    if (page < 0) continue;
    float *mass = a.mass + (at << a.c.lp) + slot;
    if (t >= own) {
      *mass = sum;
    } else {
      unsafeAtomicAdd(mass, sum);
    }
  }
}

// ---------------------------------------------------------------------------
// The choice of the tokens that stay.

constexpr int kChooseThreads = 1024, kBins = 256;

struct Choose {
  Cache c;
  Batch s;
  const float *mass;
  int64_t keep;
  int first, recent;
  int32_t *index, *kept;
};

// A number that rises with the mass: 0 for a token that is none, 1 for a NaN,
// the largest for one that always stays.
__device__ inline uint32_t rank_of(float mass, bool always) {
  if (always) return 0xffffffffu;
  if (mass != mass) return 1;
  const uint32_t u = __float_as_uint(mass + 0.0f);  // -0 is 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A workgroup has a sequence and head.  The least rank that stays is found
// digit by digit from the highest, with a histogram of the ranks that begin with
// the digits found; then the tokens are written in order.
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(Choose a) {
  __shared__ int hist[kBins], waves[2][kChooseThreads / 64];
  const int h = blockIdx.x % a.c.heads, b = blockIdx.x / a.c.heads, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Span p = span_of(a.s, b);
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len;
  auto rank = [&](int64_t t) -> uint32_t {
    if (t >= top) return 0;
    const int page = page_of(a.s, b, t >> a.c.lp, a.c.pages);
    if (page < 0) return 0;
    const int64_t at = static_cast<int64_t>(page) * a.c.heads + h;
    return rank_of(a.mass[(at << a.c.lp) + (t & ((1 << a.c.lp) - 1))], t < a.first || t >= static_cast<int64_t>(p.len) - a.recent);
  };
  uint32_t least = 0;
  int64_t want = a.keep;  // of the ranks that begin with least's digits
  int total = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < kBins) hist[tid] = 0;
    __syncthreads();
    for (int64_t t = tid; t < top; t += kChooseThreads) {
      const uint32_t r = rank(t);
      if (r != 0 && (shift == 24 || (r >> (shift + 8)) == (least >> (shift + 8)))) atomicAdd(&hist[(r >> shift) & (kBins - 1)], 1);
    }
    __syncthreads();
    if (shift == 24)
      for (int i = 0; i < kBins; ++i) total += hist[i];
    if (total <= a.keep) break;
    int digit = kBins - 1;
    while (digit > 0 && hist[digit] < want) want -= hist[digit--];
    least |= static_cast<uint32_t>(digit) << shift;
    __syncthreads();
  }
  const bool all = total <= a.keep;
  int32_t *out = a.index + (static_cast<int64_t>(b) * a.c.heads + h) * a.keep;
  int done = 0, ties = 0;
  for (int64_t t0 = 0; t0 < top; t0 += kChooseThreads) {
    const uint32_t r = rank(t0 + tid);
    const bool tie = !all && r != 0 && r == least;
    const uint64_t same = __ballot(tie), below = (uint64_t{1} << lane) - 1;
    if (lane == 0) waves[0][wave] = __popcll(same);
    __syncthreads();
    int before = ties;
    for (int i = 0; i < kChooseThreads / 64; ++i) {
      before += i < wave ? waves[0][i] : 0;
      ties += waves[0][i];
    }
    const bool stays = r != 0 && (all || r > least || (tie && before + __popcll(same & below) < want));
    const uint64_t mine = __ballot(stays);
    if (lane == 0) waves[1][wave] = __popcll(mine);
    __syncthreads();
    int place = done;
    for (int i = 0; i < kChooseThreads / 64; ++i) {
      place += i < wave ? waves[1][i] : 0;
      done += waves[1][i];
    }
    if (stays) out[place + __popcll(mine & below)] = static_cast<int32_t>(t0 + tid);
  }
  for (int64_t i = done + tid; i < a.keep; i += kChooseThreads) out[i] = -1;
  if (h == 0 && tid == 0) a.kept[b] = done;
}

// ---------------------------------------------------------------------------
// The move of chosen tokens to fresh pages.

struct Move {
  Cache c;
  Batch s;
  const int32_t *index, *kept, *to;
  int64_t keep, to_stride;
  int to_blocks, blocks;  // blocks: page slots of a sequence in the grid
  float *mass;
};

// A workgroup has a page, a head, and K or V.
__global__ void __launch_bounds__(kThreads) move_kernel(Move a) {
  __shared__ int64_t src[KV8_MAX_PAGE];
  __shared__ float scale[KV8_MAX_PAGE], red[kThreads / 64];
  const int tid = threadIdx.x, P = 1 << a.c.lp, D = a.c.dim;
  const bool value = blockIdx.x & 1;
  const int place = blockIdx.x >> 1, h = place % a.c.heads, rest = place / a.c.heads, b = rest / a.blocks;
  const Span p = span_of(a.s, b);
  const int64_t asked = a.kept[b], kept = asked < 0 ? 0 : asked < a.keep ? asked : a.keep;
  for (int64_t j = rest % a.blocks; j < a.to_blocks && (j << a.c.lp) < kept; j += a.blocks) {
    const int to = a.to[b * a.to_stride + j];
    if (to < 0 || to >= a.c.pages) continue;
    const int n = static_cast<int>(kept - (j << a.c.lp) < P ? kept - (j << a.c.lp) : P);
    const int64_t dest = static_cast<int64_t>(to) * a.c.heads + h;
    __syncthreads();
    if (tid < n) {
      const int64_t t = a.index[(static_cast<int64_t>(b) * a.c.heads + h) * a.keep + (j << a.c.lp) + tid];
      const int page = t >= 0 && t < p.len ? page_of(a.s, b, t >> a.c.lp, a.c.pages) : -1;
      const int64_t at = static_cast<int64_t>(page) * a.c.heads + h, slot = t & (P - 1);
      src[tid] = page < 0 ? -1 : (at << a.c.lp) * D + (value ? slot : slot * D);
      scale[tid] = page < 0 ? 0.0f : (value ? a.c.v_scale : a.c.k_scale)[at];
      if (!value && a.mass) a.mass[(dest << a.c.lp) + tid] = page < 0 ? 0.0f : a.mass[(at << a.c.lp) + slot];
    }
    __syncthreads();
    const int8_t *codes = value ? a.c.v : a.c.k;
    int8_t *out = (value ? a.c.v : a.c.k) + (dest << a.c.lp) * D;
    auto get = [&](int i, int d) { return src[i] < 0 ? 0.0f : static_cast<float>(codes[src[i] + (value ? d * P : d)]) * scale[i]; };
    float amax = 0.0f;
    for (int x = tid; x < P * D; x += kThreads) {
      const int i = value ? x % P : x / D, d = value ? x / P : x % D;
      if (i < n) amax = fmaxf(amax, fabsf(get(i, d)));
    }
    amax = wave_max(amax);
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float s = fmaxf(amax, kAmaxFloor) / 127.0f;
    if (tid == 0) (value ? a.c.v_scale : a.c.k_scale)[dest] = s;
    for (int x = tid; x < P * D; x += kThreads) {
      const int i = value ? x % P : x / D, d = value ? x / P : x % D;
      if (i < n) out[x] = static_cast<int8_t>(code_of(get(i, d) / s));
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.

// I2S_OK, or what is wrong with the scores' shape.
inline int check_shape(float scale, int64_t window, float cap, const float *slopes, const int32_t *prefix) {
  if (window < 0 || !(fabsf(scale) < INFINITY)) return I2S_EINVAL;
  if (!(cap == 0.0f || (cap >= 0x1p-60f && cap <= 0x1p60f)) || !aligned(slopes, 4) || !aligned(prefix, 4)) return I2S_EINVAL;
  return I2S_OK;
}

// Tokens of a batch's sequences that a grid is laid out for.
inline int64_t tokens_of(const kv8_batch *batch, const Cache &c, const Batch &s) {
  const int64_t held = static_cast<int64_t>(s.blocks) << c.lp;
  return batch->max_len > 0 && batch->max_len < held ? batch->max_len : held;
}

// Workgroups for `wanted` pieces of each of `each` sequences and heads, at
// least one: fewer where a grid could not hold them (they then take several).
inline int pieces_of(int64_t wanted, int64_t each) {
  const int64_t most = 0x7fffffff / (each > 0 ? each : 1);
  return static_cast<int>(wanted < 1 ? 1 : wanted < most ? wanted : most);
}

}  // namespace

extern "C" int kv8_attention_scored(const kv8_cache *cache, const kv8_batch *batch, int type, const void *q, int64_t q_stride,
                                    int64_t q_heads, int64_t rows, float scale, int causal, int64_t window, float cap,
                                    const float *slopes, const int32_t *prefix, void *out, int64_t out_stride, float *lse,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  Shaped a;
  if (const int st = check_attention(cache, batch, type, q_heads, rows, a.c, a.s)) return st;
  if (const int st = check_shape(scale, window, cap, slopes, prefix)) return st;
  a.cap = cap * kLog2e;
  a.icap = cap > 0.0f ? 1.0f / a.cap : 0.0f;
  a.slopes = slopes;
  a.prefix = prefix;
  const Rowset r = {q, q_stride, q_heads, rows, out, out_stride, lse, workspace, workspace_bytes};
  return attend(a, batch, type, r, scale, causal, window, stream);
}

extern "C" size_t kv8_weigh_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch, int64_t q_heads, int64_t rows) {
  return 0;
}

extern "C" int kv8_weigh(const kv8_cache *cache, const kv8_batch *batch, int type, const void *q, int64_t q_stride,
                         int64_t q_heads, int64_t rows, float scale, int causal, int64_t window, float cap,
                         const float *slopes, const int32_t *prefix, const float *lse, float *mass, void *workspace,
                         size_t workspace_bytes, void *stream) {
  Weigh a;
  if (const int st = check_attention(cache, batch, type, q_heads, rows, a.c, a.s)) return st;
  if (const int st = check_shape(scale, window, cap, slopes, prefix)) return st;
  if (rows == 0 || a.s.seqs == 0) return I2S_OK;
  if (const int st = check_rows(q, q_stride, q_heads * a.c.dim, value_bytes(type))) return st;
  if (!lse || !aligned(lse, 4) || !mass || !aligned(mass, 4)) return I2S_EINVAL;
  if (rows * q_heads > 0x7fffffff) return I2S_ERANGE;
  a.q = q;
  a.lse = lse;
  a.slopes = slopes;
  a.prefix = prefix;
  a.mass = mass;
  a.q_stride = q_stride;
  a.scale = scale * kLog2e;
  a.cap = cap * kLog2e;
  a.icap = cap > 0.0f ? 1.0f / a.cap : 0.0f;
  a.window = static_cast<int>(window_of(window));
  a.q_heads = static_cast<int>(q_heads);
  a.group = static_cast<int>(q_heads / a.c.heads);
  a.causal = causal != 0;
  const int64_t each = static_cast<int64_t>(a.s.seqs) * a.c.heads;
  a.blocks = pieces_of((tokens_of(batch, a.c, a.s) + kThreads - 1) / kThreads, each);
  return by_type(type, [&](auto t) {
    weigh_kernel<decltype(t)><<<static_cast<unsigned>(each * a.blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
    return hip_status();
  });
}

extern "C" int kv8_choose(const kv8_cache *cache, const kv8_batch *batch, const float *mass, int64_t keep, int64_t first,
                          int64_t recent, int32_t *index, int32_t *kept, void *stream) {
  Choose a;
  if (const int st = check_batch(cache, batch, KV8_F32, 0, a.c, a.s)) return st;
  if (keep < 0 || first < 0 || recent < 0 || first > keep || recent > keep - first) return I2S_EINVAL;
  if (keep > kMaxRows - 1024 || (static_cast<int64_t>(a.s.blocks) << a.c.lp) > kMaxRows - 1024) return I2S_ERANGE;
  if (a.s.seqs == 0) return I2S_OK;
  if (!mass || !aligned(mass, 4) || (keep > 0 && !index) || !aligned(index, 4) || !kept || !aligned(kept, 4)) return I2S_EINVAL;
  a.mass = mass;
  a.keep = keep;
  a.first = static_cast<int>(first);
  a.recent = static_cast<int>(recent);
  a.index = index;
  a.kept = kept;
  choose_kernel<<<static_cast<unsigned>(a.s.seqs * a.c.heads), kChooseThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return hip_status();
}

extern "C" int kv8_move(const kv8_cache *cache, const kv8_batch *batch, const int32_t *index, const int32_t *kept, int64_t keep,
                        const int32_t *to_table, int64_t to_stride, int64_t to_blocks, float *mass, void *stream) {
  Move a;
  if (const int st = check_batch(cache, batch, KV8_F32, 0, a.c, a.s)) return st;
  if (keep < 0 || to_blocks < 0 || to_stride < to_blocks) return I2S_EINVAL;
  if (keep > kMaxRows - 1024 || to_blocks > 0x7fffffff || to_stride > kMaxStride) return I2S_ERANGE;
  if (a.s.seqs == 0 || keep == 0 || to_blocks == 0) return I2S_OK;
  if (!index || !aligned(index, 4) || !kept || !aligned(kept, 4) || !to_table || !aligned(to_table, 4) || !aligned(mass, 4))
    return I2S_EINVAL;
  a.index = index;
  a.kept = kept;
  a.to = to_table;
  a.keep = keep;
  a.to_stride = to_stride;
  a.to_blocks = static_cast<int>(to_blocks);
  a.mass = mass;
  const int64_t wanted = (keep + (INT64_C(1) << a.c.lp) - 1) >> a.c.lp, each = static_cast<int64_t>(a.s.seqs) * a.c.heads * 2;
  a.blocks = pieces_of(wanted < to_blocks ? wanted : to_blocks, each);
  move_kernel<<<static_cast<unsigned>(each * a.blocks), kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  return hip_status();
}
