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
//
// A workgroup owns 256 tokens of a sequence and head, a wave 64 of them, as the
// columns of S = Q K^T: their codes stay in registers, turned into f16 or bf16
// once (both hold them exactly), and the rows that see any of them pass by in
// stages of 64 through shared memory, where each wave lays down 16 rows.  Lane
// (n, g) gets the logits of token n of a 16-token tile and rows 4 g .. 4 g + 3,
// so a token's sum stays in its lane until the end.  Tokens that are none need
// no mask: nothing of their columns is written.
// Queries: F16 and BF16 are operands as they are, an F32 query, brought to 2^15
// by a power of two, is the sum of two f16 (22 bits).
// Few token blocks are split along their rows into parts of whole stages; the
// parts' sums are joined in order.

struct Weigh {
  Cache c;
  Batch s;
  const void *q;
  const float *lse, *slopes;
  const int32_t *prefix;
  float *mass, *sums;  // sums [parts][seqs][heads][blocks][kBlockTokens]
  int64_t q_stride;
  float scale, cap, icap;  // in units of log2
  int window, q_heads, group, causal;
  int blocks, parts;  // token blocks of a sequence in the grid, parts of each
  Divisor by_group, by_blocks, by_parts;
};

constexpr int kBlockTokens = 256, kStage = 64;
constexpr int kLeastStages = 4;  // of a part

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Rows [lo, hi) of a sequence see tokens of a block, in `stages` stages, of
// which a part has `each`.
struct Passing {
  int lo, hi, stages, each;
};

__device__ inline Passing passing(const Weigh &a, const Span &p, int t0, int t1, bool split) {
  const int64_t own = static_cast<int64_t>(p.len) - p.n;
  const int prefix = a.prefix ? a.prefix[p.b] : 0;
  int64_t lo = 0, hi = p.n;
  if (a.causal && t0 >= prefix) lo = t0 - own > 0 ? t0 - own : 0;
  if (a.window > 0 && t1 - 1 + static_cast<int64_t>(a.window) - own < hi) hi = t1 - 1 + static_cast<int64_t>(a.window) - own;
  Passing r;
  r.lo = static_cast<int>(lo) * a.group;
  r.hi = hi > lo ? static_cast<int>(hi) * a.group : r.lo;
  r.stages = (r.hi - r.lo + kStage - 1) / kStage;
  r.each = split ? a.by_parts.of(r.stages + a.parts - 1) : r.stages;
  if (split && r.each < kLeastStages) r.each = kLeastStages;
  return r;
}

// Adds a token's weight to its mass, or (one of the call's own) sets it.
__device__ inline void settle_mass(const Weigh &a, int page, int h, int t, bool own, float w) {
  float *mass = a.mass + ((static_cast<int64_t>(page) * a.c.heads + h) << a.c.lp) + (t & ((1 << a.c.lp) - 1));
  if (own) {
    *mass = w;
  } else {
    unsafeAtomicAdd(mass, w);
  }
}

// 16 codes as two operands.
__device__ inline void operands_of(i32x4 codes, f16x8 (&out)[2]) {
#pragma unroll
  for (int z = 0; z < 2; ++z) out[z] = codes_to_f16(codes[2 * z], codes[2 * z + 1]);
}
__device__ inline void operands_of(i32x4 codes, bf16x8 (&out)[2]) {
#pragma unroll
  for (int z = 0; z < 2; ++z) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      out[z][k] = static_cast<bf16>(static_cast<float>(static_cast<int8_t>(codes[2 * z + k / 4] >> (8 * (k % 4)))));
  }
}

__device__ inline f32x4 product(f16x8 q, f16x8 k, f32x4 f) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(q, k, f, 0, 0, 0); }
__device__ inline f32x4 product(bf16x8 q, bf16x8 k, f32x4 f) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, k, f, 0, 0, 0); }

template <typename T, int kChunks, bool kFull, bool kShaped>
__global__ void __launch_bounds__(kThreads, kChunks > 2 ? 1 : 2) weigh_kernel(Weigh a) {
  typedef typename std::conditional<std::is_same<T, bf16>::value, bf16x8, f16x8>::type Op;
  typedef typename Row<T>::Vec Vec;
  constexpr int kVecs = 16 / Row<T>::kValues, kTerms = std::is_same<T, float>::value ? 2 : 1, kTiles = 4;
  __shared__ Op op[kTiles][kChunks][2][kTerms][64];
  __shared__ f32x4 factor[kTiles][4], less[kTiles][4], slope[kShaped ? kTiles : 1][4];
  __shared__ i32x4 place[kTiles][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int D = kFull ? 64 * kChunks : a.c.dim;
  int rest = a.c.by_heads.of(blockIdx.x);
  const int h = blockIdx.x - rest * a.c.heads;
  int x = a.by_parts.of(rest);
  const int part = rest - x * a.parts;
  const int b = a.by_blocks.of(x), block0 = x - b * a.blocks;
  const Span p = span_of(a.s, b);
  if (p.n == 0) return;
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len, own = p.len - p.n;
  const int prefix = a.prefix ? a.prefix[b] : 0;

  // Blocks behind those of the grid (lengths past the bound) are part 0's, whole.
  for (int64_t block = block0; block * kBlockTokens < top; block += a.blocks) {
    const bool split = a.parts > 1 && block < a.blocks;
    if (part > 0 && !split) return;
    const int t0 = static_cast<int>(block) * kBlockTokens, t1 = t0 + kBlockTokens < top ? t0 + kBlockTokens : top;
    const Passing r = passing(a, p, t0, t1, split);
    const int first = part * r.each, last = first + r.each < r.stages ? first + r.each : r.stages;
    if (part > 0 && first >= last) continue;
    if (r.stages == 0 && t1 <= own) continue;  // behind every row's window

    // The wave's tokens: lane's own is tw + lane; those of a 16-token tile share a page.
    const int tw = t0 + 64 * wave, tl = tw + lane;
    const int page = tl < top ? page_of(a.s, b, tl >> a.c.lp, a.c.pages) : -1;
    const float scale = a.c.k_scale[static_cast<int64_t>(page < 0 ? 0 : page) * a.c.heads + h];
    float ks[4];
    i32x4 codes[4][kChunks];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = __builtin_amdgcn_readlane(page, 16 * j);
      ks[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), 16 * j));
      const int slot = (tw + 16 * j) & ((1 << a.c.lp) - 1);
      const int8_t *k = a.c.k + (((static_cast<int64_t>(at < 0 ? 0 : at) * a.c.heads + h) << a.c.lp) + slot + n) * D + 16 * g;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        codes[j][c] = i32x4{0, 0, 0, 0};
        if (kFull || 64 * c + 16 * g < D) codes[j][c] = *reinterpret_cast<const i32x4 *>(k + 64 * c);
      }
    }

    // Row n of the wave's tile of a stage.
    Vec qv[kChunks][kVecs];
    float lse;
    int i, hq;
    bool live;
    auto load = [&](int stage) {
      const int row = r.lo + stage * kStage + 16 * wave + n;
      live = row < r.hi;
      i = a.by_group.of(live ? row : r.lo);
      hq = h * a.group + (live ? row : r.lo) - i * a.group;
      lse = a.lse[static_cast<int64_t>(p.first + i) * a.q_heads + hq];
      const T *src = static_cast<const T *>(a.q) + (p.first + i) * a.q_stride + static_cast<int64_t>(hq) * D + 16 * g;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          qv[c][k] = Vec{};
          if (kFull || 64 * c + 16 * g < D) qv[c][k] = reinterpret_cast<const Vec *>(src + 64 * c)[k];
        }
      }
    };
    auto lay_down = [&]() {
      const bool adds = live && fabsf(lse) < INFINITY;
      float qs = a.scale;
      if constexpr (kTerms == 2) {
        float v[kChunks][16], amax = 0.0f, nan = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            v[c][k] = adds ? qv[c][k / 4][k % 4] : 0.0f;
            amax = fmaxf(amax, fabsf(v[c][k]));
            nan = fmaf(v[c][k], 0.0f, nan);
          }
        }
        if (nan != 0.0f) amax = INFINITY;
        amax = over_lanes_max(amax);
        const int shift = 14 - __builtin_amdgcn_frexp_expf(amax * 0.504f);
        qs = amax < INFINITY ? ldexpf(qs, -shift) : NAN;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            f16x8 term[2];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float y = ldexpf(v[c][8 * z + k], shift);
              term[0][k] = static_cast<f16>(y);
              term[1][k] = static_cast<f16>(y - static_cast<float>(term[0][k]));
            }
            op[wave][c][z][0][lane] = term[0];
            op[wave][c][z][1][lane] = term[1];
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int z = 0; z < 2; ++z) op[wave][c][z][0][lane] = adds ? __builtin_bit_cast(Op, qv[c][z]) : Op{};
        }
      }
      if (g == 0) {
        reinterpret_cast<float *>(factor)[16 * wave + n] = adds ? qs : 0.0f;
        reinterpret_cast<float *>(less)[16 * wave + n] = adds ? -lse * kLog2e : -INFINITY;
        reinterpret_cast<int *>(place)[16 * wave + n] = own + i;
        if constexpr (kShaped) reinterpret_cast<float *>(slope)[16 * wave + n] = a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
      }
    };

    float total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (first < last) load(first);
    Op kop[4][kChunks][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) operands_of(codes[j][c], kop[j][c]);
    }
    for (int stage = first; stage < last; ++stage) {
      __syncthreads();
      lay_down();
      __syncthreads();
      if (stage + 1 < last) load(stage + 1);
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int tile = 0; tile < kTiles; ++tile) {
        const int row = r.lo + stage * kStage + 16 * tile;
        if (row >= r.hi || tw >= top) break;
        const int p0 = own + a.by_group.of(row), p1 = own + a.by_group.of(row + 15 < r.hi ? row + 15 : r.hi - 1);
        const int tend = tw + 64 < top ? tw + 64 : top;
        const bool early = tend <= prefix || !a.causal;  // in front of what all rows see
        const int64_t far = a.window > 0 ? a.window : INT64_C(1) << 40;
        if ((!early && tw >= prefix && tw > p1) || tend - 1 <= p0 - far) continue;  // no row sees any
        const bool edge = (!early && tend - 1 > p0) || tw <= p1 - far;
        f32x4 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int m = 0; m < kTerms; ++m) {
              const Op q = op[tile][c][z][m][lane];
#pragma unroll
              for (int j = 0; j < 4; ++j) f[j] = product(q, kop[j][c][z], f[j]);
            }
          }
        }
        const f32x4 qs = factor[tile][g], off = less[tile][g];
        float e[16];
        if constexpr (kShaped) {
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] = f[k / 4][k % 4] * (qs[k % 4] * ks[k / 4]);
          if (a.cap > 0.0f) capped(e, a.cap, a.icap);
          if (a.slopes) {
            const f32x4 down = slope[tile][g];
            const i32x4 pos = place[tile][g];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              e[k] = fmaf(-down[k % 4], fabsf(static_cast<float>(sub_sat(pos[k % 4], tw + 16 * (k / 4) + n))), e[k]);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] += off[k % 4];
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) e[k] = fmaf(f[k / 4][k % 4], qs[k % 4] * ks[k / 4], off[k % 4]);
        }
        if (edge) {
          const i32x4 pos = place[tile][g];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int t = tw + 16 * (k / 4) + n, at = pos[k % 4];
            const bool seen = (!a.causal || t <= at || t < prefix) && t > at - far;
            e[k] = seen ? e[k] : -INFINITY;
            asm volatile("" : "+v"(e[k]));  // keeps this a branch: few tiles take it
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[k / 4] += __builtin_amdgcn_exp2f(e[k]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) total[j] += sum[j];
    }
    float w = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = over_lanes_sum(total[j]);
      w = g == j ? v : w;
    }
    if (split && r.stages > r.each) {
      const int64_t all = static_cast<int64_t>(a.s.seqs) * a.c.heads * a.blocks;
      a.sums[(part * all + (static_cast<int64_t>(b) * a.c.heads + h) * a.blocks + block) * kBlockTokens + threadIdx.x] = w;
    } else if (page >= 0) {
      settle_mass(a, page, h, tl, tl >= own, w);
    }
  }
}

// Joins the parts of token blocks that were split: a workgroup a block.
__global__ void __launch_bounds__(kThreads) weigh_join_kernel(Weigh a) {
  const int rest = a.c.by_heads.of(blockIdx.x), h = blockIdx.x - rest * a.c.heads;
  const int b = a.by_blocks.of(rest), block = rest - b * a.blocks;
  const Span p = span_of(a.s, b);
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len, t0 = block * kBlockTokens, t = t0 + threadIdx.x;
  if (p.n == 0 || t >= top) return;
  const Passing r = passing(a, p, t0, t0 + kBlockTokens < top ? t0 + kBlockTokens : top, true);
  if (r.stages <= r.each) return;
  const int page = page_of(a.s, b, t >> a.c.lp, a.c.pages);
  if (page < 0) return;
  const int64_t all = static_cast<int64_t>(a.s.seqs) * a.c.heads * a.blocks;
  const float *at = a.sums + ((static_cast<int64_t>(b) * a.c.heads + h) * a.blocks + block) * kBlockTokens + threadIdx.x;
  float w = 0.0f;
  for (int k = 0; k * r.each < r.stages; ++k) w += at[k * all * kBlockTokens];
  settle_mass(a, page, h, t, t >= p.len - p.n, w);
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

// How a kv8_weigh call is laid out.
struct WeighPlan {
  int64_t each;  // sequences and heads
  int blocks, parts;
  size_t bytes;

  WeighPlan(const Cache &c, const Batch &s, const kv8_batch *batch, int64_t q_heads) {
    each = static_cast<int64_t>(s.seqs) * c.heads;
    blocks = pieces_of((tokens_of(batch, c, s) + kBlockTokens - 1) / kBlockTokens, each);
    // Parts for about eight workgroups a compute unit.
    const int64_t stages = (static_cast<int64_t>(s.rows) * (q_heads / c.heads) + kStage - 1) / kStage;
    int64_t wanted = 8 * kUnits / (each * blocks);
    if (wanted > stages / kLeastStages) wanted = stages / kLeastStages;
    parts = wanted > 1 ? static_cast<int>(wanted) : 1;
    bytes = parts > 1 ? sizeof(float) * kBlockTokens * parts * each * blocks : 0;
  }
};

template <typename T, int kChunks, bool kFull>
int launch_weigh(const WeighPlan &p, const Weigh &a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.each * p.blocks * p.parts);
  if (a.cap > 0.0f || a.slopes) {
    weigh_kernel<T, kChunks, kFull, true><<<grid, kThreads, 0, stream>>>(a);
  } else {
    weigh_kernel<T, kChunks, kFull, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return hip_status();
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
  Cache c;
  Batch s;
  if (check_attention(cache, batch, KV8_F32, q_heads, rows, c, s) || rows == 0 || s.seqs == 0) return 0;
  const WeighPlan p(c, s, batch, q_heads);
  return p.bytes;
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
  const WeighPlan p(a.c, a.s, batch, q_heads);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || !aligned(workspace, 256))) return I2S_EWORKSPACE;
  a.q = q;
  a.lse = lse;
  a.slopes = slopes;
  a.prefix = prefix;
  a.mass = mass;
  a.sums = static_cast<float *>(workspace);
  a.q_stride = q_stride;
  a.scale = scale * kLog2e;
  a.cap = cap * kLog2e;
  a.icap = cap > 0.0f ? 1.0f / a.cap : 0.0f;
  a.window = static_cast<int>(window_of(window));
  a.q_heads = static_cast<int>(q_heads);
  a.group = static_cast<int>(q_heads / a.c.heads);
  a.causal = causal != 0;
  a.blocks = p.blocks;
  a.parts = p.parts;
  a.by_group = Divisor(a.group);
  a.by_blocks = Divisor(a.blocks);
  a.by_parts = Divisor(a.parts);
  const hipStream_t on = static_cast<hipStream_t>(stream);
  return by_type(type, [&](auto t) {
    typedef decltype(t) T;
    const int st = a.c.dim == 128  ? launch_weigh<T, 2, true>(p, a, on)
                   : a.c.dim == 64 ? launch_weigh<T, 1, true>(p, a, on)
                   : a.c.dim < 64  ? launch_weigh<T, 1, false>(p, a, on)
                   : a.c.dim < 128 ? launch_weigh<T, 2, false>(p, a, on)
                                   : launch_weigh<T, 4, false>(p, a, on);
    if (st || p.parts == 1) return st;
    weigh_join_kernel<<<static_cast<unsigned>(p.each * p.blocks), kThreads, 0, on>>>(a);
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
