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
// columns of S = Q K^T: their codes stay in registers, turned into f16 once (which
// holds them exactly), and the rows that see any of them pass by in
// stages of 64 through shared memory, where each wave lays down 16 rows.  Lane
// (n, g) gets the logits of token n of a 16-token tile and rows 4 g .. 4 g + 3,
// so a token's sum stays in its lane until the end.  Tokens that are none need
// no mask: nothing of their columns is written.
// Queries: F16 is an operand as it is, BF16 is exact when brought to 2^15 by a
// power of two (to 2^-40 of the row's largest magnitude), F32 is then the sum of
// two f16 (22 bits).
// Few token blocks are split along their rows into parts of whole stages; the
// parts' sums are joined in order.
//
// A prompt of 4096 F32 rows, 12 heads over 2 of 128: 80 us, 0.32 PFLOP/s of the
// formula's operations (two f16 a query double them); the matrix units are busy in
// 27% of the SIMDs' cycles, vector instructions (a weight's scale, exponent and
// sum, the queries' two parts) in 43%, the rest is a workgroup's begin and the
// barriers of its stages.  Blocks of 512 tokens (two waves a SIMD, 103 us against
// then 82) and a tile's operands read ahead (91) were slower.

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
constexpr int kLeastStages = 2;  // of a part

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

// A row on its way to shared memory: lane g takes 16 bytes of every 64, so that a
// load's four lanes of a row are neighbours.
template <typename T, int kChunks>
struct Queries {
  typedef typename Row<T>::Vec Vec;
  static constexpr int kLoads = 16 * kChunks / Row<T>::kValues;
  Vec q[kLoads];
  float lse;
  int i, hq;  // query token of the sequence, query head
  bool live;

  // Row `row` of the sequence's rows below `end`, for row0 one of them.
  __device__ void load(const Weigh &a, const Span &p, int h, int D, int row, int end, int row0) {
    const int g = (threadIdx.x & 63) >> 4;
    live = row < end;
    i = a.by_group.of(live ? row : row0);
    hq = h * a.group + (live ? row : row0) - i * a.group;
    lse = a.lse[static_cast<int64_t>(p.first + i) * a.q_heads + hq];
    const T *src = static_cast<const T *>(a.q) + (p.first + i) * a.q_stride + static_cast<int64_t>(hq) * D;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int d = (4 * k + g) * Row<T>::kValues;
      q[k] = Vec{};
      if (d < D) q[k] = *reinterpret_cast<const Vec *>(src + d);
    }
  }
};

// A stage's rows in shared memory, as operands, and what their weights take.
template <typename T, int kChunks, bool kShaped>
struct Stage {
  static constexpr int kTerms = std::is_same<T, float>::value ? 2 : 1, kTiles = 4;
  typedef f16x8 Op;
  typedef typename Row<T>::Vec Vec;
  static constexpr int kLoads = Queries<T, kChunks>::kLoads;
  Op op[kTiles][kChunks][2][kTerms][64];
  f32x4 factor[kTiles][4], less[kTiles][4], slope[kShaped ? kTiles : 1][4];
  i32x4 place[kTiles][4];

  // The wave's rows to tile `tile`.
  __device__ void lay_down(const Weigh &a, Queries<T, kChunks> &row, int tile, int own) {
    const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const bool adds = row.live && fabsf(row.lse) < INFINITY;
    if (__any(!adds)) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) row.q[k] = adds ? row.q[k] : Vec{};
    }
    float qs = a.scale;
    int shift = 0;
    if constexpr (!std::is_same<T, f16>::value) {
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
#pragma unroll
        for (int m = 0; m < Row<T>::kValues; ++m) amax = fmaxf(amax, fabsf(static_cast<float>(row.q[k][m])));
      }
      amax = over_lanes_max(amax);
      // amax <= 127/128 2^over: an f16 is below 2^15.  A NaN or an infinity
      // makes its row's products NaN.
      shift = 14 - __builtin_amdgcn_frexp_expf(amax * 0.504f);
      qs = ldexpf(qs, -shift);
    }
    if constexpr (kTerms == 2) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        // Components 16 k + 4 g ..: of chunk k / 4 and of lane 16 (k % 4) + n
        // there, half g / 2, its lower or upper four.
        union {
          f16x2 pair[2];
          f32x2 all;
        } term[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float y0 = ldexpf(row.q[k][2 * m], shift), y1 = ldexpf(row.q[k][2 * m + 1], shift);
          term[0].pair[m] = f16x2{static_cast<f16>(y0), static_cast<f16>(y1)};
          term[1].pair[m] = rest_of(y0, y1, term[0].pair[m]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
          reinterpret_cast<f32x2 *>(&op[tile][k / 4][g >> 1][m][16 * (k % 4) + n])[g & 1] = term[m].all;
      }
    } else {
      // Components 32 k + 8 g ..: lane 16 (2 (k % 2) + g / 2) + n, half g % 2.
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        f16x8 term;
        if constexpr (std::is_same<T, f16>::value) {
          term = row.q[k];
        } else {
#pragma unroll
          for (int m = 0; m < 8; ++m) term[m] = static_cast<f16>(ldexpf(static_cast<float>(row.q[k][m]), shift));
        }
        op[tile][k / 2][g & 1][0][16 * (2 * (k % 2) + (g >> 1)) + n] = term;
      }
    }
    if (g == 0) {
      reinterpret_cast<float *>(factor)[16 * tile + n] = adds ? kShaped ? in_range(qs) : qs : 0.0f;
      reinterpret_cast<float *>(less)[16 * tile + n] = adds ? -row.lse * kLog2e : -INFINITY;
      reinterpret_cast<int *>(place)[16 * tile + n] = own + row.i;
      if constexpr (kShaped) reinterpret_cast<float *>(slope)[16 * tile + n] = adds ? slope_of(a.slopes, row.hq) : 0.0f;
    }
  }

  // Exponents, in units of log2, of a tile's rows 4 g .. and the tokens n of the
  // four 16-token tiles from tw on: f their products, ks the tokens' scales.
  // edge: some row does not see some token.
  __device__ void exponents(const Weigh &a, int tile, const f32x4 (&f)[4], const float (&ks)[4], int tw, int prefix, int64_t far, bool edge,
                            float (&e)[16]) const {
    const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const f32x4 qs = factor[tile][g], off = less[tile][g];
    if constexpr (kShaped) {
      // Before a cap a score may be past F32's range: see Rows::weigh.
#pragma unroll
      for (int k = 0; k < 16; ++k) e[k] = f[k / 4][k % 4] * __builtin_amdgcn_fmed3f(qs[k % 4] * ks[k / 4], -FLT_MAX, FLT_MAX);
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
  }
};

template <typename T, int kChunks, bool kFull, bool kShaped>
__global__ void __launch_bounds__(kThreads, kChunks > 2 ? 1 : kChunks == 2 ? 3 : 4) weigh_kernel(Weigh a) {
  typedef Stage<T, kChunks, kShaped> S;
  typedef typename S::Op Op;
  constexpr int kTerms = S::kTerms, kTiles = S::kTiles;
  __shared__ S laid;
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

    // The wave's tokens: lane's own is tw + lane; those of a 16-token tile share a
    // page.  Loads in the order of their uses: pages, queries, then what waits for
    // the pages.
    const int tw = t0 + 64 * wave, tl = tw + lane;
    const int entry = a.s.table[b * a.s.table_stride + ((tl < top ? tl : top - 1) >> a.c.lp)];

    Queries<T, kChunks> row;  // n of the wave's tile of a stage
    auto has_rows = [&](int stage) { return r.lo + stage * kStage + 16 * wave < r.hi; };
    auto load = [&](int stage) { row.load(a, p, h, D, r.lo + stage * kStage + 16 * wave + n, r.hi, r.lo); };
    auto lay_down = [&]() { laid.lay_down(a, row, wave, own); };
    if (first < last && has_rows(first)) load(first);
    const int page = tl < top && static_cast<unsigned>(entry) < static_cast<unsigned>(a.c.pages) ? entry : -1;
    const float scale = a.c.k_scale[static_cast<int64_t>(page < 0 ? 0 : page) * a.c.heads + h];
    i32x4 codes[4][kChunks];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = __builtin_amdgcn_readlane(page, 16 * j);
      const int slot = (tw + 16 * j) & ((1 << a.c.lp) - 1);
      const int8_t *k = a.c.k + (((static_cast<int64_t>(at < 0 ? 0 : at) * a.c.heads + h) << a.c.lp) + slot + n) * D + 16 * g;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        codes[j][c] = i32x4{0, 0, 0, 0};
        if (kFull || 64 * c + 16 * g < D) codes[j][c] = *reinterpret_cast<const i32x4 *>(k + 64 * c);
      }
    }

    float total[4] = {0.0f, 0.0f, 0.0f, 0.0f}, ks[4];
    Op kop[4][kChunks][2];
    __syncthreads();  // the block before has been read
    if (first < last && has_rows(first)) lay_down();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ks[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), 16 * j));
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int z = 0; z < 2; ++z) kop[j][c][z] = codes_to_f16(codes[j][c][2 * z], codes[j][c][2 * z + 1]);
      }
    }
    for (int stage = first; stage < last; ++stage) {
      const bool more = stage + 1 < last && has_rows(stage + 1);
      __syncthreads();
      if (more) load(stage + 1);
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int tile = 0; tile < kTiles; ++tile) {
        const int row0 = r.lo + stage * kStage + 16 * tile;
        if (row0 >= r.hi || tw >= top) break;
        const int p0 = own + a.by_group.of(row0), p1 = own + a.by_group.of(row0 + 15 < r.hi ? row0 + 15 : r.hi - 1);
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
              const Op q = laid.op[tile][c][z][m][lane];
#pragma unroll
              for (int j = 0; j < 4; ++j) f[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q, kop[j][c][z], f[j], 0, 0, 0);
            }
          }
        }
        float e[16];
        laid.exponents(a, tile, f, ks, tw, prefix, far, edge, e);
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[k / 4] += __builtin_amdgcn_exp2f(e[k]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) total[j] += sum[j];
      __syncthreads();
      if (more) lay_down();
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

constexpr int kHeldBlocks = 4;  // whose sums a workgroup of few rows holds over the stages

// Few rows (a decode step): a workgroup keeps a stage of rows in shared memory
// and walks blocks of tokens, `blocks` apart; a wave's codes of the next block are
// loaded into the registers that its products have just left, the pages are
// looked up one block further ahead, and no wave waits for another.  Rows past a
// stage are another walk, over kHeldBlocks blocks at a time.
// One token of each of 64 sequences of 500 to 8000 tokens, 32 query heads over 8
// of 128, BF16: 66 us for 299 MB (4.5 TB/s), bound by how much of the cache is on
// its way with four waves a SIMD; weigh_kernel, with three and a begin for every
// block, takes 76.
template <typename T, int kChunks, bool kFull, bool kShaped>
__global__ void __launch_bounds__(kThreads, (kChunks > 2 ? 2 : 4)) weigh_few_kernel(Weigh a) {
  typedef Stage<T, kChunks, kShaped> S;
  typedef typename S::Op Op;
  constexpr int kTerms = S::kTerms, kTiles = S::kTiles;
  __shared__ S laid;
  __shared__ float held_sums[kHeldBlocks][kBlockTokens];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int D = kFull ? 64 * kChunks : a.c.dim;
  const int x = a.c.by_heads.of(blockIdx.x), h = blockIdx.x - x * a.c.heads;
  const int b = a.by_blocks.of(x), block0 = x - b * a.blocks;
  const Span p = span_of(a.s, b);
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len, own = p.len - p.n;
  const int prefix = a.prefix ? a.prefix[b] : 0;
  // The first block that the first row sees of, where there is a window.
  const int64_t seen = a.window > 0 ? static_cast<int64_t>(own) - a.window + 1 : 0;
  const int64_t begin = (seen > 0 ? seen & -kBlockTokens : 0) + static_cast<int64_t>(block0) * kBlockTokens;
  if (p.n == 0 || begin >= top) return;
  const int rows = p.n * a.group, pages = a.c.pages;
  const int64_t stride = static_cast<int64_t>(a.blocks) * kBlockTokens;
  const int32_t *table = a.s.table + b * a.s.table_stride;
  const int64_t far = a.window > 0 ? a.window : INT64_C(1) << 40;

  // With one stage all blocks in one go; else as many as there is room to hold the
  // sums of, so that a token's weights reach the mass as one sum.
  const int64_t reach = rows <= kStage ? top : kHeldBlocks * stride;
  for (int64_t from = begin; from < top; from += reach) {
    const int64_t end = from + reach < top ? from + reach : top;
    for (int row0 = 0; row0 < rows; row0 += kStage) {
      __syncthreads();  // the stage before has been read
      if (row0 + 16 * wave < rows) {
        Queries<T, kChunks> row;
        row.load(a, p, h, D, row0 + 16 * wave + n, rows, row0);
        laid.lay_down(a, row, wave, own);
      }
      __syncthreads();
      const int tiles = (rows - row0 + 15) / 16 < kTiles ? (rows - row0 + 15) / 16 : kTiles;
      int64_t t0 = from + 64 * wave;
      if (t0 >= end) continue;
      int turn = 0;
      auto entry_of = [&](int64_t t) { return table[((t + lane < top ? static_cast<int>(t) + lane : top - 1)) >> a.c.lp]; };
      int page = entry_of(t0), then = entry_of(t0 + stride);
      float scale;
      i32x4 codes[4][kChunks];
      auto fetch = [&](int64_t t) {
        page = t + lane < top && static_cast<unsigned>(page) < static_cast<unsigned>(pages) ? page : -1;
        scale = a.c.k_scale[static_cast<int64_t>(page < 0 ? 0 : page) * a.c.heads + h];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = __builtin_amdgcn_readlane(page, 16 * j);
          const int slot = (static_cast<int>(t) + 16 * j) & ((1 << a.c.lp) - 1);
          const int8_t *k = a.c.k + (((static_cast<int64_t>(at < 0 ? 0 : at) * a.c.heads + h) << a.c.lp) + slot + n) * D + 16 * g;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            codes[j][c] = i32x4{0, 0, 0, 0};
            if (kFull || 64 * c + 16 * g < D) codes[j][c] = *reinterpret_cast<const i32x4 *>(k + 64 * c);
          }
        }
      };
      fetch(t0);
      while (true) {
        const int tw = static_cast<int>(t0), mine = page, tend = tw + 64 < top ? tw + 64 : top;
        float ks[4], total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) ks[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), 16 * j));
        for (int tile = 0; tile < tiles; ++tile) {
          const int row = row0 + 16 * tile;
          const int p0 = own + a.by_group.of(row), p1 = own + a.by_group.of(row + 15 < rows ? row + 15 : rows - 1);
          const bool early = tend <= prefix || !a.causal;  // in front of what all rows see
          const bool none = (!early && tw >= prefix && tw > p1) || tend - 1 <= p0 - far;  // no row sees any
          const bool edge = (!early && tend - 1 > p0) || tw <= p1 - far;
          f32x4 f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (!none) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                Op q[kTerms];
#pragma unroll
                for (int m = 0; m < kTerms; ++m) q[m] = laid.op[tile][c][z][m][lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const Op k = codes_to_f16(codes[j][c][2 * z], codes[j][c][2 * z + 1]);
#pragma unroll
                  for (int m = 0; m < kTerms; ++m) f[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[m], k, f[j], 0, 0, 0);
                }
              }
            }
          }
          if (tile + 1 == tiles && t0 + stride < end) {
            page = then;
            fetch(t0 + stride);
            then = entry_of(t0 + 2 * stride);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (none) continue;
          float e[16];
          laid.exponents(a, tile, f, ks, tw, prefix, far, edge, e);
#pragma unroll
          for (int k = 0; k < 16; ++k) total[k / 4] += __builtin_amdgcn_exp2f(e[k]);
        }
        float w = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v = over_lanes_sum(total[j]);
          w = g == j ? v : w;
        }
        if (row0 > 0) w += held_sums[turn][threadIdx.x];
        if (row0 + kStage < rows) {
          held_sums[turn][threadIdx.x] = w;
        } else if (mine >= 0) {
          settle_mass(a, mine, h, tw + lane, tw + lane >= own, w);
        }
        t0 += stride;
        if (t0 >= end) break;
        ++turn;
      }
    }
  }
}

// Joins the parts of token blocks that were split: a workgroup has 64 tokens, 16
// teams of 16 lanes sum every 16th part (a thread a token and all parts in turn
// took 19 us for a prompt of 4096, 64 parts).
constexpr int kJoinTokens = 64, kTeams = 16;

__global__ void __launch_bounds__(kThreads) weigh_join_kernel(Weigh a) {
  __shared__ f32x4 sum[kTeams][kJoinTokens / 4];
  const int h = blockIdx.x % a.c.heads, x = blockIdx.x / a.c.heads;
  constexpr int kPer = kBlockTokens / kJoinTokens;
  const int b = a.by_blocks.of(x / kPer), block = x / kPer - b * a.blocks;
  const Span p = span_of(a.s, b);
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < p.len ? static_cast<int>(held) : p.len, t0 = block * kBlockTokens, part0 = x % kPer * kJoinTokens;
  if (p.n == 0 || t0 + part0 >= top) return;
  const Passing r = passing(a, p, t0, t0 + kBlockTokens < top ? t0 + kBlockTokens : top, true);
  if (r.stages <= r.each) return;
  const int team = threadIdx.x >> 4, lane = threadIdx.x & 15, used = (r.stages + r.each - 1) / r.each;
  const int64_t all = static_cast<int64_t>(a.s.seqs) * a.c.heads * a.blocks;
  const float *at = a.sums + ((static_cast<int64_t>(b) * a.c.heads + h) * a.blocks + block) * kBlockTokens + part0 + 4 * lane;
  f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int k = team; k < used; k += kTeams) w += *reinterpret_cast<const f32x4 *>(at + k * all * kBlockTokens);
  sum[team][lane] = w;
  __syncthreads();
  if (threadIdx.x >= kJoinTokens) return;
  const int t = t0 + part0 + threadIdx.x;
  const int page = t < top ? page_of(a.s, b, t >> a.c.lp, a.c.pages) : -1;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < kTeams; ++k) v += reinterpret_cast<const float *>(sum[k])[threadIdx.x];
  if (page >= 0) settle_mass(a, page, h, t, t >= p.len - p.n, v);
}

// ---------------------------------------------------------------------------
// The choice of the tokens that stay.

constexpr int kBins = 2048;

struct Choose {
  Cache c;
  Batch s;
  const float *mass;
  int keep, first, recent;
  int32_t *index, *kept;
};

// A number that rises with the mass, 1 for a NaN.  0 is left for a token that
// is none, the largest for one that always stays.
__device__ inline uint32_t rank_of(float mass) {
  const uint32_t u = __float_as_uint(mass + 0.0f);  // -0 is 0
  return mass != mass ? 1 : u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

template <int kCtrl, int kRows>
__device__ inline int dpp_or_zero(int v) { return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xF, false); }

// Sum over the wave's lanes up to this one.
__device__ inline int wave_scan(int v) {
  v += dpp_or_zero<0x111, 0xF>(v);  // row_shr:1
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);  // row_bcast:15, to rows 1 and 3
  v += dpp_or_zero<0x143, 0xC>(v);  // row_bcast:31, to rows 2 and 3
  return v;
}

// A workgroup has a sequence and head, a lane four neighbouring tokens of each
// of kLoads rounds, whose ranks stay in registers; a sequence of more tokens is
// walked in segments, each pass again.  The least rank that stays is found in
// digits of 11, 11 and 10 bits from the highest, with a histogram of the ranks
// that begin with the digits found; then the tokens are written in order.
// A bin is four counters, of lanes 0, 4, ..; 1, 5, .. and so on: masses share
// few exponents, and lanes that add to one counter take turns.
// A sequence and head is one compute unit's work, bound by its barriers where it
// is short and by its vector instructions (ranks, histograms, places) where it is
// long: 2 of 65536 tokens 27 us, 384 of 1000 to 9000 14 us.
template <int kChooseThreads, int kLoads>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(Choose a) {
  constexpr int kChooseWaves = kChooseThreads / 64, kSegment = kLoads * kChooseThreads * 4, kMine = kBins / kChooseThreads;
  typedef float F4 __attribute__((ext_vector_type(4), aligned(4)));
  typedef int I4 __attribute__((ext_vector_type(4)));
  __shared__ I4 hist[kBins];
  __shared__ int waves[kChooseWaves], pick[2];
  __shared__ int base[2][kLoads * kChooseWaves];
  const int b = a.c.by_heads.of(blockIdx.x), h = blockIdx.x - b * a.c.heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int length = a.s.lens[b] > 0 ? a.s.lens[b] : 0;
  const int64_t held = static_cast<int64_t>(a.s.blocks) << a.c.lp;
  const int top = held < length ? static_cast<int>(held) : length;
  const int newest = length - a.recent;  // tokens from here on stay
  const int segments = top > 0 ? (top - 1) / kSegment + 1 : 0;
  uint32_t rank[kLoads][4];
  auto load = [&](int segment) {
    const int begin = segment * kSegment + 4 * tid;
    int entry[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t t = begin + static_cast<int64_t>(i) * (4 * kChooseThreads);
      entry[i] = a.s.table[b * a.s.table_stride + ((t < top ? t : top - 1) >> a.c.lp)];
    }
    F4 m[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int page = static_cast<unsigned>(entry[i]) < static_cast<unsigned>(a.c.pages) ? entry[i] : 0;
      const int slot = (begin + i * (4 * kChooseThreads)) & ((1 << a.c.lp) - 1);
      m[i] = *reinterpret_cast<const F4 *>(a.mass + ((static_cast<int64_t>(page) * a.c.heads + h) << a.c.lp) + slot);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool hole = static_cast<unsigned>(entry[i]) >= static_cast<unsigned>(a.c.pages);
      const int64_t t = begin + static_cast<int64_t>(i) * (4 * kChooseThreads);
#pragma unroll
      for (int k = 0; k < 4; ++k) rank[i][k] = rank_of(m[i][k]);
      if (__any(hole || t < a.first || t + 3 >= newest || t + 3 >= top)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rank[i][k] = t + k < a.first || t + k >= newest ? 0xffffffffu : rank[i][k];
          rank[i][k] = hole || t + k >= top ? 0 : rank[i][k];
        }
      }
    }
  };

  int *counter = reinterpret_cast<int *>(hist) + (tid & 3);
  uint32_t least = 0;
  int want = a.keep, total = 0;  // want: of the ranks that begin with least's digits
  if (segments == 1) load(0);
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0}, kAbove[3] = {32, 21, 10};
#pragma unroll
    for (int i = 0; i < kMine; ++i) hist[tid + i * kChooseThreads] = I4{0, 0, 0, 0};
    __syncthreads();
    for (int segment = 0; segment < segments; ++segment) {
      if (segments > 1) load(segment);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (pass == 2) {  // few waves still have one
          bool any = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) any |= (rank[i][k] >> kAbove[pass]) == (least >> kAbove[pass]);
          if (!__any(any)) continue;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t r = rank[i][k];
          const bool in = pass == 0 ? r != 0 : (r >> kAbove[pass]) == (least >> kAbove[pass]);
          if (in) atomicAdd(counter + 4 * ((r >> kShift[pass]) & (pass == 2 ? 1023 : kBins - 1)), 1);
        }
      }
    }
    __syncthreads();
    // Bins from the highest: a thread has kMine.
    int bins[kMine], mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const I4 four = hist[kBins - 1 - i - kMine * tid];
      bins[i] = (four[0] + four[1]) + (four[2] + four[3]);
      mine += bins[i];
    }
    int upto = wave_scan(mine);
    if (lane == 63) waves[wave] = upto;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kChooseWaves; ++i) {
      upto += i < wave ? waves[i] : 0;
      sum += waves[i];
    }
    if (pass == 0) {
      total = sum;
      if (total <= a.keep) break;
    }
    int before = upto - mine;
    if (before < want && want <= upto) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (before < want && want <= before + bins[i]) {
          pick[0] = kBins - 1 - i - kMine * tid;
          pick[1] = want - before;
        }
        before += bins[i];
      }
    }
    __syncthreads();
    least |= static_cast<uint32_t>(pick[0]) << kShift[pass];
    want = pick[1];
  }
  const bool all = total <= a.keep;
  if (all) least = 1, want = total;  // every token, those of rank 1 in order
  int32_t *out = a.index + (static_cast<int64_t>(b) * a.c.heads + h) * a.keep;
  int done = 0, ties = 0;  // tokens over the least rank and at it, of earlier segments
  for (int segment = 0; segment < segments && a.keep > 0; ++segment) {
    if (segments > 1) load(segment);
    __syncthreads();  // base has been read
    int upto[kLoads];  // tokens over the least rank of the lanes up to this one, and at it, in 16 bits each
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int count = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        count += rank[i][k] > least ? 1 : 0;
        count += rank[i][k] == least ? 1 << 16 : 0;
      }
      upto[i] = wave_scan(count);
      if (lane == 63) {
        base[0][i * kChooseWaves + wave] = upto[i] & 0xffff;
        base[1][i * kChooseWaves + wave] = upto[i] >> 16;
      }
      upto[i] -= count;
    }
    __syncthreads();
    if (wave < 2) {  // sums in front of each
      int carry = wave == 0 ? done : ties;
      for (int i = 0; i < kLoads * kChooseWaves; i += 64) {
        const bool in = i + lane < kLoads * kChooseWaves;
        const int v = in ? base[wave][i + lane] : 0, sum = wave_scan(v);
        if (in) base[wave][i + lane] = carry + sum - v;
        carry += __builtin_amdgcn_readlane(sum, 63);
      }
      if (lane == 0) pick[wave] = carry;
    }
    __syncthreads();
    done = pick[0];
    ties = pick[1];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int t = segment * kSegment + i * (4 * kChooseThreads) + 4 * tid;
      int over = base[0][i * kChooseWaves + wave] + (upto[i] & 0xffff), at = base[1][i * kChooseWaves + wave] + (upto[i] >> 16);
      // Over the least rank, then those at it that are wanted: `over` counts both.
      at = at < want ? at : want;
      over += at;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool tie = rank[i][k] == least && at < want;
        if (rank[i][k] > least || tie) out[over++] = t + k;
        at += tie;
      }
    }
  }
  const int kept = all ? total : a.keep;
  for (int i = kept + tid; i < a.keep; i += kChooseThreads) out[i] = -1;
  if (h == 0 && tid == 0) a.kept[b] = kept;
}

// ---------------------------------------------------------------------------
// The move of chosen tokens to fresh pages.

struct Move {
  Cache c;
  Batch s;
  const int32_t *index, *kept, *to;
  int64_t to_stride, items;
  int keep, to_blocks, blocks, waves;  // blocks: pages of a sequence in the grid; waves of an item
  float *mass;
  Divisor by_blocks, by_units;  // units: 16 bytes of a token's key
};

constexpr int kMoveUnits = 2, kMoveBytes = 32;  // of a lane at a time
constexpr int kMovePages = 2;                   // source pages that a wave looks at together
constexpr int kTileBytes = 64 * kMoveBytes, kTilePad = 64;  // rows of 64 bytes in different pages: other banks

// The largest and least of codes, in the high bytes of pairs of 16 bits (what is
// below them does not reach up).
struct Extremes {
  typedef short S2 __attribute__((ext_vector_type(2)));
  S2 high = {0, 0}, low = {0, 0};

  __device__ void take(int codes) {
    const S2 odd = __builtin_bit_cast(S2, codes), even = __builtin_bit_cast(S2, codes << 8);
    high = __builtin_elementwise_max(high, __builtin_elementwise_max(odd, even));
    low = __builtin_elementwise_min(low, __builtin_elementwise_min(odd, even));
  }
  __device__ float magnitude() const {
    const int up = (high[0] > high[1] ? high[0] : high[1]) >> 8, down = -((low[0] < low[1] ? low[0] : low[1]) >> 8);
    return static_cast<float>(up > down ? up : down);
  }
};

// Four codes of scale s as codes of scale now: round_half_away((c s) / now),
// |c s| <= 127 now.  With ratio = s (1 / now) c ratio and that quotient, each
// rounded twice, lie within 4 127 2^-24 = 3.1e-5 of each other, so where c ratio
// is 2^-14 and more off the middle of two integers both round to the same: one
// fused product and sum (1.5 * 2^23 leaves the integer lowest), and a second for
// what is left of it.
__device__ inline uint32_t recoded(int codes, float ratio, float s, float now) {
  float r[4], most = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float c = static_cast<float>(static_cast<int8_t>(codes >> (8 * j)));
    r[j] = fmaf(c, ratio, 0x1.8p23f);
    most = fmaxf(most, fabsf(fmaf(c, ratio, 0x1.8p23f - r[j])));
  }
  if (most > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = static_cast<float>(code_of(static_cast<float>(static_cast<int8_t>(codes >> (8 * j))) * s / now)) + 0x1.8p23f;
  }
  return pack_bytes(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]), __float_as_uint(r[3]));
}

// Byte i of the four lanes of a quad, in their order, to its lane i.
__device__ inline uint32_t quad_turned(uint32_t code) {
  const int c = static_cast<int>(code);
  const uint32_t a = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(c, c, 0x00, 0xF, 0xF, false));  // lane 0's
  const uint32_t b = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(c, c, 0x55, 0xF, 0xF, false));
  const uint32_t d = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(c, c, 0xAA, 0xF, 0xF, false));
  const uint32_t e = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(c, c, 0xFF, 0xF, 0xF, false));
  const uint32_t i = threadIdx.x & 3, pair = i | (i + 4) << 8 | 0x0c0c0000u;
  return __builtin_amdgcn_perm(b, a, pair) | __builtin_amdgcn_perm(e, d, pair) << 16;
}

// An item is a page to fill and a head, its keys and values at once: what it
// takes is the chain of count, index, page, codes, maximum and stores, and the
// more of it is on its way at a time the better (keys and values apart: a batch
// of 40 in 132 us, together 115).  Keys are gathered 16 bytes a lane.  Of V,
// tokens innermost, a lane has one token and up to 32 of its components, single
// bytes: a wave brings its components of the pages that its tokens lie in, two
// at a time, to its own part of shared memory in whole lines and picks them there
// (picked from memory, 64 bytes were some 25 accesses of the cache: 272 us).
// Pages of over 64 tokens are picked from memory.  kOnce: the item's codes stay
// in registers between the maximum and the new codes; else they are gathered
// again.
template <bool kOnce, bool kStaged>
__global__ void __launch_bounds__(kThreads) move_kernel(Move a) {
  __shared__ float red[2][kThreads / 64];
  __shared__ i32x4 tiles[kStaged ? kThreads / 64 : 1][kStaged ? kMovePages : 1][(kTileBytes + kTilePad) / 16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (4 / a.waves) + wave / a.waves;
  const int P = 1 << a.c.lp, D = a.c.dim, part = wave % a.waves, first = part * 64 + lane, threads = a.waves * 64;
  const int rest = a.c.by_heads.of(static_cast<int>(item)), h = static_cast<int>(item) - rest * a.c.heads;
  const int b = a.by_blocks.of(rest), j = rest - b * a.blocks;
  const int per = D / 16, begin = j << a.c.lp, left = a.keep - begin;
  const int mine = first & (P - 1);  // the lane's token
  int n = 0, len = 0, chosen = -1;
  int64_t dest = 0;  // page and head
  const int32_t *index = nullptr;
  if (item < a.items) {
    index = a.index + (static_cast<int64_t>(b) * a.c.heads + h) * a.keep + begin;
    // Loads that wait for nothing, together.
    const int asked = a.kept[b], to = a.to[b * a.to_stride + j];
    len = a.s.lens[b];
    chosen = index[mine < left ? mine : left - 1];
    const int kept = asked < a.keep ? asked : a.keep;
    if (begin < kept && to >= 0 && to < a.c.pages) n = kept - begin < P ? kept - begin : P;
    dest = static_cast<int64_t>(to) * a.c.heads + h;
  }
  // The page that a token lies in, -1 for none, and that page's place for the head.
  auto page_of_token = [&](int t) { return t >= 0 && t < len ? page_of(a.s, b, t >> a.c.lp, a.c.pages) : -1; };
  auto at_page = [&](int page) { return static_cast<int64_t>(page) * a.c.heads + h; };
  const int from = mine < n ? page_of_token(chosen) : -1, slot = chosen & (P - 1);

  // Keys: units first, first + threads, ... of 16 bytes.
  const int units = n * per;
  i32x4 key[kMoveUnits];
  float key_scale[kMoveUnits];
  auto load_keys = [&](int u0) {
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const int u = u0 + k * threads, i = a.by_units.of(u);
      int page, s;
      if constexpr (kStaged) {  // lane i has token i
        page = __shfl(from, i & 63);
        s = __shfl(slot, i & 63);
      } else {
        const int t = u < units ? index[i] : -1;
        page = page_of_token(t);
        s = t & (P - 1);
      }
      key[k] = i32x4{0, 0, 0, 0};
      key_scale[k] = 0.0f;
      if (u >= units || page < 0) continue;
      key[k] = reinterpret_cast<const i32x4 *>(a.c.k)[((at_page(page) << a.c.lp) + s) * per + (u - i * per)];
      key_scale[k] = a.c.k_scale[at_page(page)];
    }
  };

  // Values: components start, start + step, ... below end of token `mine`, 32 a
  // round.  Staged: a wave has a share of the components of all tokens.
  const int share = D / a.waves;
  const int start = kStaged ? part * share + (lane >> a.c.lp) : first >> a.c.lp, end = kStaged ? (part + 1) * share : D;
  const int step = (kStaged ? 64 : threads) >> a.c.lp;
  const float value_scale = from < 0 ? 0.0f : a.c.v_scale[at_page(from)];
  int packed[kMoveBytes / 4];
  auto load_values = [&](int d0) {
    if constexpr (kStaged) {
#pragma unroll
      for (int k = 0; k < kMoveBytes / 4; ++k) packed[k] = 0;
      // The wave's rows of a page: components row0 .. row0 + rows - 1.
      const int row0 = __builtin_amdgcn_readfirstlane(d0), rows = end - row0 < kMoveBytes * step ? end - row0 : kMoveBytes * step;
      const int bytes = rows << a.c.lp;
      uint64_t pending = __ballot(from >= 0);
      while (pending) {
        i32x4 tile[kMovePages][2];
        int held = -1;
#pragma unroll
        for (int k = 0; k < kMovePages; ++k) {
          const int page = __builtin_amdgcn_readlane(from, pending ? __builtin_ctzll(pending) : 0);
          const uint64_t same = pending & __ballot(from == page);
          if ((same >> lane) & 1) held = k;
          const i32x4 *src = reinterpret_cast<const i32x4 *>(a.c.v + ((at_page(page < 0 ? 0 : page) * D + row0) << a.c.lp));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            tile[k][u] = i32x4{0, 0, 0, 0};
            if (pending && 16 * (lane + 64 * u) < bytes) tile[k][u] = src[lane + 64 * u];
          }
          pending &= ~same;
        }
#pragma unroll
        for (int k = 0; k < kMovePages; ++k) {
#pragma unroll
          for (int u = 0; u < 2; ++u) tiles[wave][k][lane + 64 * u] = tile[k][u];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (held >= 0) {
          const uint8_t *src = reinterpret_cast<const uint8_t *>(tiles[wave][held]) + ((lane >> a.c.lp) << a.c.lp) + slot;
#pragma unroll
          for (int k = 0; k < kMoveBytes; k += 4) {
            uint8_t byte[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) byte[i] = src[64 * (k + i)];  // step components further on: 64 bytes
            packed[k / 4] = static_cast<int>(pack_bytes(byte[0], byte[1], byte[2], byte[3]));
          }
        }
        __builtin_amdgcn_wave_barrier();
      }
    } else {
      const int8_t *p = a.c.v + ((at_page(from < 0 ? 0 : from) * D + d0) << a.c.lp) + slot;
#pragma unroll
      for (int k = 0; k < kMoveBytes; k += 16) {
        uint8_t byte[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          byte[i] = 0;
          if (d0 + (k + i) * step < D) byte[i] = static_cast<uint8_t>(*p);
          p += step << a.c.lp;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          packed[(k + i) / 4] = static_cast<int>(pack_bytes(byte[i], byte[i + 1], byte[i + 2], byte[i + 3]));
      }
    }
  };

  float amax = 0.0f;
  Extremes values;
  if (n > 0) {
    if (a.mass && start == 0 && mine < n)
      a.mass[(dest << a.c.lp) + mine] = from < 0 ? 0.0f : a.mass[(at_page(from) << a.c.lp) + slot];
    for (int u0 = part * 64; u0 < units; u0 += kMoveUnits * threads) {
      load_keys(u0 + lane);
      if (kOnce) break;
#pragma unroll
      for (int k = 0; k < kMoveUnits; ++k) {
        Extremes x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.take(key[k][i]);
        amax = fmaxf(amax, x.magnitude() * key_scale[k]);  // the largest product is the largest code's
      }
    }
    for (int d0 = start; kStaged ? __builtin_amdgcn_readfirstlane(d0) < end : d0 < end; d0 += kMoveBytes * step) {
      load_values(d0);
#pragma unroll
      for (int k = 0; k < kMoveBytes / 4; ++k) values.take(packed[k]);
      if (kOnce) break;
    }
    if (kOnce && part * 64 < units) {
#pragma unroll
      for (int k = 0; k < kMoveUnits; ++k) {
        Extremes x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x.take(key[k][i]);
        amax = fmaxf(amax, x.magnitude() * key_scale[k]);
      }
    }
  }
  amax = wave_max(amax);
  float vmax = wave_max(values.magnitude() * value_scale);
  if (lane == 0) {
    red[0][wave] = amax;
    red[1][wave] = vmax;
  }
  __syncthreads();
  if (n == 0) return;
  for (int k = 0; k < a.waves; ++k) {
    amax = fmaxf(amax, red[0][wave / a.waves * a.waves + k]);
    vmax = fmaxf(vmax, red[1][wave / a.waves * a.waves + k]);
  }
  const float know = fmaxf(amax, kAmaxFloor) / 127.0f, kinv = 1.0f / know;
  const float vnow = fmaxf(vmax, kAmaxFloor) / 127.0f, vinv = 1.0f / vnow;
  if (first == 0) {
    a.c.k_scale[dest] = know;
    a.c.v_scale[dest] = vnow;
  }
  if (kOnce) {
    // The codes alone are kept until here, not what was made of them: a third of
    // the registers.
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) asm volatile("" : "+v"(key[k]));
#pragma unroll
    for (int k = 0; k < kMoveBytes / 4; ++k) asm volatile("" : "+v"(packed[k]));
  }
  i32x4 *keys = reinterpret_cast<i32x4 *>(a.c.k) + (dest << a.c.lp) * per;
  for (int u0 = part * 64; u0 < units; u0 += kMoveUnits * threads) {
    if (!kOnce) load_keys(u0 + lane);
#pragma unroll
    for (int k = 0; k < kMoveUnits; ++k) {
      const int u = u0 + lane + k * threads;
      if (u >= units) continue;
      i32x4 code;
#pragma unroll
      for (int w = 0; w < 4; ++w) code[w] = static_cast<int>(recoded(key[k][w], key_scale[k] * kinv, key_scale[k], know));
      keys[u] = code;
    }
    if (kOnce) break;
  }
  // Four lanes turn their 4 x 4 bytes: each then has four tokens of one
  // component, and stores four bytes where all four tokens are new ones.
  const bool whole = (mine | 3) < n;
  for (int d0 = start; kStaged ? __builtin_amdgcn_readfirstlane(d0) < end : d0 < end; d0 += kMoveBytes * step) {
    if (!kOnce) load_values(d0);
    int8_t *out = a.c.v + ((dest * D + d0) << a.c.lp) + mine;
    int8_t *out4 = out - (lane & 3) + static_cast<int64_t>(lane & 3) * (step << a.c.lp);
#pragma unroll
    for (int k = 0; k < kMoveBytes; k += 4) {
      const uint32_t code = recoded(packed[k / 4], value_scale * vinv, value_scale, vnow);
      const uint32_t turned = quad_turned(code);
      if (whole) {
        if (d0 + (k + (lane & 3)) * step < end) *reinterpret_cast<uint32_t *>(out4) = turned;
      } else if (mine < n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (d0 + (k + i) * step < end) out[i * (step << a.c.lp)] = static_cast<int8_t>(code >> (8 * i));
      }
      out += 4 * (step << a.c.lp);
      out4 += 4 * (step << a.c.lp);
    }
    if (kOnce) break;
  }
}

// ---------------------------------------------------------------------------
// Host side.

// I2S_OK, or what is wrong with the scores' shape.  A scale within 2^126 is one
// in units of log2, too.
inline int check_shape(float scale, int64_t window, float cap, const float *slopes, const int32_t *prefix) {
  if (window < 0 || !(fabsf(scale) <= 0x1p126f)) return I2S_EINVAL;
  if (!(cap == 0.0f || (cap >= 0x1p-60f && cap <= 0x1p60f)) || !aligned(slopes, 4) || !aligned(prefix, 4)) return I2S_EINVAL;
  return I2S_OK;
}

// Tokens of a batch's sequences that a grid is laid out for.
inline int64_t tokens_of(const kv8_batch *batch, const Cache &c, const Batch &s) {
  const int64_t held = static_cast<int64_t>(s.blocks) << c.lp;
  return batch->max_len > 0 && batch->max_len < held ? batch->max_len : held;
}

// A grid has fewer than 2^32 threads.
inline bool fits(int64_t groups, int threads) { return groups <= 0xffffffffll / threads; }

// Workgroups a unit of calls with few rows, which are on a unit four at a time (8,
// 12, 16 and 32: 70, 68, 67 and 69 us for the batch of 64).
constexpr int kFewGroups = 16;

// How a kv8_weigh call is laid out.
struct WeighPlan {
  int64_t each;  // sequences and heads
  int blocks, parts;
  bool few;
  size_t bytes;

  WeighPlan(const Cache &c, const Batch &s, const kv8_batch *batch, int64_t q_heads) {
    each = static_cast<int64_t>(s.seqs) * c.heads;
    // Workgroups for every block of tokens, or fewer, which then take several
    // each: where a grid could not hold them, and for 16 a unit where no bound of
    // the lengths is known (a table's rows may be far longer than a sequence).
    int64_t most = (0xffffffffll / kThreads) / each;
    if (batch->max_len == 0 && most > 16 * kUnits / each) most = 16 * kUnits / each;
    int64_t all = (tokens_of(batch, c, s) + kBlockTokens - 1) / kBlockTokens;
    if (all > most) all = most;
    // Few rows, up to 32 a sequence and head on average: workgroups that walk
    // several blocks.  64 sequences of 4000 tokens, 8 heads of 128, BF16, with 4, 16,
    // 32, 48 and 64 rows: 47, 49, 62, 77 and 93 us against the other kernel's 55, 56,
    // 67, 75 and 84.  The host knows the mean alone: of 255 sequences with a row
    // each and one with 1000 that one is a few workgroups' work, and 1540 us pass
    // (the two apart 107 and 50).
    few = static_cast<int64_t>(s.rows) * (q_heads / c.heads) <= 32 * static_cast<int64_t>(s.seqs);
    if (few && all > kFewGroups * kUnits / each) all = kFewGroups * kUnits / each;
    blocks = all > 1 ? static_cast<int>(all) : 1;
    // Parts for about eight workgroups a compute unit.
    const int64_t stages = (static_cast<int64_t>(s.rows) * (q_heads / c.heads) + kStage - 1) / kStage;
    int64_t wanted = 16 * kUnits / (each * blocks);
    if (wanted > stages / kLeastStages) wanted = stages / kLeastStages;
    if (few || stages <= kLeastStages * s.seqs) wanted = 1;  // on average there is nothing to split, and a join takes 5 us
    parts = wanted > 1 ? static_cast<int>(wanted) : 1;
    bytes = parts > 1 ? sizeof(float) * kBlockTokens * parts * each * blocks : 0;
  }
};

template <typename T, int kChunks, bool kFull>
int launch_weigh(const WeighPlan &p, const Weigh &a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.each * p.blocks * p.parts);
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a); };
  if (a.cap > 0.0f || a.slopes) {
    launch(p.few ? weigh_few_kernel<T, kChunks, kFull, true> : weigh_kernel<T, kChunks, kFull, true>);
  } else {
    launch(p.few ? weigh_few_kernel<T, kChunks, kFull, false> : weigh_kernel<T, kChunks, kFull, false>);
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
  if (!fits(p.each * p.blocks * p.parts, kThreads)) return I2S_ERANGE;
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
    weigh_join_kernel<<<static_cast<unsigned>(p.each * p.blocks * (kBlockTokens / kJoinTokens)), kThreads, 0, on>>>(a);
    return hip_status();
  });
}

extern "C" int kv8_choose(const kv8_cache *cache, const kv8_batch *batch, const float *mass, int64_t keep, int64_t first,
                          int64_t recent, int32_t *index, int32_t *kept, void *stream) {
  Choose a;
  if (const int st = check_batch(cache, batch, KV8_F32, 0, a.c, a.s)) return st;
  if (keep < 0 || first < 0 || recent < 0 || first > keep || recent > keep - first) return I2S_EINVAL;
  if (keep > kMaxRows - 1024 || (static_cast<int64_t>(a.s.blocks) << a.c.lp) > kMaxRows - 65536) return I2S_ERANGE;
  if (a.s.seqs == 0) return I2S_OK;
  if (!mass || !aligned(mass, 4) || (keep > 0 && !index) || !aligned(index, 4) || !kept || !aligned(kept, 4)) return I2S_EINVAL;
  a.mass = mass;
  a.keep = static_cast<int>(keep);
  a.first = static_cast<int>(first);
  a.recent = static_cast<int>(recent);
  a.index = index;
  a.kept = kept;
  if (!fits(static_cast<int64_t>(a.s.seqs) * a.c.heads, 1024)) return I2S_ERANGE;
  const int64_t tokens = tokens_of(batch, a.c, a.s);
  auto launch = [&](auto kernel, int threads) {
    kernel<<<static_cast<unsigned>(a.s.seqs * a.c.heads), threads, 0, static_cast<hipStream_t>(stream)>>>(a);
    return hip_status();
  };
  // As few threads as keep 16 or 32 ranks each: their barriers are the cheaper
  // (384 sequences and heads of up to 4000 tokens 11.0 us with 256 threads, 19.8
  // with 1024; 1024 of up to 8000 19.7 with 512, 40.2).  32 ranks where there is
  // a workgroup for every unit (384 of up to 9000 17.1 against 20.9 us, but 2 of
  // up to 16000 12.3 against 11.0).
  if (tokens <= 4096) return launch(choose_kernel<256, 4>, 256);
  if (tokens <= 8192) return launch(choose_kernel<512, 4>, 512);
  if (tokens > 16384) return launch(choose_kernel<1024, 16>, 1024);
  return a.s.seqs * a.c.heads > kUnits ? launch(choose_kernel<512, 8>, 512) : launch(choose_kernel<1024, 4>, 1024);
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
  a.keep = static_cast<int>(keep);
  a.to_stride = to_stride;
  a.to_blocks = static_cast<int>(to_blocks);
  a.mass = mass;
  const int64_t wanted = (keep + (INT64_C(1) << a.c.lp) - 1) >> a.c.lp, P = INT64_C(1) << a.c.lp;
  a.blocks = static_cast<int>(wanted < to_blocks ? wanted : to_blocks);
  a.by_blocks = Divisor(a.blocks);
  a.by_units = Divisor(a.c.dim / 16);
  const int64_t places = static_cast<int64_t>(a.s.seqs) * a.c.heads;
  if (places > 0x7fffffff / a.blocks) return I2S_ERANGE;
  a.items = places * a.blocks;
  a.waves = P * a.c.dim <= 1024 ? 1 : P * a.c.dim <= 2048 ? 2 : 4;
  const int64_t grid = (a.items * a.waves + 3) / 4;
  if (!fits(grid, kThreads)) return I2S_ERANGE;
  auto launch = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, static_cast<hipStream_t>(stream)>>>(a);
  };
  const bool once = P * a.c.dim <= 16 * kMoveUnits * kThreads;
  if (P <= 64) {
    launch(once ? move_kernel<true, true> : move_kernel<false, true>);
  } else {
    launch(once ? move_kernel<true, false> : move_kernel<false, false>);
  }
  return hip_status();
}
