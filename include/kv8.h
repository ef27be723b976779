/* Attention over an int8 K/V cache on MI355X (gfx950): what a decoder layer
 * runs between its q/k/v projections and its o projection.
 *
 *   kv8_qk_norm_rope   per-head RMS norms of queries and keys and the position
 *                      rotation, in one pass
 *   kv8_append         new K/V rows quantized into the cache's pages
 *   kv8_read           cached tokens back as values
 *   kv8_attention      queries over the cache: one token per sequence or many,
 *                      causal, with a sliding window
 *
 * The decoder of "VibeASR in audio.cpp" (Architecture / Decoder: 12 query and
 * 2 K/V heads of width 128, rotation base 1e6, context 65536) fixes the
 * geometry the kernels are built for; the quantization is the convention of
 * the library's other types (a multiplier scale amax/127, amax floored at
 * 1e-5, x / scale rounded half away from zero, clamped to +-127), with one
 * scale per block of tokens and head.
 *
 * The cache is paged.  A page holds `page_tokens` (P) tokens of every K/V
 * head, and is the block that shares a scale:
 *   k       int8 [pages][heads][P][dim]
 *   v       int8 [pages][heads][dim][P]   (tokens innermost: the operand order
 *                                          of the matrix instruction that
 *                                          multiplies by the probabilities)
 *   k_scale, v_scale   F32 [pages][heads], finite, >= 0; value = code * scale
 * A sequence's block j (its tokens j*P .. j*P + P-1) is in page table[b][j].
 * An entry outside 0..pages-1 (-1, say) is a hole: appended rows that fall
 * into one are dropped, reading one gives zeros, attention does not see its
 * tokens (so pages that a window has left behind can be handed on).  Nothing
 * past a sequence's length is read, neither of the table's entries nor of the
 * pages' contents.
 *
 * A batch names the sequences of one call.  `lens[b]` counts the tokens in
 * the cache, those of this call included; the call's rows starts[b] ..
 * starts[b+1]-1 are the newest n_b = starts[b+1] - starts[b] of them, so row
 * starts[b] + i is the token at position lens[b] - n_b + i.  With starts NULL
 * every sequence has rows / seqs rows.  The same batch serves the append, the
 * attention and a read-back of one step.  A row whose position is negative
 * (n_b > lens[b]) is dropped by the append and read back as zeros; a causal
 * attention lets it see nothing, any other what its formula says.  Rows outside
 * starts[0] .. starts[seqs]-1 are left as they were.
 *
 * Conventions as in i2s.h: data pointers are device pointers owned by the
 * caller, on the device that is current; `stream` is a hipStream_t or NULL;
 * arguments are checked on the host before anything is launched, calls
 * neither allocate nor synchronize, and keep nothing from one call to the
 * next.  Structs are host memory, read before the call returns.  Strides are
 * at most 2^40 elements (I2S_ERANGE beyond).  Lengths, starts, positions and
 * the table are read on the device when the kernels run, so a captured graph
 * follows their contents.
 */
#ifndef KV8_H
#define KV8_H

#include <stddef.h>
#include <stdint.h>

#include "i2s.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of rows (queries, keys, values, outputs). */
#define KV8_F32 0
#define KV8_F16 1
#define KV8_BF16 2

#define KV8_MAX_DIM 256
#define KV8_MAX_PAGE 256

typedef struct kv8_cache {
    int8_t *k;            /* [pages][heads][page_tokens][dim], 16-byte aligned */
    int8_t *v;            /* [pages][heads][dim][page_tokens], 16-byte aligned */
    float *k_scale;       /* [pages][heads] */
    float *v_scale;       /* [pages][heads] */
    int64_t pages;        /* 1 .. 2^31 - 1 */
    int32_t heads;        /* K/V heads, 1 .. 1024 */
    int32_t dim;          /* width of a head: a multiple of 16, 16 .. KV8_MAX_DIM */
    int32_t page_tokens;  /* a power of two, 16 .. KV8_MAX_PAGE */
} kv8_cache;

typedef struct kv8_batch {
    const int32_t *table;   /* [seqs][table_stride]: page of each block of tokens */
    int64_t table_stride;   /* elements between rows of the table, >= blocks */
    int64_t blocks;         /* entries of a row; tokens from blocks*P on are holes */
    const int32_t *lens;    /* [seqs] tokens in the cache (a negative one counts as 0) */
    const int32_t *starts;  /* NULL, or [seqs + 1]: first row of each sequence, rising */
    int64_t seqs;           /* 0 .. 2^20 */
    int64_t max_len;        /* 0, or what no length exceeds: it only steers how the
                             * attention is split, results do not rest on it */
} kv8_batch;

/* Quantize the rows' keys and values into the cache.  For each page and head
 * that receives rows (everything F32, each step one rounded operation):
 *   need = max(max |x|, 1e-5) / 127 over the page's new values;
 *   s = need if the page holds no earlier token of the sequence, else
 *       max(s_old, need) (need alone if s_old is a NaN);
 *   where s > s_old, the earlier tokens' codes become
 *       round_half_away(q * (s_old / s));
 *   new codes are round_half_away(x / s) clamped to +-127.
 * Codes behind the sequence's length keep their bytes.
 *   k, v     [rows][heads][dim] of `type`, finite, 16-byte aligned, heads
 *            dense; k_stride, v_stride: elements from row to row, multiples of
 *            16 bytes, >= heads * dim.
 * A page that receives rows stands once in the batch's table: in one sequence,
 * for one block (its contents are undefined otherwise).
 * Errors: I2S_EINVAL (a null or misaligned pointer, an unknown type, a
 * negative size, a stride, starts NULL with rows not a multiple of seqs),
 * I2S_EALIGN (dim, page_tokens), I2S_ERANGE, I2S_EHIP. */
int kv8_append(const kv8_cache *cache, const kv8_batch *batch, int type,
               const void *k, int64_t k_stride, const void *v, int64_t v_stride,
               int64_t rows, void *stream);

/* The inverse: row starts[b] + i of k and v receives token lens[b] - n_b + i
 * as code * scale (one F32 multiply, rounded to `type`).  Layout, strides and
 * errors as kv8_append. */
int kv8_read(const kv8_cache *cache, const kv8_batch *batch, int type,
             void *k, int64_t k_stride, void *v, int64_t v_stride,
             int64_t rows, void *stream);

/* Bytes of the workspace kv8_attention needs for this call (0: none): partial
 * results of sequences that are split over several workgroups.  It depends on
 * sizes alone, never on device contents.  0 for arguments that kv8_attention
 * refuses. */
size_t kv8_attention_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch,
                                     int64_t q_heads, int64_t rows);

/* Attention of each row's q_heads queries over its sequence's cached tokens;
 * query head h reads K/V head h / (q_heads / heads).  For a row at position p
 * and a sequence of length L a token t (in no hole) is seen if
 *   t < L, t <= p where causal, and t > p - window where window > 0;
 *   e_t = scale * sum_d q[d] * (k_scale * K_t[d])
 *   out = sum_t exp(e_t) * (v_scale * V_t) / sum_t exp(e_t)
 *   lse = log sum_t exp(e_t).
 * Exponents e_t are F32: they resolve to their last bit, and have to stay in
 * its range.  Queries are held in 22 bits of each component or more, or in 30 of
 * the row's largest magnitude.  Sums are F32; weights exp(e_t) are multiplied by V
 * in 22 bits, of many BF16 rows in 11.
 * Value scales below 1e-20 count as 0 (their tokens still do in the sum).
 * A row that sees no token gives zeros and lse = -inf.  A query with a NaN or
 * an infinity gives NaN in its own output row and nowhere else.
 *   q        [rows][q_heads][dim] of `type`, 16-byte aligned, heads dense;
 *            q_stride elements from row to row, a multiple of 16 bytes.
 *   out      the same layout with out_stride; may not overlap q.
 *   lse      NULL, or F32 [rows][q_heads].
 *   workspace  >= kv8_attention_workspace_bytes(...), 256-byte aligned,
 *            overwritten; not shared by overlapping calls (two graphs that
 *            may run at once need one each).  NULL where none is needed.
 * q_heads is a multiple of cache->heads, scale finite, window >= 0.
 * Errors as kv8_append, and I2S_EWORKSPACE. */
int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, int type,
                  const void *q, int64_t q_stride, int64_t q_heads, int64_t rows,
                  float scale, int causal, int64_t window,
                  void *out, int64_t out_stride, float *lse,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Queries and keys of each row: RMS-normed per head where a weight is given,
 *   y = x / sqrt(mean(x^2) + eps) * weight,
 * then rotated in their first 2 * pairs components by the row's position:
 *   a = pos * inv_freq[i];  (u, v) -> (u cos a - v sin a, v cos a + u sin a)
 * for pair i = components (i, i + pairs), or (2i, 2i + 1) where `neighbours`.
 * The angle is formed and reduced in 64 bits; statistics and rotation are F32.
 *   q, k     [rows][q_heads][dim] and [rows][k_heads][dim] of `type`, 16-byte
 *            aligned, heads dense, strides (elements from row to row) multiples
 *            of 16 bytes; q_heads or k_heads may be 0 (its pointers then NULL).
 *   q_out, k_out  the same layout with strides of their own; each may be its
 *            input itself (same pointer and stride), else no overlap.
 *   pos      int32 [rows].   inv_freq F32 [pairs] (NULL where pairs is 0).
 *   q_weight, k_weight  NULL (no norm), or F32 [dim].
 * dim a multiple of 16 up to KV8_MAX_DIM, pairs a multiple of 8 with
 * 2 * pairs <= dim.  Errors: I2S_EINVAL, I2S_EALIGN (dim, pairs), I2S_ERANGE,
 * I2S_EHIP. */
int kv8_qk_norm_rope(int type, int64_t rows, int64_t dim,
                     const void *q, int64_t q_stride, int64_t q_heads,
                     const void *k, int64_t k_stride, int64_t k_heads,
                     const int32_t *pos, const float *inv_freq, int64_t pairs, int neighbours,
                     const float *q_weight, const float *k_weight, float eps,
                     void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KV8_H */
