/* Scores, weights and eviction over the int8 K/V cache of kv8.h on MI355X
 * (gfx950): attention whose scores have a shape, how much weight each cached
 * token gets, and a smaller cache of the tokens that matter.
 *
 *   kv8_attention_scored   kv8_attention with capped scores, a bias by
 *                          distance, a prefix that all rows see
 *   kv8_weigh              the weight that a call's rows give each token,
 *                          added to the token's mass
 *   kv8_choose             the tokens of each sequence and head that stay
 *   kv8_move               chosen tokens, gathered into fresh pages
 *
 * Caches, batches, types, layouts and conventions are those of kv8.h.
 *
 * Scores.  For a row at position p (of sequence b, of length L) and a token t
 * in no hole, with query head h:
 *   e_t = scale * sum_d q[d] * (k_scale * K_t[d])
 *   e_t = cap * tanh(e_t / cap)            where cap > 0
 *   e_t = e_t - slopes[h] * |p - t|        where slopes are given
 * and t is seen if t < L, and t <= p or t < prefix[b] where causal (prefix
 * NULL: 0), and t > p - window where window > 0.
 *   scale    within +-2^126.
 *   window   >= 0.
 *   cap      0 (none), or 2^-60 .. 2^60.
 *   slopes   NULL, or F32 [q_heads], finite.
 *   prefix   NULL, or int32 [seqs] (a negative one counts as 0).
 * Exponents e_t and the lse are F32: they resolve to their last bit, and have to
 * stay within +-2^127 (before the cap, where there is one, they need not).
 * Queries are held as kv8_attention's, in kv8_weigh F32 ones in 22 bits of each
 * component.  Sums are F32; the attention multiplies weights by V in 22 bits, for
 * rows of any type.
 * Positions are places in the cache.  After kv8_move they are the places that
 * the chosen tokens then have: windows, distances and prefixes go by those,
 * and rotated keys keep the angles of the positions that they were written at.
 *
 * The mass of a token and K/V head is F32 mass[page][head][slot], a companion
 * of the cache's pages: [pages][heads][page_tokens], 4-byte aligned.
 */
#ifndef KV8_SCORES_H
#define KV8_SCORES_H

#include <stddef.h>
#include <stdint.h>

#include "kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kv8_attention with shaped scores.  The workspace is
 * kv8_attention_workspace_bytes(...); everything else and the errors are as
 * kv8_attention's (I2S_EINVAL for a scale or cap out of its range, misaligned slopes
 * or prefix).  A row in front of position 0 sees, where causal, its prefix
 * alone. */
int kv8_attention_scored(const kv8_cache *cache, const kv8_batch *batch, int type,
                         const void *q, int64_t q_stride, int64_t q_heads, int64_t rows,
                         float scale, int causal, int64_t window,
                         float cap, const float *slopes, const int32_t *prefix,
                         void *out, int64_t out_stride, float *lse,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the workspace kv8_weigh needs for this call (0: none): sums of rows
 * that several workgroups share.  It depends on sizes alone.  0 for arguments
 * that kv8_weigh refuses. */
size_t kv8_weigh_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch,
                                 int64_t q_heads, int64_t rows);

/* The weight that the batch's rows give each cached token, for each K/V head
 * (laid out by the sequences' mean number of rows: a prompt's chunk among decode
 * steps is better a call of its own):
 *   w_t = sum over rows i and the head's query heads h, of those that see t,
 *         of exp(e_t - lse[i][h])
 *   mass_t = w_t for the call's own tokens (those at positions L - n_b and on),
 *            mass_t + w_t for earlier ones,
 * Where every token that is appended is a row of one such call, masses need no
 * clearing when a page is begun.  Where some are not (only a prompt's last rows
 * are weighed, or not every step's), theirs are added to from the first call on:
 * the caller sets their masses to 0 before it (a whole page's when it is begun,
 * by an append or a move), else what the page held before counts as theirs.
 *   q, q_stride, q_heads, rows   the queries, as kv8_attention's.
 *   lse      F32 [rows][q_heads], as the attention with the same scores wrote
 *            it.  A row and head whose lse is not finite (it saw nothing, its
 *            query holds a NaN) adds nothing.
 *   mass     the masses; tokens in holes and slots behind a sequence's length
 *            are left as they were.
 *   workspace  >= kv8_weigh_workspace_bytes(...), 256-byte aligned,
 *            overwritten, not shared by overlapping calls.  NULL where none is
 *            needed.
 * Tokens in a page that several of the batch's sequences read (a shared
 * prompt) get the weights of all, added atomically: in an order, and so with a
 * last bit, that may differ from call to call.  Without shared pages results
 * are the same every time.  A page that receives the call's own tokens stands
 * once in the batch's table, as for kv8_append.
 * Errors as kv8_attention. */
int kv8_weigh(const kv8_cache *cache, const kv8_batch *batch, int type,
              const void *q, int64_t q_stride, int64_t q_heads, int64_t rows,
              float scale, int causal, int64_t window,
              float cap, const float *slopes, const int32_t *prefix,
              const float *lse, float *mass,
              void *workspace, size_t workspace_bytes, void *stream);

/* The tokens of each sequence and K/V head that stay: of its tokens in no
 * hole all, if they are at most `keep`, else `keep` of them: the first `first`
 * tokens of the sequence (t < first), the newest `recent` (t >= L - recent),
 * then those of the largest mass, of equal masses those of the lowest index
 * (0 and -0 are equal; a NaN is less than any number).
 *   mass     the masses of the cache's pages.
 *   keep     0 .. 2^31 - 1025;  first, recent >= 0, first + recent <= keep.
 *   index    int32 [seqs][heads][keep]: the tokens, rising, then -1.
 *   kept     int32 [seqs]: how many stay (of every head as many).
 * The batch's starts are not looked at.
 * Errors: I2S_EINVAL (a null or misaligned pointer, a negative size, first and
 * recent over keep), I2S_EALIGN (dim, page_tokens), I2S_ERANGE, I2S_EHIP. */
int kv8_choose(const kv8_cache *cache, const kv8_batch *batch, const float *mass,
               int64_t keep, int64_t first, int64_t recent,
               int32_t *index, int32_t *kept, void *stream);

/* Chosen tokens into fresh pages of the cache: for each sequence and head
 * token index[b][head][i], i < kept[b], becomes token i of the sequence that
 * to_table names, as if kv8_read had given its values (code * scale, F32) and
 * kv8_append had written them to pages begun now: for each page and head
 *   s = max(max |x|, 1e-5) / 127,  code = round_half_away(x / s).
 * Codes behind the last token keep their bytes.
 *   index    int32 [seqs][heads][keep].  One outside 0 .. L - 1, or in a hole,
 *            gives a token of zeros (and of mass 0).
 *   kept     int32 [seqs], counted as 0 .. keep.
 *   to_table int32 [seqs][to_stride], to_stride >= to_blocks: the pages.  An
 *            entry outside 0 .. pages - 1, and blocks from to_blocks on, drop
 *            their tokens.
 *   mass     NULL, or the masses, of which the tokens' go along.
 * A page that receives tokens stands once in to_table, and holds none of the
 * tokens that the batch's table and index name (its contents are undefined
 * otherwise).  kept and to_table are the lens and the table of the batch that
 * follows, with to_blocks >= the blocks that it needs for its new tokens, too.
 * Errors as kv8_choose. */
int kv8_move(const kv8_cache *cache, const kv8_batch *batch,
             const int32_t *index, const int32_t *kept, int64_t keep,
             const int32_t *to_table, int64_t to_stride, int64_t to_blocks,
             float *mass, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KV8_SCORES_H */
