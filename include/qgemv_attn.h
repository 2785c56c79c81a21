/*
 * qgemv_attn.h -- C ABI of libqgemv.so, second part: attention and the paged
 * key/value cache, the work between the linear layers of qgemv.h in a decoder
 * layer.
 *
 * Conventions of qgemv.h hold: [dev] pointers, the caller owns every buffer,
 * calls enqueue kernels on `stream` and return at once (no allocation, no
 * synchronization, no memset or copy nodes, so they can be captured in a HIP
 * graph), arguments are checked before anything is enqueued, and a failing
 * call enqueues nothing.  Data on the device (row offsets, page numbers,
 * positions, masks) is not validated on the host; the kernels check every
 * index they take from it, so malformed values give wrong results or a status
 * bit, never an access outside the caller's buffers.
 *
 * Element types: QGEMV_F16 or QGEMV_BF16 for queries, keys, values and
 * outputs alike, passed as uint16_t bits.  Scores, softmax statistics and
 * output sums are kept in fp32; the softmax weights are rounded to the element
 * type for the matrix-core product with the values (their sum is not), and
 * the output is rounded to nearest even once.  Results are deterministic.
 *
 * Heads: `heads` query heads, `heads_kv` key/value heads, heads a multiple of
 * heads_kv; query head h reads key head h / (heads / heads_kv).  head_dim is
 * 64 or 128 (QGEMV_ERR_UNSUPPORTED otherwise).
 *
 * Rows ("sequences"): offsets cu[0 .. rows] int32 [dev], cu[0] = 0, ascending;
 * row b holds tokens cu[b] .. cu[b + 1] - 1 (none where they are equal).
 *
 * What a masked or missing key holds (also infinities and NaN) does not reach
 * the output, and a query that sees no key has output 0.  A seen key whose
 * score is -inf has no weight (where scale is not 0), and a query all of whose
 * scores are -inf has output 0 too.  A seen key's infinite value makes its column
 * infinite, or NaN where its weight is too small for the element type.
 */
#ifndef QGEMV_ATTN_H
#define QGEMV_ATTN_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { QGEMV_F16 = 0, QGEMV_BF16 = 1 } qgemv_dtype;

/* A [tokens, heads, head_dim] array whose last dimension is contiguous:
 * element (t, h, d) is data[t * token + h * head + d].  data is 16-byte
 * aligned and the strides, in elements, are multiples of 8 (QGEMV_ERR_ALIGN),
 * and not negative (QGEMV_ERR_SHAPE); the stride of a dimension of one is not
 * looked at.  So the parts of a fused QKV product are read in place. */
typedef struct {
  uint16_t *data;
  int64_t token, head;
} qgemv_heads;

/* ------------------------------------------------------------------------
 * Attention over packed prompts:
 *     o[i] = sum_j exp(s[i,j] - m[i]) v[j] / sum_j exp(s[i,j] - m[i]),
 *     s[i,j] = scale * (q[i] . k[j]),   j over the keys that query i sees.
 * Sequence b has queries cu_q[b] .. cu_q[b+1]-1 and keys cu_k[b] ..
 * cu_k[b+1]-1.  With `causal`, query i (from 0 in its sequence) sees key j
 * where j <= i + nk - nq: the queries are the last nq of the nk tokens, so a
 * prompt that continues earlier keys needs no mask, and queries in front of
 * the first key (nq > nk) see none.
 *
 *   scale              finite and not negative (VALUE otherwise)
 *   tokens, tokens_k   rows of q and o, rows of k and v (cu_q[batch] and
 *                      cu_k[batch]; offsets past them are clamped)
 *   ws [dev]           scratch of at least qgemv_attn_prompt_workspace_bytes
 *                      bytes, 16-byte aligned, no initial contents; calls that
 *                      share it must not overlap in time.  May be NULL when
 *                      that is 0.
 *
 * Checks, in order: null, dtype / head_dim (UNSUPPORTED), shape (counts not
 * negative, heads % heads_kv, tokens * heads < 2^31 and about
 * tokens * heads / 128 + batch * heads_kv < 2^21, tokens_k at most 2^31 - 1024,
 * tokens * heads * tokens_k under about 2^61 and, times batch, 2^73,
 * strides, k's and v's token strides < 2^26), scale, alignment,
 * o overlapping an input (VALUE), workspace.  o's elements must not overlap
 * each other (SHAPE).  tokens or batch of 0 does nothing.
 * ------------------------------------------------------------------------ */
size_t qgemv_attn_prompt_workspace_bytes(int tokens, int tokens_k, int batch, int heads, int heads_kv, int head_dim);
int qgemv_attn_prompt(int dtype, int causal, int tokens, int tokens_k, int batch, int heads, int heads_kv,
                      int head_dim, float scale, const qgemv_heads *q, const qgemv_heads *k, const qgemv_heads *v,
                      const int32_t *cu_q, const int32_t *cu_k, const qgemv_heads *o, void *ws, size_t ws_bytes,
                      qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * The paged cache.  Keys and values of all layers live in two pools
 *     k, v [dev] [layers][pages][page_size][heads_kv][head_dim]   (16-byte aligned)
 * and position p of row b in page tables[b][p / page_size] of every layer.
 *     tables [dev] int32 [rows][max_pages], -1 where there is no page
 *     lens   [dev] int32 [rows]  tokens of each row
 *     refs   [dev] int32 [pages] rows that hold the page; 0 = free
 *     status [dev] int32 [1]     QGEMV_KV_* bits that calls OR into it; the
 *                                caller clears and reads it when it likes
 * page_size is 16, 32, 64, 128 or 256 (UNSUPPORTED otherwise), and a row holds
 * at most max_pages * page_size <= 2^31 - 1024 tokens (SHAPE).  A new cache
 * has tables -1 and lens, refs and status 0.  Pages are taken lowest number
 * first and counted on the device, so a decode loop needs no host in between.
 * Invariant kept by the calls below: a row's last page is shared with another
 * row only if it is full.
 * ------------------------------------------------------------------------ */
typedef struct {
  int layers, pages, page_size, heads_kv, head_dim, rows, max_pages;
  uint16_t *k, *v;
  int32_t *tables, *lens, *refs, *status;
} qgemv_kv_cache;

#define QGEMV_KV_NO_PAGES 1   /* the pool has too few free pages                    */
#define QGEMV_KV_TABLE_FULL 2 /* a row would need more than max_pages pages         */
#define QGEMV_KV_BAD_INDEX 4  /* a parent, kept node or count outside its range     */
#define QGEMV_KV_SHARED 8     /* kv_compact would write to a page another row holds */

/* Every call: QGEMV_ERR_VALUE where something that it writes (its results, the
 * workspace, the state above) overlaps something else that it writes or reads;
 * kv_compact's pos, keep and count may lie in lens.  (qgemv_kv_write, _fork and
 * _compact do not look whether k and v lie over each other.) */

/* Scratch of kv_reserve, kv_fork and kv_compact: [dev], 16-byte aligned, no
 * initial contents.  rows: the larger of the caches' rows. */
size_t qgemv_kv_workspace_bytes(int rows, int pages);

/* Grows row b by cu[b + 1] - cu[b] tokens and takes the pages that it lacks:
 * pos[b] = lens[b], then lens[b] grows.  Pages go to the rows in order; a row
 * that does not get all it needs (NO_PAGES), would outgrow its table
 * (TABLE_FULL) or has a negative count (BAD_INDEX) stays as it was with
 * pos[b] = -1.  Once per step, for all layers. */
int qgemv_kv_reserve(const qgemv_kv_cache *c, const int32_t *cu, int32_t *pos, void *ws, size_t ws_bytes,
                     qgemv_stream_t stream);

/* Writes one layer's new keys and values: token cu[b] + i of k and v goes to
 * position pos[b] + i of row b (pos from kv_reserve; rows at -1 are skipped,
 * and tokens at a position without a page are too).  Up to 2^26 - 4 tokens
 * (SHAPE otherwise). */
int qgemv_kv_write(const qgemv_kv_cache *c, int layer, int tokens, const qgemv_heads *k, const qgemv_heads *v,
                   const int32_t *cu, const int32_t *pos, qgemv_stream_t stream);

/* Row i of `out` becomes a fork of row parents[i] of `c` (-1: empty), for
 * i < out->rows.  `out` has tables and lens of its own and c's pools, refs and
 * status; c's tables and lens are stale afterwards.  Full pages are shared
 * (refs counts them); a partly filled last page stays with its first child,
 * and each later child gets a fresh page with a copy of its tokens, in every
 * layer.  A row without a child gives its pages back before fresh ones are
 * taken.  A child that finds no fresh page keeps its full pages only
 * (NO_PAGES); a parent outside the rows counts as -1 (BAD_INDEX). */
int qgemv_kv_fork(const qgemv_kv_cache *c, const int32_t *parents, const qgemv_kv_cache *out, void *ws,
                  size_t ws_bytes, qgemv_stream_t stream);

/* Keeps count[b] of the tokens from position pos[b] on: those at pos[b] +
 * keep[b][0 .. count[b]-1] (strictly ascending, keep is [rows][max_keep]) move
 * to pos[b], pos[b] + 1, ..., in every layer; lens[b] = pos[b] + count[b], and
 * pages past the end are given back.  pos[b] = count[b] = 0 empties the row;
 * pos[b] = -1 leaves it alone, and so does a row whose keep, count or pos lies
 * outside it (BAD_INDEX) or that would write to, or end inside, a page that
 * another row holds too (SHARED). */
int qgemv_kv_compact(const qgemv_kv_cache *c, const int32_t *pos, const int32_t *keep, int max_keep,
                     const int32_t *count, void *ws, size_t ws_bytes, qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention of new tokens over the cache (one layer): row b's tokens cu[b] ..
 * cu[b+1]-1 are at positions pos[b], pos[b]+1, ... of the cache (kv_reserve,
 * kv_write) and each sees every position before pos[b], and of the new tokens
 * those that its mask names:
 *
 *   mask [dev] uint64 [tokens][mask_words], bit j of token i: it sees token j
 *              of its row (a drafted tree: its ancestors and itself); tokens
 *              past 64 * mask_words are not seen.  NULL: each sees the new
 *              tokens up to itself (mask_words 0), so one token per row is
 *              plain decode.
 *
 * A row with pos[b] < 0 has output 0.  Every position that a row sees must
 * have a page (kv_reserve sees to that; a missing one reads some other page of
 * the pool).  scale, tokens, o, ws and the checks as in qgemv_attn_prompt, with
 * max_pages * page_size for tokens_k.
 * ------------------------------------------------------------------------ */
size_t qgemv_attn_tree_workspace_bytes(int tokens, int rows, int heads, int heads_kv, int head_dim);
int qgemv_attn_tree(int dtype, const qgemv_kv_cache *c, int layer, int tokens, int heads, float scale,
                    const qgemv_heads *q, const int32_t *cu, const int32_t *pos, const uint64_t *mask,
                    int mask_words, const qgemv_heads *o, void *ws, size_t ws_bytes, qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * Writing new keys and values with their position rotation, which turns the
 * queries too: pair i < rot / 2 of a head turns by the angle
 * t = position * freqs[i],
 *     (a, b) -> (a cos t - b sin t, a sin t + b cos t),
 * in fp32 (t's whole turns are taken off in 64 bits), rounded once; elements
 * from rot on stay as they are, and so do values.
 *   dtype       of q, k, v and o: QGEMV_F16 or QGEMV_BF16 (of a cache of 16
 *               bits: its own)
 *   heads       query heads, any number; 0: no queries (q and o may be NULL)
 *   rot         elements of a head that turn: a multiple of 16 up to head_dim
 *               (UNSUPPORTED otherwise), 0: none (freqs may be NULL)
 *   freqs [dev] fp32 [rot / 2], 16-byte aligned: radians a position
 *   interleaved pair i is elements 2 i and 2 i + 1; else i and i + rot / 2
 *   at [dev]    int32 [tokens]: positions for the angles, or NULL: those in the
 *               row (a drafted tree's nodes turn by their depth, say)
 *   o           takes the rotated queries; it may be q itself (the same data
 *               and strides)
 * Token cu[b] + i goes to position pos[b] + i of row b (pos from
 * qgemv_kv_reserve).  Tokens of rows at -1 and tokens of no row are skipped, in
 * o too; keys and values at a position without a page are.  tokens * (heads +
 * 2 * heads_kv + 8) + 32 * rows * heads_kv is below 2^29 - 64 (SHAPE otherwise).
 * Checks, in order: null, dtype, cache, rot, shape, alignment, overlap.
 * ------------------------------------------------------------------------ */
int qgemv_kv_append(int dtype, const qgemv_kv_cache *c, int layer, int tokens, int heads, const qgemv_heads *q,
                    const qgemv_heads *k, const qgemv_heads *v, const int32_t *cu, const int32_t *pos,
                    const float *freqs, int rot, int interleaved, const int32_t *at, const qgemv_heads *o,
                    qgemv_stream_t stream);

/* Copies tokens of the cache into packed arrays: token cu[b] + i of k and v
 * becomes position start[b] + i of row b (rows at -1, tokens of no row and
 * positions without a page are skipped: k and v stay as they were there).  Up to
 * 2^26 - 4 tokens (SHAPE otherwise). */
int qgemv_kv_read(const qgemv_kv_cache *c, int layer, int tokens, const int32_t *cu, const int32_t *start,
                  const qgemv_heads *k, const qgemv_heads *v, qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * The paged cache in 8 bits: pools of e4m3 codes (bias 7, no infinities, 0x7F
 * and 0xFF are NaN), and an exponent for every block of 16 tokens and head,
 *     k, v           [dev] uint8 [layers][pages][page_size][heads_kv][head_dim]
 *     k_exps, v_exps [dev] uint8 [layers][pages][page_size / 16][heads_kv]
 *     value = code * 2^(exponent - 127)
 * (exponents 1 to 254; 0 and 255 count as those).  The rest is as in
 * qgemv_kv_cache, and so are the calls, but for what follows; qgemv_kv_write's
 * place is taken by qgemv_kv8_append (with rot 0).
 *
 * Writing a token: keys after their rotation and values, in fp32, are rounded to
 * nearest even under the block's exponent e, the least with
 * max |x| <= 448 * 2^(e - 127) over the block's new tokens and heads' elements,
 * at least 63, and at least what the block has where it holds earlier tokens of
 * the row.  If it grows, the codes of the earlier tokens are written anew under
 * it, rounded to nearest even (exact but for codes that become subnormal).
 * Infinities and NaN become NaN and do not count in the maximum.
 *
 * kv8_compact: a block that gains tokens has the largest exponent of the blocks
 * that its tokens come from, and codes of others are rewritten under it
 * likewise.
 * ------------------------------------------------------------------------ */
typedef struct {
  int layers, pages, page_size, heads_kv, head_dim, rows, max_pages;
  uint8_t *k, *v, *k_exps, *v_exps;
  int32_t *tables, *lens, *refs, *status;
} qgemv_kv8_cache;

int qgemv_kv8_reserve(const qgemv_kv8_cache *c, const int32_t *cu, int32_t *pos, void *ws, size_t ws_bytes,
                      qgemv_stream_t stream);
int qgemv_kv8_append(int dtype, const qgemv_kv8_cache *c, int layer, int tokens, int heads, const qgemv_heads *q,
                     const qgemv_heads *k, const qgemv_heads *v, const int32_t *cu, const int32_t *pos,
                     const float *freqs, int rot, int interleaved, const int32_t *at, const qgemv_heads *o,
                     qgemv_stream_t stream);
/* Values in either type: exact where it holds them, from 2^-21 to 65504 in fp16
 * and from 2^-130 to 2^128 in bf16; smaller ones are rounded to nearest even,
 * larger ones infinite.  (Appending may round past that: tokens of 63488 and more
 * in fp16, or 1.9375 * 2^127 in bf16, come back infinite.) */
int qgemv_kv8_read(int dtype, const qgemv_kv8_cache *c, int layer, int tokens, const int32_t *cu, const int32_t *start,
                   const qgemv_heads *k, const qgemv_heads *v, qgemv_stream_t stream);
int qgemv_kv8_fork(const qgemv_kv8_cache *c, const int32_t *parents, const qgemv_kv8_cache *out, void *ws,
                   size_t ws_bytes, qgemv_stream_t stream);
int qgemv_kv8_compact(const qgemv_kv8_cache *c, const int32_t *pos, const int32_t *keep, int max_keep,
                      const int32_t *count, void *ws, size_t ws_bytes, qgemv_stream_t stream);

/* qgemv_attn_tree over a cache of 8 bits: keys and values are its values in the
 * queries' type, exact or rounded as qgemv_kv8_read gives them. */
int qgemv_attn_tree8(int dtype, const qgemv_kv8_cache *c, int layer, int tokens, int heads, float scale,
                     const qgemv_heads *q, const int32_t *cu, const int32_t *pos, const uint64_t *mask,
                     int mask_words, const qgemv_heads *o, void *ws, size_t ws_bytes, qgemv_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QGEMV_ATTN_H */
