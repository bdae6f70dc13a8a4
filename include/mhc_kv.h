/*
 * mhc_kv.h -- C ABI of the paged 8-bit key/value cache of libmhc.so: the
 * attention sublayer's cache that a decoder keeps next to the mHC seam
 * (mhc.h).  Between mhc_pre_delayed, which forms the sublayer's input, and
 * mhc_post, which takes its output, an attention sublayer projects queries,
 * keys and values; mhc_kv_append rotates them (mhc_kv_append_norm norms them
 * first) and stores keys and values, and mhc_kv_attend is the causal attention
 * of the new tokens over the cache (mhc_kv_attend_window with a sliding
 * window).  mhc_kv_fork and mhc_kv_compact say which pages are whose.
 *
 * The conventions of mhc.h hold: caller-owned device pointers of the current
 * device, bf16 as uint16_t, asynchronous calls on the given stream, host-side
 * checks before any launch, no allocation and no synchronisation inside a
 * call; every call can be captured in a CUDA graph.  What only the device
 * knows (lengths, page numbers) is checked there: see "Bad indices" below.
 */
#ifndef MHC_KV_H
#define MHC_KV_H

#include "mhc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One layer's cache.  k and v hold e4m3 numbers (4 exponent bits, bias 7, 3
 * mantissa bits, no infinity, NaN = 0x7f / 0xff), dense
 * [num_pages][heads][page_tokens][head_dim]; a stored number stands for
 * code * scale[page][head].  k and v are 16-byte aligned, the scales 4-byte.
 * Scales are finite and not negative; those of pages that mhc_kv_append goes on
 * with are powers of two, as it writes them (mhc_kv_attend takes any).
 * page_tokens is 16, 32, 64 or 128; head_dim 64 or 128; num_pages * heads
 * at most 2^31 - 1.
 */
typedef struct mhc_kv_cache {
    uint8_t *k, *v;
    float *k_scale, *v_scale; /* [num_pages][heads] */
    int64_t num_pages;
    int heads; /* key/value heads */
    int page_tokens;
    int head_dim;
} mhc_kv_cache;

/*
 * Which token is where.  Sequence b keeps its token at position i in page
 * block_table[b * table_width + i / page_tokens], slot i % page_tokens.  The
 * T new tokens of a call lie one sequence after the other: sequence b's are
 * rows cu_q[b] .. cu_q[b+1]-1 (cu_q has B + 1 ascending entries from 0 to T);
 * cu_q NULL means one new token for each sequence (T == B).  seq_lens[b]
 * counts b's tokens WITH its new ones, which take its last positions.  A
 * sequence may be empty (length 0) and may have no new tokens; a new token
 * whose position would be negative (an unused place of a padded batch) has no
 * place in the cache and sees no key.
 *
 * Bad indices.  A page number outside [0, num_pages), a length above
 * table_width * page_tokens or below zero, cu_q entries out of order or
 * range, and a position without a row in the rotation's tables touch no
 * memory, and mhc_device_status returns MHC_ERR_INDEX once.
 *   mhc_kv_append does not write the tokens concerned: those of the page or of
 *     the positions; with a bad length or offset all of the sequence's new
 *     tokens, which then have no place.
 *   mhc_kv_attend does not attend to the keys of a bad page, and takes a bad
 *     length as the nearest one that the table can hold; with a bad offset it
 *     does not write the rows of the sequence's tokens.
 */

/*
 * mhc_kv_append -- for each new token t at position p of sequence b:
 *   q_out[t][h]  = bf16( R_p q[t][h] )                        (when q is given)
 *   cache.k      <- R_p k[t][h],   cache.v <- v[t][h]
 * R_p rotates the first rotary_dim elements of a head in pairs (x, y):
 *   x' = x cos - y sin,  y' = y cos + x sin,  cos/sin[p][i], i = the pair,
 * each product and sum rounded to fp32; pair i is elements (i, i +
 * rotary_dim/2), or (2i, 2i + 1) when interleaved.
 *
 * Scales.  Page scales are powers of two, so that a scale can grow without a
 * second rounding of numbers in e4m3's normal range.  With a = the largest
 * finite magnitude among the page's new numbers (one head, k and v apart):
 *   need  = 2^e, the smallest with a <= 448 * 2^e, e >= -116
 *   scale = need when the call begins the page (writes its slot 0),
 *           else max(scale, need); when it grows, the page's earlier slots
 *           are rounded once more: code = e4m3(code * old / new)
 *   code  = e4m3(x / scale), to nearest, ties to even
 * Infinities and NaN are stored as NaN.  Slots after the new tokens keep
 * their bytes.
 *
 *  k, v       bf16, token t's head h at t * stride + h * head_dim (stride in
 *             elements): rows of a fused projection can be passed as they are
 *  q, q_out   bf16, q_heads heads, likewise; both NULL (q_heads ignored): no
 *             queries.  q_out may be exactly q; otherwise it must not overlap
 *             an input.  Rows without a place in the cache are copied
 *             unrotated.
 *  cos, sin   fp32 [rope_rows][rotary_dim / 2]; both NULL or rotary_dim 0: no
 *             rotation.  rotary_dim is a multiple of 16, at most head_dim.
 *  strides    multiples of 8 elements; every pointer 16-byte aligned but
 *             block_table, seq_lens and cu_q (4-byte)
 * No two of the call's tokens may share a page and slot, and no two sequences
 * may append to one page in one call.  One kernel launch.  T == 0 launches
 * nothing.  Errors: MHC_ERR_INVALID_ARGUMENT, MHC_ERR_UNSUPPORTED (head_dim,
 * page_tokens, rotary_dim), MHC_ERR_CUDA.
 */
mhc_status mhc_kv_append(const mhc_kv_cache *cache, const uint16_t *k, int64_t k_stride,
                         const uint16_t *v, int64_t v_stride, const uint16_t *q, int64_t q_stride,
                         int q_heads, uint16_t *q_out, int64_t q_out_stride, const float *cos,
                         const float *sin, int64_t rope_rows, int rotary_dim, int interleaved,
                         const int32_t *block_table, int64_t table_width, const int32_t *seq_lens,
                         const int32_t *cu_q, int64_t B, int64_t T, void *stream);

/*
 * mhc_kv_append_norm -- mhc_kv_append with a norm of each head's query and key
 * before the rotation, as decoders have it that norm queries and keys:
 *   N x = x * r * w[h],  r = 1 / sqrt(sum_i x_i^2 / head_dim + norm_eps)
 *   q_out[t][h] = bf16( R_p N q[t][h] ),   cache.k <- R_p N k[t][h]
 * held in fp32 from the inputs to the one rounding at the end; values are
 * written as they are.  Rows without a place in the cache, or with a position
 * that the rotation's tables lack, are copied as they are.  A head that holds
 * an infinity or NaN gives what the formula gives.
 *
 *  q_norm, k_norm  bf16 weights, head h's at h * stride (in elements: a
 *                  multiple of 8, at least head_dim; 0: all heads have the
 *                  same), 16-byte aligned.  NULL: no norm of these; q_norm
 *                  without q is refused where there are tokens.
 *  norm_eps        1e-20 or more, finite; read when there is a norm
 */
mhc_status mhc_kv_append_norm(const mhc_kv_cache *cache, const uint16_t *k, int64_t k_stride,
                              const uint16_t *v, int64_t v_stride, const uint16_t *q, int64_t q_stride,
                              int q_heads, uint16_t *q_out, int64_t q_out_stride,
                              const uint16_t *q_norm, int64_t q_norm_stride, const uint16_t *k_norm,
                              int64_t k_norm_stride, float norm_eps, const float *cos,
                              const float *sin, int64_t rope_rows, int rotary_dim, int interleaved,
                              const int32_t *block_table, int64_t table_width,
                              const int32_t *seq_lens, const int32_t *cu_q, int64_t B, int64_t T,
                              void *stream);

/*
 * mhc_kv_attend -- for each new token t at position p and query head h, with
 * the key/value head h / (q_heads / heads):
 *   s_j    = softmax_scale * q[t][h] . k_j,   j = 0 .. p
 *   lse    = log(sum_j exp(s_j))
 *   out    = bf16( sum_j exp(s_j - lse) v_j )
 * A token that sees no key gets out = 0 and lse = -infinity.  A key after p
 * never reaches the output, whatever its bytes stand for.  A query that holds
 * an infinity or NaN gives NaN in out and lse if it sees a key.
 *
 * Accuracy.  With p_j = exp(s_j - lse), out is off by its own rounding, 2^-10
 * of sum_j p_j |v_j| (as the weights are f16 numbers), and for each key 2^-26 of
 * the largest value scale among the sequence's keys up to p, whatever that key
 * weighs (f16's range); a logit by 2^-20 of sum_i |q_i k_i| softmax_scale.
 *
 *  q          bf16 as in mhc_kv_append (already rotated)
 *  q_heads    a multiple of cache->heads, at most 128 times as many
 *  out        bf16 [T][q_heads][head_dim] dense; must not overlap q or the cache
 *  lse        fp32 [T][q_heads] or NULL
 *  workspace  device scratch of mhc_kv_attend_workspace_bytes bytes, 256-byte
 *             aligned, as for mhc_pre_delayed (contents on entry do not
 *             matter; calls that can run concurrently need separate ones)
 * Errors as mhc_kv_append; also for a short or misaligned workspace.
 */
mhc_status mhc_kv_attend(const mhc_kv_cache *cache, const uint16_t *q, int64_t q_stride, int q_heads,
                         const int32_t *block_table, int64_t table_width, const int32_t *seq_lens,
                         const int32_t *cu_q, int64_t B, int64_t T, float softmax_scale,
                         uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * mhc_kv_attend_window -- mhc_kv_attend with a sliding window and a few first
 * keys that stay visible: token t at position p sees the keys j <= p with
 *   j > p - window  or  j < sinks
 * A page of which no new token of its sequence sees a key is not looked at:
 * its place in the table may hold any number (-1, say, once the page has been
 * given to somebody else), which is not a bad index.
 *
 * Accuracy as mhc_kv_attend, the value scales being those of the pages of
 * which a token of the sequence sees a key.
 *
 *  window     1 or more
 *  sinks      0 or more
 *  workspace  as for mhc_kv_attend, of as many bytes
 * Errors as mhc_kv_attend.
 */
mhc_status mhc_kv_attend_window(const mhc_kv_cache *cache, const uint16_t *q, int64_t q_stride,
                                int q_heads, const int32_t *block_table, int64_t table_width,
                                const int32_t *seq_lens, const int32_t *cu_q, int64_t B, int64_t T,
                                float softmax_scale, int64_t window, int64_t sinks, uint16_t *out,
                                float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes mhc_kv_attend needs on the current device (0: none). */
size_t mhc_kv_attend_workspace_bytes(const mhc_kv_cache *cache, int q_heads, int64_t B, int64_t T);

/*
 * mhc_kv_fork -- the tables of the next step: place b of its batch goes on with
 * the tokens of place parents[b] of this one, or, with -1, begins without any.
 * Beams that follow their parents, several answers to one prompt, sequences
 * that begin and end, and a plain step (parents NULL: b goes on with b, B ==
 * B_in) are all of this form.  With n = the parent's length and P =
 * page_tokens:
 *   seq_lens_out[b] = n
 *   Full pages, entries i < n / P, are shared: block_table_out[b][i] is the
 *     parent's.  With a window (see mhc_kv_attend_window) only those of which a
 *     token at position n can see a key: (i + 1) P > n - window + 1 or i P <
 *     sinks; the others become -1.
 *   A part-filled page (n % P > 0) is gone on with by the first place that has
 *     it, unless it is held or is also somebody's full page; every other place
 *     gets a copy: a free page whose slots below n % P, and scales, are the
 *     original's, in every cache.  Its other slots keep their bytes.
 *   room[b] further tokens (NULL: room_all for every place) get free pages in
 *     the entries from ceil(n / P) to ceil((n + room) / P).
 *   All other entries become -1.
 * A page is free if block_table_out does not name it by the above and it is not
 * held: what no place goes on with is free at once, and nothing is kept between
 * calls.  Free pages are handed out from the lowest number on, in the order of
 * the places and within a place of the entries.
 *
 * So a decoding loop is: mhc_kv_fork with room 1, lengths + 1, mhc_kv_append,
 * mhc_kv_attend.  Pages for tokens that were not appended are free again in
 * the next call, as they lie beyond the length.
 *
 *  caches     num_caches (1 to 512) caches that share their page numbers, the
 *             layers of a model: num_pages and page_tokens alike; heads and
 *             head_dim may differ.  Their arrays must not overlap.
 *  block_table, seq_lens   [B_in][table_width], [B_in]: of this step
 *  parents    [B], each -1 to B_in - 1, or NULL; with B 0 (a batch that has
 *             ended) nothing is done, and parents may be NULL for any B_in
 *  room       [B], or NULL; not negative.  room_all not negative.
 *  held       [num_pages] bytes, not zero for pages that others go on using
 *             (a prefix cache, say), 4-byte aligned, or NULL
 *  window     1 or more; 0: none, then sinks is 0 as well
 *  block_table_out, seq_lens_out   [B][table_width], [B]; may be exactly
 *             block_table and seq_lens if parents is NULL
 *  workspace  as for mhc_pre_delayed, mhc_kv_fork_workspace_bytes bytes
 * Bad indices are reported as for mhc_kv_append: a length is taken as the
 * nearest one that the table can hold, as is a length with its room; a parent
 * out of range as -1; an entry that is neither a page nor -1 as -1.  -1 is no
 * page and nothing is reported.  Where free pages run out, entries that should
 * have one stay -1, and mhc_device_status returns MHC_ERR_PAGES once (after
 * MHC_ERR_INDEX if there was a bad index as well).
 * Two kernel launches, three and a memset for large tables, and one more for
 * each 64 caches beyond the first.
 * Errors as mhc_kv_append; MHC_ERR_UNSUPPORTED for num_pages above 2^30 or
 * B * (table_width + 1) or B_in * (table_width + 1) above 2^30 - 1.
 */
mhc_status mhc_kv_fork(const mhc_kv_cache *caches, int num_caches, const int32_t *block_table,
                       int64_t table_width, const int32_t *seq_lens, int64_t B_in,
                       const int32_t *parents, int64_t B, const int32_t *room, int64_t room_all,
                       const uint8_t *held, int64_t window, int64_t sinks, int32_t *block_table_out,
                       int32_t *seq_lens_out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * mhc_kv_compact -- moves the pages in use to the lowest numbers, so that the
 * caches can be cut to their first *pages pages.  A page is in use if one of
 * the first ceil(seq_lens[b] / page_tokens) entries of a row names it.  With U
 * pages in use that are not held, these end up as the U lowest numbers that
 * are not held: the k-th used one above them moves to the k-th free one among
 * them, all of its slots and its scales, in every cache.
 *   block_table_out  the same entries with the pages' new numbers; the others,
 *                    and those that are no page, -1
 *   pages            one number: 1 + the highest page in use or held, 0 if none
 * held pages are not moved, whoever else uses them.  Pages that moved keep
 * their bytes in their old place too.  block_table_out may be exactly
 * block_table.  Two kernel launches, four and a memset for large tables, and
 * one more for each 64 caches beyond the first.  Arguments, bad indices and
 * errors as mhc_kv_fork.
 */
mhc_status mhc_kv_compact(const mhc_kv_cache *caches, int num_caches, const int32_t *block_table,
                          int64_t table_width, const int32_t *seq_lens, int64_t B,
                          const uint8_t *held, int32_t *block_table_out, int32_t *pages,
                          void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of the two calls (0 for sizes that they refuse). */
size_t mhc_kv_fork_workspace_bytes(int64_t num_pages, int64_t table_width, int64_t B);
size_t mhc_kv_compact_workspace_bytes(int64_t num_pages, int64_t B);

#ifdef __cplusplus
}
#endif

#endif /* MHC_KV_H */
