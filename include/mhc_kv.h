/*
 * mhc_kv.h -- C ABI of the paged 8-bit key/value cache of libmhc.so: the
 * attention sublayer's cache that a decoder keeps next to the mHC seam
 * (mhc.h).  Between mhc_pre_delayed, which forms the sublayer's input, and
 * mhc_post, which takes its output, an attention sublayer projects queries,
 * keys and values; mhc_kv_append rotates them and stores keys and values, and
 * mhc_kv_attend is the causal attention of the new tokens over the cache.
 *
 * The conventions of mhc.h hold: caller-owned device pointers of the current
 * device, bf16 as uint16_t, asynchronous calls on the given stream, host-side
 * checks before any launch, no allocation and no synchronisation inside a
 * call; both calls can be captured in a CUDA graph.  What only the device
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

/* Workspace bytes mhc_kv_attend needs on the current device (0: none). */
size_t mhc_kv_attend_workspace_bytes(const mhc_kv_cache *cache, int q_heads, int64_t B, int64_t T);

#ifdef __cplusplus
}
#endif

#endif /* MHC_KV_H */
