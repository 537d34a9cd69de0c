/*
 * fa_rope.h - rotary positions (libfa.so): queries and keys rotated by their
 * positions, their gradients rotated back, and the writes into a paged cache
 * that rotate on the way.
 *
 * The attention calls of fa.h, fa_window.h and fa_kvcache.h take queries and
 * keys that carry their positions already; these calls put them there.  A head
 * of d values holds rot_dim / 2 pairs (a, b), pair i at
 *   half layout        : a = x[i],     b = x[i + rot_dim / 2]
 *   interleaved layout : a = x[2 i],   b = x[2 i + 1]
 * and x[rot_dim .. d) is passed through as it is.  At position p
 *   a' = factor (a cos t - b sin t),   b' = factor (a sin t + b cos t),
 *   t = p * inv_freq[i].
 *   inv_freq : fp64 DEVICE array [rot_dim / 2], radians a position (finite).
 *              How contexts are stretched (slower frequencies for some pairs)
 *              is in these values and in factor.
 *   factor   : finite and > 0 (1, or what a stretched context wants)
 * The angle is the exact product, reduced to one turn in 64-bit integers (turns a
 * position are held to 2^-53 of themselves or 2^-64, the angle to 2^-56 of a turn): a
 * position of 2^31 costs no accuracy that bf16 values show, and the sine of a small
 * angle of either sign is as near as that of a large one.  Values are rotated in
 * fp32 and rounded once.
 *
 * Conventions and statuses are those of fa.h.  Rows of one token are dense
 * ([heads, d]); tokens lie `stride` elements apart, a multiple of 8 and at
 * least heads * d, so views of a fused projection serve.  q, k, v and the
 * outputs are 16-byte aligned.  An output may be its input itself (same
 * address and stride); other overlaps are not allowed.
 * Supported: d in {64, 128}, rot_dim a multiple of 16 up to d.
 */
#ifndef FA_ROPE_H_
#define FA_ROPE_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotates queries and keys.
 *   q, q_out  : bf16 [total_tokens, H, d];  k, k_out : bf16 [total_tokens, Hkv, d]
 *               (Hkv 0: no keys, k and k_out are not looked at)
 *   positions : int32 DEVICE array [total_tokens] (any value, packed batches
 *               and offsets alike), or NULL: token t stands at t % seq_len, a
 *               dense batch [B, N, ...] with seq_len = N (>= 1)
 */
int fa_rope(const void *q, const void *k, int64_t q_stride, int64_t k_stride, void *q_out,
            void *k_out, int64_t q_out_stride, int64_t k_out_stride, const double *inv_freq,
            int rot_dim, float factor, int interleaved, const int32_t *positions, int seq_len,
            int total_tokens, int H, int Hkv, int d, fa_stream_t stream);

/*
 * The gradient of fa_rope: dq, dk of its outputs become those of its inputs,
 * the transposed rotation  a = factor (a' cos t + b' sin t),  b = factor
 * (b' cos t - a' sin t).  Arguments as fa_rope.
 */
int fa_rope_bwd(const void *dq, const void *dk, int64_t dq_stride, int64_t dk_stride, void *dq_out,
                void *dk_out, int64_t dq_out_stride, int64_t dk_out_stride, const double *inv_freq,
                int rot_dim, float factor, int interleaved, const int32_t *positions, int seq_len,
                int total_tokens, int H, int Hkv, int d, fa_stream_t stream);

/*
 * Writes new keys, rotated, and values into the bf16 cache of fa_fwd_paged and
 * fa_decode_paged, and rotates the queries that come with them: for sequence b
 * the n = cu_seqlens[b + 1] - cu_seqlens[b] tokens that end at position
 * ctx_lens[b] - 1 (ctx_lens counts them already, as the attention calls want
 * it), prompts and single tokens alike.
 *   q, q_out       : bf16 [total_tokens, H, d], or both NULL (H is not looked
 *                    at): keys and values alone
 *   k, v           : bf16 [total_tokens, Hkv, d]
 *   inv_freq       : NULL with rot_dim 0: nothing is rotated, rows are copied
 *   k_pool, v_pool : bf16 [num_blocks, block_size, Hkv, d], block_size == 16
 *   cu_seqlens     : int32 DEVICE array [batch + 1] (rules as fa_fwd_varlen)
 *   max_new        : an upper bound of every sequence's n (sizes the launch; 0:
 *                    nothing is done, nor looked at)
 * Slots behind the new ones, rows of q_out behind the last sequence and every
 * other block stay as they are.  A written block belongs to one sequence.
 * Device-side checks: FA_DEV_BAD_SEQLEN (bad cu_seqlens, or n > max_new),
 * FA_DEV_BAD_CTX (ctx_lens < n, or beyond the table) - the sequence is
 * skipped; FA_DEV_BAD_BLOCK - the block's keys and values are.
 */
int fa_cache_append_rope(const void *q, const void *k, const void *v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, void *q_out, int64_t q_out_stride,
                         const double *inv_freq, int rot_dim, float factor, int interleaved,
                         void *k_pool, void *v_pool, const int32_t *block_table,
                         int max_blocks_per_seq, const int32_t *ctx_lens,
                         const int32_t *cu_seqlens, int batch, int total_tokens, int max_new,
                         int H, int Hkv, int d, int block_size, int num_blocks,
                         fa_stream_t stream);

/*
 * The same into the 8-bit cache of fa_kvcache.h: fa_cache_append_fp8 with its
 * keys rotated on the way, in fp32, without a rounding to bf16 between, and
 * the queries as above (rot_dim >= 16).  The rule of the scales is
 * fa_cache_append_fp8's with, for keys, amax times max(1, fp32(sqrt(2)
 * factor)), amax of the block's new keys before the rotation, which grows none
 * by more: so scales come from the inputs' bits alone and no rounding of an
 * angle moves them; they are at most twice what the largest of the rotated
 * keys could need.  Where amax times that leaves fp32, the scale is 2^120.
 */
int fa_cache_append_rope_fp8(const void *q, const void *k, const void *v, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, void *q_out,
                             int64_t q_out_stride, const double *inv_freq, int rot_dim,
                             float factor, int interleaved, void *k_pool, void *v_pool,
                             float *k_scale, float *v_scale, const int32_t *block_table,
                             int max_blocks_per_seq, const int32_t *ctx_lens,
                             const int32_t *cu_seqlens, int batch, int total_tokens, int max_new,
                             int H, int Hkv, int d, int block_size, int num_blocks,
                             fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_ROPE_H_ */
