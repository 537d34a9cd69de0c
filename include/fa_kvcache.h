/*
 * fa_kvcache.h - a paged KV cache held in 8 bits, and attention over it
 * (libfa.so).
 *
 * The cache is that of fa_decode_paged and fa_fwd_paged with e4m3 codes in
 * place of bf16 values, and one fp32 scale for each (block, KV head):
 *   k_pool,  v_pool  : [num_blocks, 16, Hkv, d] e4m3 codes (one byte each)
 *   k_scale, v_scale : [num_blocks, Hkv] fp32, finite and > 0 for blocks in use
 *   key j of a sequence, KV head h : code * k_scale[block of j][h]
 * The attention calls take any such scales; fa_cache_append_fp8 writes powers
 * of two.  Pools must be 16-byte aligned; conventions, statuses and remaining
 * arguments are those of fa.h.
 *
 * window and sinks: 0, 0 for every key (a causal chunk's up to each query's
 * own), or as in fa_window.h (window >= 1, sinks >= 0).  sinks without a
 * window, or a negative value, is FA_ERR_INVALID_ARG.
 */
#ifndef FA_KVCACHE_H_
#define FA_KVCACHE_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantises new keys and values and writes them into the cache: for sequence
 * b the n = cu_seqlens[b + 1] - cu_seqlens[b] tokens that end at position
 * ctx_lens[b] - 1 (ctx_lens counts them already, as the attention calls want
 * it), prompts and single tokens alike.
 *   k, v         : bf16 [total_tokens, Hkv, d], the heads of a token dense,
 *                  tokens k_stride / v_stride elements apart (a multiple of
 *                  8, >= Hkv * d), so views of a fused projection serve
 *   cu_seqlens   : int32 DEVICE array [batch + 1] (rules as fa_fwd_varlen)
 *   max_new      : an upper bound of every sequence's n (sizes the launch)
 * Each block and head that gets a token gets the scale
 *   need = the smallest power of two >= 2^-100 with amax <= 448 need, amax the
 *          largest finite magnitude among the block's new values, and
 *   scale' = need if the block's slot 0 is new, else max(scale, need).
 * Where an older block's scale grows, its codes in the slots before the new
 * ones become e4m3(code * (scale / scale')); new codes are e4m3(x / scale').
 * Roundings are to nearest, ties to even; infinities saturate to +-448
 * scale', NaN stays NaN.  Slots behind the new ones, and every other block,
 * stay as they are.  A written block belongs to one sequence (a block shared
 * by several is copied before one of them writes on it).
 * Device-side checks: FA_DEV_BAD_SEQLEN (bad cu_seqlens, or n > max_new),
 * FA_DEV_BAD_CTX (ctx_lens < n, or beyond the table) - the sequence is
 * skipped; FA_DEV_BAD_BLOCK - the block is.
 */
int fa_cache_append_fp8(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                        void *k_pool, void *v_pool, float *k_scale, float *v_scale,
                        const int32_t *block_table, int max_blocks_per_seq,
                        const int32_t *ctx_lens, const int32_t *cu_seqlens, int batch,
                        int total_tokens, int max_new, int Hkv, int d, int block_size,
                        int num_blocks, fa_stream_t stream);

/*
 * fa_decode_paged over the 8-bit cache: one query token per sequence.  The
 * scores are formed from the codes and from Q in two 8-bit terms, exact to
 * 2^-21 of a query row's largest value; weights (times their blocks' v_scale) are
 * rounded to 11 bits, below 2^-26 of a head's largest to multiples of 2^-36 of it;
 * sums are fp32.
 *   q, out    : [batch, H, d] bf16;  lse : [batch, H] fp32, may be NULL
 *   workspace : fa_decode_workspace_size(), or with a window
 *               fa_decode_window_workspace_size() bytes (fa_window.h);
 *               the conventions of fa_decode_paged
 * Slots outside the context and hidden ones never reach the result; blocks
 * without a visible key are not read.  An infinite or NaN value of q makes its
 * row's out and lse NaN (0 and -inf stand for a context without keys alone).
 * Supported: H / Hkv <= 16.
 */
int fa_decode_paged_fp8(const void *q, const void *k_pool, const void *v_pool,
                        const float *k_scale, const float *v_scale, const int32_t *block_table,
                        int max_blocks_per_seq, const int32_t *ctx_lens, int max_ctx_len,
                        int batch, int H, int Hkv, int d, int block_size, int num_blocks,
                        float scale, int window, int sinks, void *out, float *lse,
                        void *workspace, size_t workspace_bytes, fa_stream_t stream);

/*
 * fa_fwd_paged (causal) over the 8-bit cache: query chunks, the last rows of
 * each sequence's context.  The products run as in fa_fwd_paged: on K's codes
 * as they are, with q exact down to 2^-13 of its row's largest value and off
 * by at most 2^-21 of that below, and on V widened to bf16, exactly where a
 * block's scale is a power of two, with one bf16 rounding where it is not.  An
 * infinite or NaN value of q makes its row's out and lse NaN.
 *   q, out : [total_q, H, d] bf16;  lse : [H, total_q] fp32, may be NULL
 * Slots past the context never reach the result; a block that no query of a
 * 128-row tile sees (a window's) is not read and may be freed.  A query that
 * sees no key gets out = 0 and lse = -inf.
 */
int fa_fwd_paged_fp8(const void *q, const void *k_pool, const void *v_pool, const float *k_scale,
                     const float *v_scale, const int32_t *block_table, int max_blocks_per_seq,
                     const int32_t *ctx_lens, const int32_t *cu_seqlens_q, int batch, int total_q,
                     int max_seqlen_q, int max_ctx_len, int H, int Hkv, int d, int block_size,
                     int num_blocks, float scale, int window, int sinks, void *out, float *lse,
                     fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_KVCACHE_H_ */
