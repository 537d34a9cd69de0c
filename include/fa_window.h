/*
 * fa_window.h - windowed attention with sinks (libfa.so).
 *
 * Every call here is the call of fa.h with the same name less `_window`, for
 * causal attention in which a query also leaves out keys that lie too far
 * back.  Positions count from the start of a sequence; a query's position is
 * that of its own token (bottom-right alignment over a cache: query i of a
 * chunk of Nq over ctx_len keys stands at i + ctx_len - Nq; a decode query at
 * ctx_len - 1).  The query at position p sees key j when
 *
 *     j <= p  and  (j > p - window  or  j < sinks),
 *
 * that is the last `window` keys, its own among them, and the first `sinks`
 * keys of the sequence, which stay visible.  The softmax runs over the
 * visible keys alone.  A query that sees none (possible over a cache shorter
 * than its chunk) gets out = 0 and lse = -inf.
 *   window : >= 1; a window longer than the sequence leaves plain causal attention
 *   sinks  : >= 0; 0 for none
 * (window < 1 or sinks < 0: FA_ERR_INVALID_ARG.)
 *
 * Conventions, layouts, types, statuses, workspaces and the remaining
 * arguments are those of fa.h.  Work and traffic grow with
 * tokens * (window + sinks): key tiles between the sinks and the window are
 * neither read nor computed.  The products multiply whole tiles of 128 keys
 * by weights that are 0 for hidden keys, so a value (V; in a backward pass
 * also K, Q and dO) that is infinite or NaN reaches the rows of its sequence
 * whose tiles hold it, as in fa.h's calls; rows of other sequences, and
 * packed rows behind the last sequence, never reach a sequence's results.
 * A query with a NaN gets out = NaN and lse = NaN.
 */
#ifndef FA_WINDOW_H_
#define FA_WINDOW_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fa_fwd (causal) with a window: q, out [B, N, H, d]; k, v [B, N, Hkv, d]. */
int fa_fwd_window(const void *q, const void *k, const void *v, void *out, float *lse, int B, int H,
                  int Hkv, int N, int d, float scale, int window, int sinks, fa_stream_t stream);

/* fa_fwd_varlen (causal) with a window: packed sequences, each with its own
   positions and sinks.  Rows behind the last sequence are left as they were. */
int fa_fwd_varlen_window(const void *q, const void *k, const void *v, void *out, float *lse,
                         const int32_t *cu_seqlens, int num_seqs, int total_tokens, int max_seqlen,
                         int H, int Hkv, int d, float scale, int window, int sinks,
                         fa_stream_t stream);

/* fa_fwd_paged (causal) with a window: query chunks over a paged KV cache.
   Blocks that no query of a 128-row tile sees are not read and their table
   entries are not looked at, so a serving loop may free the blocks that lie
   behind the window of the chunk's first query (but those that hold sinks). */
int fa_fwd_paged_window(const void *q, const void *k_pool, const void *v_pool,
                        const int32_t *block_table, int max_blocks_per_seq,
                        const int32_t *ctx_lens, const int32_t *cu_seqlens_q, int batch,
                        int total_q, int max_seqlen_q, int max_ctx_len, int H, int Hkv, int d,
                        int block_size, int num_blocks, float scale, int window, int sinks,
                        void *out, float *lse, fa_stream_t stream);

/* fa_decode_paged with a window: one query token per sequence.  Reads the
   blocks of the window and of the sinks alone; the table entries of the
   others are not looked at.  Slots outside the context, and hidden slots of
   the first window block and of the last sink block, never reach the result,
   whatever they hold.
   The workspace has fa_decode_window_workspace_size() bytes (window and
   sinks 0: those of a call over every key), which serve smaller batches and
   contexts too; it and its control block are those of fa_decode_paged. */
size_t fa_decode_window_workspace_size(int batch, int H, int Hkv, int d, int max_ctx_len,
                                       int block_size, int window, int sinks);
int fa_decode_paged_window(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *ctx_lens, int max_ctx_len, int batch, int H, int Hkv,
                           int d, int block_size, int num_blocks, float scale, int window,
                           int sinks, void *out, float *lse, void *workspace,
                           size_t workspace_bytes, fa_stream_t stream);

/* Gradients of fa_fwd_window and fa_fwd_varlen_window (the products of fa_bwd
   over the visible pairs); lse as those calls wrote it, with the same window and
   sinks.  out is not read (the row sums of dS come from P and dP) and may be
   NULL.  The workspace has
   fa_bwd_window_workspace_size() bytes (a packed batch: B = num_seqs,
   N = max_seqlen), 256-byte aligned, overwritten, one call at a time.  One sized
   for some B and N serves every smaller B and N with the same H, Hkv, d, window
   and sinks.
   A packed batch with a bad cu_seqlens entry: as fa_bwd_varlen. */
size_t fa_bwd_window_workspace_size(int B, int H, int Hkv, int N, int d, int window, int sinks);
int fa_bwd_window(const void *q, const void *k, const void *v, const void *out, const float *lse,
                  const void *dout, void *dq, void *dk, void *dv, int B, int H, int Hkv, int N,
                  int d, float scale, int window, int sinks, void *workspace,
                  size_t workspace_bytes, fa_stream_t stream);
int fa_bwd_varlen_window(const void *q, const void *k, const void *v, const void *out,
                         const float *lse, const void *dout, void *dq, void *dk, void *dv,
                         const int32_t *cu_seqlens, int num_seqs, int total_tokens, int max_seqlen,
                         int H, int Hkv, int d, float scale, int window, int sinks,
                         void *workspace, size_t workspace_bytes, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_WINDOW_H_ */
