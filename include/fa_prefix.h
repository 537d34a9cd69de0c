/*
 * fa_prefix.h - single tokens of a batch whose sequences share long prefixes
 * (libfa.so).
 *
 * A system prompt, a document or a prompt that is sampled many times is held
 * once: the block tables of its sequences begin with the same cache blocks.
 * fa_decode_paged reads and multiplies those blocks for every sequence again;
 * this call does it once for a group.  Its results are fa_decode_paged's on
 * the same table, up to the order of the sums.
 *
 * Conventions, layouts, types, statuses and remaining arguments are those of
 * fa_decode_paged (fa.h).
 */
#ifndef FA_PREFIX_H_
#define FA_PREFIX_H_

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of workspace of fa_decode_paged_prefix, 0 for invalid arguments.  A
 * workspace of this size serves every call of at most `batch` sequences and
 * at most these lengths with the same H, Hkv and d.
 */
size_t fa_decode_prefix_workspace_size(int batch, int H, int Hkv, int d, int max_prefix_len,
                                       int max_own_len, int block_size);

/*
 * One query token per sequence over a paged cache; groups of neighbouring
 * sequences share the blocks of their first keys.
 *   q, out         : [batch, H, d] bf16;  lse : [batch, H] fp32, may be NULL
 *   k_pool, v_pool : [num_blocks, block_size, Hkv, d] bf16, block_size == 16
 *   block_table    : int32 [batch, max_blocks_per_seq], each row with the
 *                    blocks of all its keys, shared ones first
 *   ctx_lens       : int32 [batch], all keys of a sequence, shared ones counted
 *   cu_groups      : int32 DEVICE array [num_groups + 1], non-decreasing: group g
 *                    is the sequences [cu_groups[g], cu_groups[g + 1]).  A
 *                    sequence in no group has no shared keys.  num_groups 0:
 *                    no groups (the array is not looked at).
 *   prefix_lens    : int32 DEVICE array [num_groups]: the first prefix_lens[g]
 *                    keys of every sequence of the group are the same.  Whole
 *                    blocks are shared, 16 * floor(prefix_lens[g] / 16) keys,
 *                    read through the table row of the group's first sequence
 *                    that has them all (of its longest one, where none has); the
 *                    keys from there on are read through each sequence's own.
 *                    A sequence may be shorter than its prefix, the first one
 *                    too, and sees its first ctx_lens keys (0 for a padded slot of
 *                    the batch); its row holds the blocks of those alone.
 *   max_prefix_len : an upper bound of prefix_lens
 *   max_own_len    : an upper bound of ctx_lens[b] less its group's prefix_lens
 *   workspace      : fa_decode_prefix_workspace_size() bytes, 256-byte aligned;
 *                    with its control block as fa_decode_paged's
 * A sequence with ctx_len 0 gets out = 0 and lse = -inf, a query with a NaN
 * NaN in both.  Shared values (V) that are infinite or NaN reach the rows of
 * the group's sequences that see them, whatever their weight; values past a
 * sequence's own context reach nothing of it.  (A sequence shorter than its
 * prefix whose group holds such values behind its keys is summed on its own.)
 * Device-side checks: FA_DEV_BAD_SEQLEN (a group outside the batch, of
 * negative size, or, behind such a one, that begins before the end of an earlier
 * one: it is passed over, and sequences in no other group read all keys as their
 * own), FA_DEV_BAD_CTX (prefix_lens outside [0, max_prefix_len] or the table:
 * nothing is shared; ctx_lens negative, beyond the table or more than
 * max_own_len + 15 keys behind the shared blocks: the row gets out = 0 and lse =
 * -inf),
 * FA_DEV_BAD_BLOCK (rows that need the block hold nothing of use).
 * Supported: d in {64, 128}, H / Hkv <= 16, num_groups <= 65535 (above the batch
 * too: groups may be empty), and, with n = ceil(batch / (2 floor(128 / (H / Hkv)))),
 * min(num_groups n, n + min(num_groups, batch)) * Hkv * ceil(max_prefix_len / 128)
 * below 2^31.  Three kernels: the shared keys on the
 * tensor cores, the own keys beside them, and the (m, l, o) combine; a call over
 * few keys reads them all as own ones (the results are the same up to the order
 * of the sums).
 */
int fa_decode_paged_prefix(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *ctx_lens, const int32_t *cu_groups,
                           const int32_t *prefix_lens, int num_groups, int max_prefix_len,
                           int max_own_len, int batch, int H, int Hkv, int d, int block_size,
                           int num_blocks, float scale, void *out, float *lse, void *workspace,
                           size_t workspace_bytes, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_PREFIX_H_ */
