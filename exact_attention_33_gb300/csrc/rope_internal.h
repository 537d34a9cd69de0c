// rope_internal.h - parameter blocks of the rotary kernels, shared by the host
// glue (fa_rope_api.cu) and the kernels.  Passed by value.
#pragma once

#include <stdint.h>

#include "fa_internal.h"

namespace fa {

// What a rotation is made of (include/fa_rope.h).
struct RopeSpec {
  const double *inv_freq;  // [pairs] radians a position
  int pairs;               // rot_dim / 2, a multiple of 8 (0: rows are copied)
  float factor;
};

// Rows [H, d] of tokens that lie `stride` elements apart, and where they go.
struct RopeRows {
  const void *src;
  void *dst;
  int64_t src_stride, dst_stride;
  int heads;
};

struct RopeParams {
  unsigned int *status;  // per-device sticky FA_DEV_* word
  RopeSpec rope;
  RopeRows q, k;             // (append: k's dst is not used)
  const int32_t *positions;  // [total_tokens], or null: token t at t % seq_len
  int seq_len, total_tokens;
  int head_lanes;  // threads that share a token's heads for each 16-value unit
  // packed tokens of a cache write
  RopeRows v;
  void *k_pool, *v_pool;       // bf16 [num_blocks, 16, Hkv, d]
  const int32_t *block_table;  // [batch, max_blocks_per_seq]
  const int32_t *ctx_lens;     // [batch], the new tokens counted
  const int32_t *cu_seqlens;   // [batch + 1]
  int batch, max_new, max_blocks_per_seq, num_blocks;
};

}  // namespace fa
