// cache_internal.h - parameter blocks of the 8-bit cache's kernels, shared by
// the host glue (fa_cache_api.cu) and the kernels.  Passed by value.
#pragma once

#include <stdint.h>

#include "fa_internal.h"

namespace fa {

struct AppendParams {
  unsigned int *status;       // per-device sticky FA_DEV_* word
  const void *k, *v;          // bf16 rows of [Hkv, d], k_stride / v_stride elements apart
  int64_t k_stride, v_stride;
  void *k_pool, *v_pool;      // e4m3 codes [num_blocks, 16, Hkv, d]
  float *k_scale, *v_scale;   // fp32 [num_blocks, Hkv]
  const int32_t *block_table;  // [batch, max_blocks_per_seq]
  const int32_t *ctx_lens;     // [batch], the new tokens counted
  const int32_t *cu_seqlens;   // [batch + 1]
  int batch, total_tokens, max_new;
  int Hkv, max_blocks_per_seq, num_blocks;
};

// The scales of an 8-bit pool, fp32 [num_blocks, Hkv].
struct CacheScales {
  const float *k, *v;
};

}  // namespace fa
