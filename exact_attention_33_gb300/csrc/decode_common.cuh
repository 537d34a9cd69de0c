// decode_common.cuh - what the decode kernels of bf16 and 8-bit caches share.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "fa_internal.h"

namespace fa {

// The cache blocks that a windowed query (at position ctx - 1) reads: the
// first nsb blocks (sinks) and those from block wb0 on, nvb in all, counted
// in that order.  The window starts at key lo.
struct WindowBlocks {
  int nsb, wb0, nvb, lo;
  __device__ __forceinline__ WindowBlocks(int ctx, int window, int sinks) {
    lo = max(0, ctx - window);
    const int nb = (ctx + kDecodeBlock - 1) / kDecodeBlock;
    nsb = min((sinks + kDecodeBlock - 1) / kDecodeBlock, nb);
    wb0 = lo / kDecodeBlock;
    if (wb0 <= nsb) nsb = wb0 = 0;  // no block lies between
    nvb = nsb + nb - wb0;
  }
  // block of the sequence that is the v-th to be read
  __device__ __forceinline__ int logical(int v) const { return v < nsb ? v : v - nsb + wb0; }
};

// The maximum that a split reports for a row, m with sum l.  A row whose scores
// are all NaN leaves its maximum at -inf, which the combine takes for a split
// without keys: it reports 0, so that its NaN sums make the row NaN.
__device__ __forceinline__ float split_max(float m, float l) {
  return (m == -CUDART_INF_F && l != l) ? 0.f : m;
}

// The (m, l, o) combine of a split decode call (decode.cu), launched as a
// programmatic dependent of the split grid on the same stream.
cudaError_t launch_decode_combine(const DecodeParams &p, int d, cudaStream_t stream);

}  // namespace fa
