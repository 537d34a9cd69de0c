// prefill_fp8cache.cu - instantiations of the prefill kernel for query chunks
// over a paged 8-bit cache, every key up to each query's own or a window with
// sinks: two heads of a KV group over the same 128 rows per CTA when the group
// is even, else two row tiles of one head.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "prefill_kernel.cuh"

namespace fa {

template <int D>
static cudaError_t launch_prefill_fp8cache_d(const CUtensorMap &tq, const CUtensorMap &tk,
                                             const CUtensorMap &tv, const CUtensorMap &to,
                                             const PrefillParams &p, bool head_pairs, int grid,
                                             cudaStream_t stream) {
  return head_pairs
             ? launch_prefill_t<D, true, kKindPagedHeads, false, 2, true, true>(tq, tk, tv, tv, to, p,
                                                                               grid, stream)
             : launch_prefill_t<D, true, kKindPaged, false, 2, true, true>(tq, tk, tv, tv, to, p,
                                                                          grid, stream);
}

cudaError_t launch_prefill_fp8cache(const CUtensorMap &tq, const CUtensorMap &tk,
                                    const CUtensorMap &tv, const CUtensorMap &to,
                                    const PrefillParams &p, int d, bool head_pairs, int grid,
                                    cudaStream_t stream) {
  return d == 64 ? launch_prefill_fp8cache_d<64>(tq, tk, tv, to, p, head_pairs, grid, stream)
                 : launch_prefill_fp8cache_d<128>(tq, tk, tv, to, p, head_pairs, grid, stream);
}

}  // namespace fa
