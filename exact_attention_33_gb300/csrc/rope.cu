// rope.cu - rotary positions: queries and keys rotated in place or from rows
// to rows, and on the way into a bf16 paged cache.
//
// A thread owns one unit of one token (rope_common.cuh): it forms the 8 angles
// once and walks over the token's heads with them, q's and k's (and copies
// v's), 4 rows in flight.  `head_lanes` threads share the heads of a unit; the
// host takes more of them the fewer tokens there are.
// Bound by HBM: 2 bytes read and 2 written for each value.  73 k packed
// tokens of 16 / 4 heads, d = 128 (752 MB): 113 us, 6.6 TB/s, 98% of a plain copy's
// rate; 2 x 8192 tokens of 32 / 32 heads (537 MB) 85 us, 93%; 34.8 k tokens of 32 / 8
// heads with their values into a bf16 cache (856 MB) 130 us, 97%.  64 single
// tokens take 5 us, of which the launch is most.
#include <cuda_runtime.h>
#include <stdint.h>

#include "rope_internal.h"
#include "rope_walk.cuh"

namespace fa {

// 80 registers a thread hold four rows in flight; three CTAs of 256 threads are
// what the register file then takes.
constexpr int kRopeCtas = 3;

template <int D, bool INTER, bool BACK, int MODE>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeParams p) {
  rope_walk<D, INTER, BACK, MODE>(p, blockIdx.x);
}

namespace {

template <int D, bool INTER, bool BACK, int MODE>
cudaError_t launch_rope_t(RopeParams p, cudaStream_t stream) {
  constexpr bool APPEND = MODE == kRopeCache;
  const int heads = (p.q.src ? p.q.heads : 0) + (APPEND ? 2 : 1) * (p.k.src ? p.k.heads : 0);
  p.head_lanes = rope_head_lanes<D>(
      APPEND ? static_cast<long long>(p.batch) * p.max_new : p.total_tokens, heads);
  const dim3 grid(rope_ctas<D>(APPEND ? p.max_new : p.total_tokens, p.head_lanes),
                  static_cast<unsigned>(APPEND ? p.batch : 1));
  rope_kernel<D, INTER, BACK, MODE><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool BACK, int MODE>
cudaError_t launch_rope_d(const RopeParams &p, int d, bool interleaved, cudaStream_t stream) {
  if (d == 64)
    return interleaved ? launch_rope_t<64, true, BACK, MODE>(p, stream)
                       : launch_rope_t<64, false, BACK, MODE>(p, stream);
  return interleaved ? launch_rope_t<128, true, BACK, MODE>(p, stream)
                     : launch_rope_t<128, false, BACK, MODE>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int d, bool interleaved, bool back,
                        cudaStream_t stream) {
  return back ? launch_rope_d<true, kRopeRows>(p, d, interleaved, stream)
              : launch_rope_d<false, kRopeRows>(p, d, interleaved, stream);
}

cudaError_t launch_append_rope(const RopeParams &p, int d, bool interleaved, cudaStream_t stream) {
  return launch_rope_d<false, kRopeCache>(p, d, interleaved, stream);
}

}  // namespace fa
