// decode_own.cu - the keys that a sequence has for itself behind a shared
// prefix (prefix.cu): decode.cu's split kernel from the prefix on.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "checks.cuh"
#include "decode_common.cuh"
#include "decode_range.cuh"
#include "fa_internal.h"
#include "launch.h"
#include "prefix_internal.h"
#include "ptx.cuh"

namespace fa {

// One warp per (sequence, KV head, split of keys [whole, ctx)).
template <int D, int NT>
__global__ void __launch_bounds__(32)
    decode_own_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefixParams pp) {
  const DecodeParams &p = pp.own;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x;
  pdl_launch_dependents();
  PrefixGroup group{};
  long long start;
  const int whole = prefix_find(pp, b, true, group, start) ? group.whole : 0;
  const int ctx = prefix_ctx(pp, b, whole, split == 0 && kvh == 0 && lane == 0);
  const int t0 = whole + split * p.split_tokens;
  if (t0 >= ctx) return;
  const int t1 = min(ctx, t0 + p.split_tokens);
  int my_blk = -1;
  if (lane < (t1 - t0 + kDecodeBlock - 1) / kDecodeBlock) {
    const size_t tidx = static_cast<size_t>(b) * p.max_blocks_per_seq + t0 / kDecodeBlock + lane;
    if (in_bounds(tidx, 1, static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status))
      my_blk = p.block_table[tidx];
  }
  const size_t part_row = static_cast<size_t>(b) * p.H + static_cast<size_t>(kvh) * p.group;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  WarpRange<D, NT> st;
  const int rc = decode_range<D, NT, false>(tm_k, tm_v, p, b, kvh, t0, t1, my_blk, smem, st,
                                            WindowBlocks(ctx, 0, 0), ctx);
  if (rc == kRangeBadBlock) store_neutral<D>(p, part_row, split);
  if (rc == kRangeOk) store_range<D, NT>(p, part_row, split, st);
}

namespace {

template <int D, int NT>
cudaError_t launch_own_t(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                         cudaStream_t stream) {
  using L = DecodeLayout<D>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = allow_smem(decode_own_kernel<D, NT>, L::kSmemAlloc, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.own.max_splits, p.own.Hkv, p.own.batch);
  decode_own_kernel<D, NT><<<grid, 32, L::kSmemAlloc, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_own(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                              int d, cudaStream_t stream) {
  const bool two = p.own.group > 8;
  if (d == 64) return two ? launch_own_t<64, 2>(tk, tv, p, stream)
                          : launch_own_t<64, 1>(tk, tv, p, stream);
  return two ? launch_own_t<128, 2>(tk, tv, p, stream) : launch_own_t<128, 1>(tk, tv, p, stream);
}

}  // namespace fa
