// decode_own.cu - the keys that a sequence has for itself behind a shared
// prefix: decode.cu's split kernel from the prefix on.
//
// Launched behind prefix.cu's kernel as its programmatic dependent: its CTAs start
// once that kernel's have, on the SMs that are left, and on the others as they
// end.  The combine waits for this grid alone, so its first CTA waits for that
// kernel.
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

// Blocks in a warp's ring.  A warp takes 0.6 us for a block that is there, so
// what counts is warps: rings of two blocks let twice as many of them run as
// decode.cu's of four.  (Alone on the GPU it reads 5.6 TB/s.)
constexpr int kOwnStages = 2;

// One warp per (sequence, KV head, split of keys [whole, ctx)).
template <int D, int NT>
__global__ void __launch_bounds__(32)
    decode_own_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefixParams pp) {
  const DecodeParams &p = pp.own;
  // the KV heads of a split side by side: their rows lie so in the pools
  const int split = blockIdx.x / p.Hkv, kvh = blockIdx.x - split * p.Hkv, b = blockIdx.y;
  const int lane = threadIdx.x;
  pdl_launch_dependents();
  // (a loose max_own_len makes many CTAs without keys: most leave here)
  if (split > 0 && split * p.split_tokens >= checked_load(p.ctx_lens, b, p.batch, p.status)) return;
  const bool first = split == 0 && kvh == 0 && b == 0;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (lane == 0) raise_status(p.status, FA_DEV_SMEM_ALIGN);
    if (first) pdl_wait_primary();
    return;
  }
  PrefixGroup group{};
  const int whole = prefix_walk<kPrefixBySeq>(pp, b, false, group, nullptr) ? group.whole : 0;
  const int ctx = prefix_ctx(pp, b, whole, split == 0 && kvh == 0 && lane == 0);
  if (pp.alone && first) {  // nobody else looks at the groups
    PrefixSums sums;
    PrefixGroup none{};
    prefix_walk<kPrefixNone>(pp, 0, true, none, &sums);
  }
  const int t0 = prefix_own_from(pp, group) + split * p.split_tokens;
  if (t0 >= ctx) {
    if (first) pdl_wait_primary();
    return;
  }
  const int t1 = min(ctx, t0 + p.split_tokens);
  int my_blk = -1;
  if (lane < (t1 - t0 + kDecodeBlock - 1) / kDecodeBlock) {
    const size_t tidx = static_cast<size_t>(b) * p.max_blocks_per_seq + t0 / kDecodeBlock + lane;
    if (in_bounds(tidx, 1, static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status))
      my_blk = p.block_table[tidx];
  }
  const size_t part_row = static_cast<size_t>(b) * p.H + static_cast<size_t>(kvh) * p.group;
  WarpRange<D, NT> st;
  const int rc = decode_range<D, NT, false, kOwnStages>(tm_k, tm_v, p, b, kvh, t0, t1, my_blk, smem,
                                                        st, WindowBlocks(ctx, 0, 0), ctx);
  if (rc == kRangeBadBlock) store_neutral<D>(p, part_row, split);
  if (rc == kRangeOk) store_range<D, NT>(p, part_row, split, st);
  if (first) pdl_wait_primary();
}

namespace {

template <int D, int NT>
cudaError_t launch_own_t(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                         cudaStream_t stream) {
  using L = DecodeLayout<D, kOwnStages>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = allow_smem(decode_own_kernel<D, NT>, L::kBytes, smem_set);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.own.max_splits) * p.own.Hkv, p.own.batch);
  if (!p.alone)
    return launch_dependent(decode_own_kernel<D, NT>, grid, dim3(32), L::kBytes, stream, tk, tv, p);
  decode_own_kernel<D, NT><<<grid, 32, L::kBytes, stream>>>(tk, tv, p);
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
