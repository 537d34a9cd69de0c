// decode.cu - paged GQA flash-decoding for sm_103a.
//
// "S12 FlashAttention", section "How this composes with what you already
// built": one loop that walks the block table, loads the KV head shared by a
// group of query heads, scores the block and updates (m, l, o).  Section
// "What this unlocks beyond speed" (flash-decoding): with one query token
// there is no parallelism over queries, so the keys of a sequence are split
// across thread blocks, each producing a partial (m, l, o), and a second
// kernel merges the partial states with the same rescaling as the tile
// recurrence (explainer page, "Show the maths").
//
// decode_split_kernel: one warp per (sequence, KV head, split of the
// context).  The 16-token KV blocks named by the block table are fetched
// with TMA (128-byte swizzle) into a ring of shared-memory stages, several
// blocks in flight per warp.  Per block:
//   S^T [16 tokens x 8 heads] = K_blk [16 x d] . Q^T   (mma.m16n8k16, the G
//       query heads of the group are the N columns, padded to 8)
//   column-wise online softmax over the 16 tokens (warp shuffles)
//   O^T [d x 8] += V_blk^T [d x 16] . P^T [16 x 8]     (P^T re-laid out with
//       movmatrix from the S^T accumulator layout)
// The work is bound by HBM reads of K and V; the tensor-core ops are a small
// fraction of the issue slots.
//
// A windowed call (WIN) reads the blocks of the sinks and of the window alone
// and masks the hidden tokens of the first window block and the last sink
// block as it masks slots past the context; its splits run over the blocks
// that are read (64 sequences of 512 to 32768 keys, 32 / 8 heads of d = 128,
// window 4096: 165 us for 1.02 GB, 6.2 TB/s).
//
// decode_combine_kernel: one CTA per (sequence, query head) merges the
// partial states: M = max m_i, L = sum 2^(m_i - M) l_i,
// o = sum 2^(m_i - M) o_i / L, lse = (M + log2 L) ln 2.  A row gets 1, 4 or
// 16 warps by its number of splits (one warp per row and four rows per CTA
// for large batches of short contexts, 16 for small batches of long ones).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "decode_common.cuh"
#include "decode_range.cuh"
#include "fa_internal.h"
#include "ptx.cuh"
#include "checks.cuh"

namespace fa {

template <int D, int NT, bool WIN>
__global__ void __launch_bounds__(32)
    decode_split_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const DecodeParams p) {
  const int split = blockIdx.x;
  const int kvh = blockIdx.y;
  const int b = blockIdx.z;
  const int lane = threadIdx.x;
  pdl_launch_dependents();

  // The block ids of the whole split are read together with the context
  // length (one memory round trip instead of two); ids past the context are
  // not used.
  const int lb0 = split * (p.split_tokens / kDecodeBlock);
  int my_blk = -1;
  auto read_block_id = [&](int lb) {
    const size_t tidx = static_cast<size_t>(b) * p.max_blocks_per_seq + lb;
    if (in_bounds(tidx, 1, static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status))
      my_blk = p.block_table[tidx];
  };
  if (!WIN && lane < p.split_tokens / kDecodeBlock && lb0 + lane < p.max_blocks_per_seq)
    read_block_id(lb0 + lane);
  const int ctx = checked_load(p.ctx_lens, b, p.batch, p.status);
  if (ctx < 0 || ctx > p.max_ctx_len ||
      ctx > p.max_blocks_per_seq * static_cast<long long>(kDecodeBlock)) {
    if (split == 0 && kvh == 0 && lane == 0) raise_status(p.status, FA_DEV_BAD_CTX);
    return;
  }
  const WindowBlocks wb(ctx, p.window, p.sinks);
  const int keys = WIN ? wb.nvb * kDecodeBlock : ctx;  // keys of the blocks to be read
  const int t0 = split * p.split_tokens;
  if (t0 >= keys) return;
  const int t1 = min(keys, t0 + p.split_tokens);
  // (which blocks a window reads depends on the context length)
  if (WIN && lane < (t1 - t0) / kDecodeBlock) read_block_id(wb.logical(lb0 + lane));
  const size_t part_row = static_cast<size_t>(b) * p.H + static_cast<size_t>(kvh) * p.group;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  WarpRange<D, NT> st;
  const int rc =
      decode_range<D, NT, WIN>(tm_k, tm_v, p, b, kvh, t0, t1, my_blk, smem, st, wb, ctx);
  if (rc == kRangeBadBlock) store_neutral<D>(p, part_row, split);
  if (rc == kRangeOk) store_range<D, NT>(p, part_row, split, st);
}

// Warps per merged row: one for rows of at most kCombineFewSplits splits
// (four rows per CTA), kCombineWarps up to kCombineManySplits, and
// kCombineWarpsMany beyond (rows of many short splits: small batches).
constexpr int kCombineFewSplits = 8;
constexpr int kCombineManySplits = 64;
constexpr int kCombineWarpsMany = 16;

template <int W>
constexpr int combine_cta_warps() { return W < 4 ? 4 : W; }

template <int D, int W>
__global__ void __launch_bounds__(32 * combine_cta_warps<W>())
    decode_combine_kernel(const DecodeParams p) {
  // W warps per (sequence, query head) row, R rows per CTA.  The W warps of
  // a row first find M together (thread t of the row reads the maxima of
  // splits t, t + 32 W, ...); then warp w of the row merges splits w, w + W,
  // ..., U of them per memory round trip, and the warps' sums are added
  // through shared memory.  Lane l owns output elements [l E, l E + E).
  constexpr int kWarps = combine_cta_warps<W>();
  constexpr int R = kWarps / W;
  constexpr int E = D / 32;
  constexpr int U = 8;
  __shared__ float s_acc[kWarps][D];
  __shared__ float s_l[kWarps];
  __shared__ float s_m[kWarps];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // this kernel's own (checked-build) index errors go to the device word only
  unsigned int *status = p.dev_status;
  const int wr = warp % W;  // warp within the row
  const int r0 = warp - wr;  // first warp of the row
  const int gw = blockIdx.x * R + warp / W;
  // a CTA's last rows may lie past the end; they still meet the barriers
  const bool row_live = gw < p.batch * p.H;
  const int b = row_live ? gw / p.H : 0;
  int ctx = row_live ? checked_load(p.ctx_lens, b, p.batch, status) : 0;
  if (ctx < 0 || ctx > p.max_ctx_len ||
      ctx > p.max_blocks_per_seq * static_cast<long long>(kDecodeBlock))
    ctx = 0;
  const int keys = p.window > 0 ? WindowBlocks(ctx, p.window, p.sinks).nvb * kDecodeBlock : ctx;
  const int ns = (keys + p.split_tokens - 1) / p.split_tokens;
  const size_t row0 = static_cast<size_t>(gw) * p.max_splits;
  const size_t part_rows = static_cast<size_t>(p.batch) * p.H * p.max_splits;
  pdl_wait_primary();  // the split grid's partial states are complete from here on
  // The split grid has raised all its status bits: one thread reads them
  // here and publishes them as the call's status when its row is done.
  const bool publisher = blockIdx.x == 0 && threadIdx.x == 0 && p.call != nullptr;
  const unsigned int call_bits = publisher ? call_status_bits(p.call) : 0u;
  // (m, l) of split i of this row (the neutral state if the index fails a
  // check of the checked build)
  auto ml = [&](int i) -> float2 {
    return in_bounds(row0 + i, 1, part_rows, status)
               ? reinterpret_cast<const float2 *>(p.ml_part)[row0 + i]
               : make_float2(-CUDART_INF_F, 0.f);
  };

  float M = -CUDART_INF_F;
  for (int i = wr * 32 + lane; i < ns; i += 32 * W) M = fmaxf(M, ml(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[r0 + w]);

  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float Lsum = 0.f;
  // Split i adds 2^(m_i - M) (l_i, o_i).  An empty split (m_i = -inf) is
  // passed over by a select, never multiplied in, so whatever its o_i slot
  // holds cannot reach the output.
  if (M != -CUDART_INF_F) {
    auto add = [&](const float2 st, const float (&v)[E]) {
      const bool live = st.x != -CUDART_INF_F;
      const float w = ex2(st.x - M);
      Lsum = live ? fmaf(w, st.y, Lsum) : Lsum;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = live ? fmaf(w, v[e], acc[e]) : acc[e];
    };
    auto load_o = [&](int i, float (&v)[E]) {
      const float *orow = p.o_part + (row0 + i) * D + lane * E;
      if (!in_bounds((row0 + i) * D + lane * E, E, part_rows * D, status)) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
        return;
      }
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(orow);
        v[0] = x.x;
        v[1 % E] = x.y;
        v[2 % E] = x.z;
        v[3 % E] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2 *>(orow);
        v[0] = x.x;
        v[1 % E] = x.y;
      }
    };
    int i = wr;
    for (; i + (U - 1) * W < ns; i += U * W) {
      float2 st[U];
      float v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        st[u] = ml(i + u * W);
        load_o(i + u * W, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add(st[u], v[u]);
    }
    for (; i < ns; i += W) {
      float v[E];
      load_o(i, v);
      add(ml(i), v);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  if (lane == 0) s_l[warp] = Lsum;
  __syncthreads();
  if (wr != 0 || !row_live) return;
  Lsum = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) Lsum += s_l[r0 + w];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += s_acc[r0 + w][lane * E + e];
    acc[e] = t;
  }
  // (0: no key seen; NaN goes on to the row)
  const float inv = (Lsum == 0.f) ? 0.f : 1.f / Lsum;
  uint16_t *dst = static_cast<uint16_t *>(p.out) + static_cast<size_t>(gw) * D + lane * E;
  const bool out_ok = in_bounds(static_cast<size_t>(gw) * D + lane * E, E,
                                static_cast<size_t>(p.batch) * p.H * D, status);
  if (out_ok && E == 4) {
    uint2 w;
    w.x = pack_bf16x2(acc[0] * inv, acc[1 % E] * inv);
    w.y = pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv);
    *reinterpret_cast<uint2 *>(dst) = w;
  } else if (out_ok) {
    *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1 % E] * inv);
  }
  if (lane == 0 && p.lse != nullptr &&
      in_bounds(gw, 1, static_cast<size_t>(p.batch) * p.H, status))
    p.lse[gw] = (Lsum == 0.f) ? -CUDART_INF_F : (M + __log2f(Lsum)) * 0.69314718055994530942f;
  if (publisher) publish_call_status(p.call, call_bits, p.dev_status);
}

// ------------------------------------------------------------------ launch

// The combine grid, launched as a programmatic dependent of the split grid
// on the same stream.
template <int D, int W>
static cudaError_t launch_combine(const DecodeParams &p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(32 * combine_cta_warps<W>());
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_combine_kernel<D, W>, p);
}

template <int D>
static cudaError_t launch_combine_d(const DecodeParams &p, cudaStream_t stream) {
  const int rows = p.batch * p.H;
  if (p.max_splits > kCombineManySplits)
    return launch_combine<D, kCombineWarpsMany>(p, rows, stream);
  if (p.max_splits > kCombineFewSplits) return launch_combine<D, kCombineWarps>(p, rows, stream);
  return launch_combine<D, 1>(p, (rows + 3) / 4, stream);
}

cudaError_t launch_decode_combine(const DecodeParams &p, int d, cudaStream_t stream) {
  return d == 64 ? launch_combine_d<64>(p, stream) : launch_combine_d<128>(p, stream);
}

template <int D, int NT, bool WIN>
static cudaError_t launch_decode_t(const CUtensorMap &tk, const CUtensorMap &tv,
                                   const DecodeParams &p, cudaStream_t stream) {
  using L = DecodeLayout<D>;
  auto kern = decode_split_kernel<D, NT, WIN>;
  // The shared-memory attribute is per device: set it once on each device
  // (one bit per device id; ids past 63 set it on every launch).
  static std::atomic<unsigned long long> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit == 0ull || (attr_set.load(std::memory_order_acquire) & bit) == 0ull) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemAlloc);
    if (e != cudaSuccess) return e;
    attr_set.fetch_or(bit, std::memory_order_release);
  }
  dim3 grid(p.max_splits, p.Hkv, p.batch);
  kern<<<grid, 32, L::kSmemAlloc, stream>>>(tk, tv, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_combine_d<D>(p, stream) : e;
}

template <int D, int NT>
static cudaError_t launch_decode_w(const CUtensorMap &tk, const CUtensorMap &tv,
                                   const DecodeParams &p, cudaStream_t stream) {
  return p.window > 0 ? launch_decode_t<D, NT, true>(tk, tv, p, stream)
                      : launch_decode_t<D, NT, false>(tk, tv, p, stream);
}

cudaError_t launch_decode(const CUtensorMap &tk, const CUtensorMap &tv, const DecodeParams &p,
                          int d, cudaStream_t stream) {
  const bool two = p.group > 8;
  if (d == 64) return two ? launch_decode_w<64, 2>(tk, tv, p, stream)
                          : launch_decode_w<64, 1>(tk, tv, p, stream);
  return two ? launch_decode_w<128, 2>(tk, tv, p, stream)
             : launch_decode_w<128, 1>(tk, tv, p, stream);
}

}  // namespace fa
