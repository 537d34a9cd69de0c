// cache_append.cu - quantises new keys and values into a paged e4m3 cache.
//
// One warp per (sequence, block that gets tokens, KV head, K or V).  It reads
// the block's new bf16 rows once (16-byte loads, all of them in flight before
// the first is used, kept in registers), takes their largest finite
// magnitude, forms the scale as a power of two and writes the codes.  Old
// codes of a partly filled block are read and written again only when its
// scale grows.  Bound by HBM: 2 bytes read and 1 written for each value.
//
// The scale is a power of two, so that x / scale and the growth of a block's
// scale are exact but for e4m3's own rounding (a code re-encoded at a larger
// scale changes only if it falls below e4m3's normal range), and a block
// filled token by token differs from one filled at once by no more than that.
// It costs up to one of the nearly 15 binades of e4m3's normal values, and no
// precision above the smallest.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_internal.h"
#include "checks.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

// Small CTAs at high occupancy, 4 warps and 10 CTAs per SM: 34.8 k tokens of 8
// heads of d = 128 (214 MB) take 37 us, 33 of them in the kernel.  (With an older
// maximum and division, 45 us, 8 warps took 49 us and 16 took 63, whose slowest
// warp holds the others' registers; 8 or 9 CTAs take as long as 10 at d = 128
// and 2 us more at d = 64.)
constexpr int kAppendWarps = 4;
constexpr int kAppendCtas = 10;
constexpr int kMinScaleExp = -100;

// Smallest e >= kMinScaleExp with the bf16 magnitude `bits` (finite) at most
// 448 * 2^e: 448 = 1.75 * 2^8, so e is the value's exponent - 8, or - 7
// when its significand is above 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - 8 + ((bits & 0x7Fu) > 0x60u ? 1 : 0);
  return max(e, kMinScaleExp);
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t word) {
  const uint32_t lo = word & 0x7FFFu, hi = (word >> 16) & 0x7FFFu;
  m = max(m, lo < 0x7F80u ? lo : 0u);
  return max(m, hi < 0x7F80u ? hi : 0u);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas)
    cache_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;        // lanes of a row: 8 values (16 bytes of bf16) each
  constexpr int kRows = 32 / kLanes;   // rows a warp loads at once
  constexpr int kIter = kDecodeBlock / kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  // unit: (block of the sequence's new tokens, head, K or V), K and V of a
  // head side by side
  const long long unit = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
  const int nth = static_cast<int>(unit / (2 * p.Hkv));
  const int h = static_cast<int>(unit % (2 * p.Hkv)) >> 1;
  const bool is_v = (unit & 1) != 0;
  const bool report = unit == 0 && lane == 0;

  const int start = checked_load(p.cu_seqlens, b, p.batch + 1, p.status);
  const int end = checked_load(p.cu_seqlens, b + 1, p.batch + 1, p.status);
  const int ctx = checked_load(p.ctx_lens, b, p.batch, p.status);
  if (start < 0 || end < start || end > p.total_tokens || end - start > p.max_new) {
    if (report) raise_status(p.status, FA_DEV_BAD_SEQLEN);
    return;
  }
  const int n = end - start;
  if (ctx < n || ctx > p.max_blocks_per_seq * static_cast<long long>(kDecodeBlock)) {
    if (report) raise_status(p.status, FA_DEV_BAD_CTX);
    return;
  }
  const int first = ctx - n;  // position of the first new token
  const int blk = first / kDecodeBlock + nth;
  if (n == 0 || blk > (ctx - 1) / kDecodeBlock) return;
  const int pos0 = blk * kDecodeBlock;
  const int s0 = max(0, first - pos0), s1 = min(kDecodeBlock, ctx - pos0);  // new slots

  // the new rows: lane reads values [8 c, 8 c + 8) of rows kRows i + r
  const int c = lane % kLanes, r = lane / kLanes;
  const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.v : p.k);
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  // extent of the input in elements (its last row ends after Hkv * D of them)
  const size_t n_src = static_cast<size_t>(p.total_tokens - 1) * stride + p.Hkv * D;
  uint4 x[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int slot = i * kRows + r;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= s0 && slot < s1) {
      const size_t off = static_cast<size_t>(start + pos0 + slot - first) * stride +
                         static_cast<size_t>(h) * D + c * 8;
      if (in_bounds(off, 8, n_src, p.status)) x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + off));  // read once
    }
  }
  const size_t tidx = static_cast<size_t>(b) * p.max_blocks_per_seq + blk;
  const int phys = checked_load(p.block_table, tidx,
                                static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status);
  if (phys < 0 || phys >= p.num_blocks) {
    if (lane == 0) raise_status(p.status, FA_DEV_BAD_BLOCK);
    return;
  }
  float *scales = is_v ? p.v_scale : p.k_scale;
  const size_t sidx = static_cast<size_t>(phys) * p.Hkv + h;
  const size_t n_scales = static_cast<size_t>(p.num_blocks) * p.Hkv;
  const float old = s0 > 0 ? checked_load(scales, sidx, n_scales, p.status) : 0.f;

  // largest magnitude, both halves of a word at once; a warp that meets an
  // infinity or a NaN looks again at the finite ones
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    m2 = __vmaxu2(m2, x[i].x & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, x[i].y & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, x[i].z & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, x[i].w & 0x7FFF7FFFu);
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  if (m >= 0x7F80u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      m = finite_max(m, x[i].x);
      m = finite_max(m, x[i].y);
      m = finite_max(m, x[i].z);
      m = finite_max(m, x[i].w);
    }
    m = __reduce_max_sync(0xffffffffu, m);
  }
  const float need = pow2(scale_exponent(m));
  const float scale = fmaxf(old, need);  // (a NaN or negative old scale counts as none)

  // row `slot` of the block's head, this lane's 8 codes
  uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool);
  const size_t n_pool = static_cast<size_t>(p.num_blocks) * kDecodeBlock * p.Hkv * D;
  auto at = [&](int slot) {
    return ((static_cast<size_t>(phys) * kDecodeBlock + slot) * p.Hkv + h) * D + c * 8;
  };
  if (s0 > 0 && !(scale <= old)) {
    // the block's older codes at its new scale
    const float ratio = old > 0.f ? old / scale : 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int slot = i * kRows + r;
      if (slot < s0 && in_bounds(at(slot), 8, n_pool, p.status)) {
        uint2 w = *reinterpret_cast<const uint2 *>(pool + at(slot));
        uint32_t *half = &w.x;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 lo = e4m3x2_to_float2(half[e]), hi = e4m3x2_to_float2(half[e] >> 16);
          half[e] = pack_e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
        }
        *reinterpret_cast<uint2 *>(pool + at(slot)) = w;
      }
    }
  }
  // A power of two is divided by through its reciprocal, which is exact; a
  // scale that someone else wrote may be none.
  const bool is_pow2 = (__float_as_uint(scale) & 0x007FFFFFu) == 0u;
  auto write = [&](auto code) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int slot = i * kRows + r;
      if (slot < s0 || slot >= s1) continue;
      const float2 a = code(bf16x2_to_float2(x[i].x)), e = code(bf16x2_to_float2(x[i].y));
      const float2 f = code(bf16x2_to_float2(x[i].z)), g = code(bf16x2_to_float2(x[i].w));
      uint2 w;
      w.x = pack_e4m3x4(a.x, a.y, e.x, e.y);
      w.y = pack_e4m3x4(f.x, f.y, g.x, g.y);
      if (in_bounds(at(slot), 8, n_pool, p.status)) *reinterpret_cast<uint2 *>(pool + at(slot)) = w;
    }
  };
  if (is_pow2) {
    const float2 inv = make_float2(1.f / scale, 1.f / scale);
    write([&](float2 v) { return fmul2(v, inv); });
  } else {
    write([&](float2 v) { return make_float2(v.x / scale, v.y / scale); });
  }
  if (lane == 0 && scale != old && in_bounds(sidx, 1, n_scales, p.status)) scales[sidx] = scale;
}

cudaError_t launch_cache_append(const AppendParams &p, int d, cudaStream_t stream) {
  // the new tokens of a sequence may begin inside a block
  const long long blocks = (p.max_new + 2LL * kDecodeBlock - 2) / kDecodeBlock;
  const long long units = blocks * p.Hkv * 2;
  const dim3 grid(static_cast<unsigned>((units + kAppendWarps - 1) / kAppendWarps),
                  static_cast<unsigned>(p.batch));
  if (d == 64)
    cache_append_kernel<64><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  else
    cache_append_kernel<128><<<grid, 32 * kAppendWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
