// cache_append_rope.cu - quantises new keys, rotated by their positions, and
// values into a paged e4m3 cache, and rotates the queries that come with them.
//
// The first CTAs of a sequence rotate its queries as rope.cu does.  In the
// others a warp takes a block of the sequence's new tokens (16 at most) and
// some of its heads, K's or V's, one after the other; a lane owns one unit of a
// row (rope_common.cuh) and walks through the rows with it.  The warps of a
// block form cos and sin of its 16 positions together, in shared memory, and
// read them for every head.  (Angles in registers, turned on from row to row by
// the angle of a step, take 48 registers more: 144 us for 34.8 k tokens of 32 / 8
// heads of d = 128 where this takes 131, and they are off by 2^-21.)
//
// Scales and older codes are cache_append.cu's, with one difference: a key's
// scale is taken from the block's values before the rotation, times the bound
// of its growth, so that it depends on the inputs' bits alone.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "cache_internal.h"
#include "checks.cuh"
#include "fa_internal.h"
#include "ptx.cuh"
#include "rope_common.cuh"
#include "rope_internal.h"
#include "rope_walk.cuh"

namespace fa {

namespace {

constexpr int kAppendWarps = kRopeThreads / 32;
constexpr int kMaxCtaBlocks = 4;
constexpr int kMinScaleExp = -100;

// Smallest e >= kMinScaleExp with x <= 448 * 2^e (x >= 0, fp32; 2^120 for what
// has left fp32): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float x) {
  const uint32_t bits = __float_as_uint(x);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExp);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// the larger of m and the finite halves of a word, magnitudes
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t word) {
  const uint32_t lo = word & 0x7FFFu, hi = (word >> 16) & 0x7FFFu;
  m = max(m, lo < 0x7F80u ? lo : 0u);
  return max(m, hi < 0x7F80u ? hi : 0u);
}

// 8 codes of values by two's, times inv (or over scale where that is no power of two)
__device__ __forceinline__ uint2 encode8(const float2 *v, float scale, float inv, bool exact) {
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = exact ? fmul2(v[i], make_float2(inv, inv)) : make_float2(v[i].x / scale, v[i].y / scale);
  return make_uint2(pack_e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y),
                    pack_e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
}

}  // namespace

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3)
    cache_append_rope_kernel(const AppendParams p, const RopeParams rp, const float grow,
                             const int q_ctas, const int block_warps, const int cta_blocks) {
  if (static_cast<int>(blockIdx.x) < q_ctas) {
    rope_walk<D, INTER, false, kRopeQueries>(rp, blockIdx.x);
    return;
  }
  constexpr int kLanes = D / 16;       // lanes of a row, one unit each
  constexpr int kRows = 32 / kLanes;   // rows at once
  constexpr int kIter = kDecodeBlock / kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  // A CTA takes cta_blocks blocks with equally many warps each, its part of the
  // block_warps that share a block's heads: warp w of them heads w, w +
  // block_warps, ... of K's and V's.
  const int cta = blockIdx.x - q_ctas, warps = kAppendWarps / cta_blocks;
  const int parts = (block_warps + warps - 1) / warps;  // CTAs of a block
  const int mine = warp / warps;                        // block of the CTA
  const int nth = cta / parts * cta_blocks + mine;
  const int w = cta % parts * warps + warp % warps;
  const bool report = cta == 0 && warp == 0 && lane == 0;

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
  const int pos0 = blk * kDecodeBlock;
  if (n == 0 || blk - mine > (ctx - 1) / kDecodeBlock) return;  // the whole CTA
  const bool active = blk <= (ctx - 1) / kDecodeBlock && w < block_warps;
  const int s0 = max(0, first - pos0), s1 = min(kDecodeBlock, ctx - pos0);  // new slots
  const int row0 = start + pos0 - first;  // the token of slot 0 (may lie before the new ones)
  const int u = lane % kLanes, r = lane / kLanes;
  const RopeUnit unit(u, rp.rope.pairs, INTER);
  const int heads = 2 * p.Hkv;
  const size_t n_scales = static_cast<size_t>(p.num_blocks) * p.Hkv;
  const size_t n_pool = n_scales * kDecodeBlock * D;

  uint4 x[kIter], y[kIter];
  auto load = [&](int h) {
    const bool is_v = h >= p.Hkv;
    const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.v : p.k);
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int hh = is_v ? h - p.Hkv : h;
    const size_t n_src =
        static_cast<size_t>(p.total_tokens - 1) * stride + static_cast<size_t>(p.Hkv) * D;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int slot = i * kRows + r;
      x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= s0 && slot < s1) {
        const size_t off = static_cast<size_t>(row0 + slot) * stride + static_cast<size_t>(hh) * D;
        if (in_bounds(off, D, n_src, p.status)) {
          x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + off + unit.o0));
          y[i] = __ldcs(reinterpret_cast<const uint4 *>(src + off + unit.o1));
        }
      }
    }
  };
  int h = w;
  if (active) load(h);  // in flight while the angles are formed
  // cos and sin of pair 8 u + i of row r of the CTA's blocks: floats i and 8 + i
  // of the 16 of (block, r, u), of which the 16-byte quarter q lies at q ^ (u / 2)
  // % 4 (so that 8 units' quarters fall on different banks)
  __shared__ __align__(16) float angles[kMaxCtaBlocks * kDecodeBlock * kLanes * 16];
  auto place = [&](int row, int unit, int i) {
    return ((row * kLanes + unit) * 4 + ((i / 4) ^ ((unit / 2) & 3))) * 4 + i % 4;
  };
  const int base = pos0 - mine * kDecodeBlock;  // position of the CTA's first row
  const int rows = min(cta_blocks * kDecodeBlock, ctx - base);
  for (int x = threadIdx.x + max(0, first - base) * rp.rope.pairs; x < rows * rp.rope.pairs;
       x += kRopeThreads) {
    const int pair = x % rp.rope.pairs, row = x / rp.rope.pairs;
    const float2 cs = rope_cos_sin(
        rope_turns(checked_load(rp.rope.inv_freq, pair, rp.rope.pairs, p.status)), base + row);
    angles[place(row, pair / 8, pair % 8)] = cs.x * rp.rope.factor;
    angles[place(row, pair / 8, 8 + pair % 8)] = cs.y * rp.rope.factor;
  }
  __syncthreads();
  if (!active) return;
  const int phys = checked_load(p.block_table, static_cast<size_t>(b) * p.max_blocks_per_seq + blk,
                                static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status);
  if (phys < 0 || phys >= p.num_blocks) {
    if (w == 0 && lane == 0) raise_status(p.status, FA_DEV_BAD_BLOCK);
    return;
  }

  for (;;) {
    const bool is_v = h >= p.Hkv;
    const bool turned = !is_v && unit.turns;
    // the rows of this head, in fp32, one after the other
    auto row = [&](int i, float2 (&v)[8]) {
      if (turned) {
        UnitAngles a;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at = mine * kDecodeBlock + i * kRows + r;
          const float4 c = *reinterpret_cast<const float4 *>(&angles[place(at, u, 4 * q)]);
          const float4 s = *reinterpret_cast<const float4 *>(&angles[place(at, u, 8 + 4 * q)]);
          a.c[2 * q] = make_float2(c.x, c.y);
          a.c[2 * q + 1] = make_float2(c.z, c.w);
          a.s[2 * q] = make_float2(s.x, s.y);
          a.s[2 * q + 1] = make_float2(s.z, s.w);
        }
        rotate_unit<INTER>(a, x[i], y[i], v);
      } else {
        const uint32_t word[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = bf16x2_to_float2(word[e]);
      }
    };
    const int hh = is_v ? h - p.Hkv : h;
    float *scales = is_v ? p.v_scale : p.k_scale;
    const size_t sidx = static_cast<size_t>(phys) * p.Hkv + hh;
    const float old = s0 > 0 ? checked_load(scales, sidx, n_scales, p.status) : 0.f;
    // largest magnitude, both halves of a word at once; a warp that meets an
    // infinity or a NaN looks again at the finite ones
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const uint32_t word[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) m2 = __vmaxu2(m2, word[e] & 0x7FFF7FFFu);
    }
    uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
    if (m >= 0x7F80u) {
      m = 0;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const uint32_t word[8] = {x[i].x, x[i].y, x[i].z, x[i].w, y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) m = finite_max(m, word[e]);
      }
      m = __reduce_max_sync(0xffffffffu, m);
    }
    const float top = __uint_as_float(m << 16);
    const float need = pow2(scale_exponent(is_v ? top : top * grow));
    const float scale = fmaxf(old, need);  // (a NaN or negative old scale counts as none)
    uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool);
    auto at = [&](int slot) {
      return ((static_cast<size_t>(phys) * kDecodeBlock + slot) * p.Hkv + hh) * D;
    };
    if (s0 > 0 && !(scale <= old)) {
      // the block's older codes at its new scale
      const float ratio = old > 0.f ? old / scale : 0.f;
      for (int slot = r; slot < s0; slot += kRows) {
        if (!in_bounds(at(slot), D, n_pool, p.status)) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t *code =
              reinterpret_cast<uint32_t *>(pool + at(slot) + (e < 2 ? unit.o0 : unit.o1)) + e % 2;
          const float2 lo = e4m3x2_to_float2(*code), hi = e4m3x2_to_float2(*code >> 16);
          *code = pack_e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
        }
      }
    }
    // A power of two is divided by through its reciprocal, which is exact; a
    // scale that someone else wrote may be none.
    const bool is_pow2 = (__float_as_uint(scale) & 0x007FFFFFu) == 0u;
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int slot = i * kRows + r;
      float2 v[8];
      row(i, v);
      if (slot < s0 || slot >= s1 || !in_bounds(at(slot), D, n_pool, p.status)) continue;
      *reinterpret_cast<uint2 *>(pool + at(slot) + unit.o0) = encode8(v, scale, inv, is_pow2);
      *reinterpret_cast<uint2 *>(pool + at(slot) + unit.o1) = encode8(v + 4, scale, inv, is_pow2);
    }
    if (lane == 0 && scale != old && in_bounds(sidx, 1, n_scales, p.status)) scales[sidx] = scale;
    h += block_warps;
    if (h >= heads) return;
    load(h);
  }
}

namespace {

template <int D, bool INTER>
cudaError_t launch_append_t(const AppendParams &p, RopeParams rp, float grow, cudaStream_t stream) {
  int q_ctas = 0;
  if (rp.q.src) {
    rp.head_lanes = rope_head_lanes<D>(static_cast<long long>(p.batch) * p.max_new, rp.q.heads);
    q_ctas = static_cast<int>(rope_ctas<D>(p.max_new, rp.head_lanes));
  }
  // the new tokens of a sequence may begin inside a block
  const long long blocks = (p.max_new + 2LL * kDecodeBlock - 2) / kDecodeBlock;
  // a warp takes two heads of its block where that leaves two rounds of warps for
  // the GPU (34.8 k tokens of 32 / 8 heads of d = 128: 131 us; four heads 137,
  // eight 149; with 2 CTAs on an SM instead of 3, 148, with 4, 164)
  const long long rounds = blocks * p.batch * 2 * p.Hkv / (2LL * 152 * 16);
  const int per_warp = static_cast<int>(std::min(2LL, std::max(1LL, rounds)));
  const int block_warps = (2 * p.Hkv + per_warp - 1) / per_warp;
  // 2, 4 or 8 warps of a CTA for a block
  int warps = 2;
  while (warps < kAppendWarps && warps < block_warps) warps *= 2;
  const int cta_blocks = kAppendWarps / warps, parts = (block_warps + warps - 1) / warps;
  const dim3 grid(static_cast<unsigned>(q_ctas + (blocks + cta_blocks - 1) / cta_blocks * parts),
                  static_cast<unsigned>(p.batch));
  cache_append_rope_kernel<D, INTER>
      <<<grid, kRopeThreads, 0, stream>>>(p, rp, grow, q_ctas, block_warps, cta_blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append_rope(const AppendParams &p, const RopeParams &rp, float grow, int d,
                                     bool interleaved, cudaStream_t stream) {
  if (d == 64)
    return interleaved ? launch_append_t<64, true>(p, rp, grow, stream)
                       : launch_append_t<64, false>(p, rp, grow, stream);
  return interleaved ? launch_append_t<128, true>(p, rp, grow, stream)
                     : launch_append_t<128, false>(p, rp, grow, stream);
}

}  // namespace fa
