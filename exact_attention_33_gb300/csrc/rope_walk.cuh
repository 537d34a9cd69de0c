// rope_walk.cuh - the walk of a CTA's threads over tokens and their heads that
// rotates rows (rope.cu), shared by the kernels that write a cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "checks.cuh"
#include "ptx.cuh"
#include "rope_common.cuh"
#include "rope_internal.h"

namespace fa {

constexpr int kRopeThreads = 256;

// Rows to rows, tokens in a line; the packed tokens of a cache write with their
// keys and values into a bf16 cache, or their queries alone.
constexpr int kRopeRows = 0, kRopeCache = 1, kRopeQueries = 2;

// What is left of [tokens, heads, D] rows from token t on, in elements.
__device__ __forceinline__ size_t rows_left(int tokens, int t, int64_t stride, int heads, int d) {
  return static_cast<size_t>(tokens - 1 - t) * stride + static_cast<size_t>(heads) * d;
}

// CTA `cta` of the call (of sequence blockIdx.y where tokens are packed).
template <int D, bool INTER, bool BACK, int MODE>
__device__ __forceinline__ void rope_walk(const RopeParams &p, int cta) {
  constexpr bool PACKED = MODE != kRopeRows, APPEND = MODE == kRopeCache;
  constexpr int kUnits = D / 16;
  const int u = threadIdx.x % kUnits;
  const int hl = (threadIdx.x / kUnits) % p.head_lanes;
  const int tokens = kRopeThreads / (kUnits * p.head_lanes);  // of a CTA
  const long long mine =
      static_cast<long long>(cta) * tokens + threadIdx.x / (kUnits * p.head_lanes);
  int t = 0, pos = 0;  // the row and its position
  bool live = true;
  uint16_t *k_dst = nullptr, *v_dst = nullptr;
  if constexpr (PACKED) {
    const int b = blockIdx.y;
    const bool report = cta == 0 && threadIdx.x == 0;
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
    if (static_cast<long long>(cta) * tokens >= n) return;  // the whole CTA
    live = mine < n;
    if (live) {
      t = start + static_cast<int>(mine);
      pos = ctx - n + static_cast<int>(mine);
    }
    if (APPEND && live) {
      const size_t at = static_cast<size_t>(b) * p.max_blocks_per_seq + pos / kDecodeBlock;
      const int phys = checked_load(p.block_table, at,
                                    static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status);
      if (phys >= 0 && phys < p.num_blocks) {
        const size_t row = (static_cast<size_t>(phys) * kDecodeBlock + pos % kDecodeBlock) *
                           p.k.heads * D;
        k_dst = static_cast<uint16_t *>(p.k_pool) + row;
        v_dst = static_cast<uint16_t *>(p.v_pool) + row;
      } else if (hl == 0 && u == 0) {
        raise_status(p.status, FA_DEV_BAD_BLOCK);
      }
    }
  } else {
    live = mine < p.total_tokens;
    if (live) t = static_cast<int>(mine);
    pos = p.positions ? checked_load(p.positions, t, p.total_tokens, p.status) : t % p.seq_len;
  }

  // The token's heads in a row: q's, k's and, into a cache, v's.  A row whose
  // block is bad keeps its queries.
  const int hq = p.q.src ? p.q.heads : 0;
  const int hk = MODE == kRopeQueries ? 0 : (APPEND ? k_dst : p.k.src) ? p.k.heads : 0;
  const int heads = live ? hq + hk + (APPEND ? hk : 0) : 0;
  const uint16_t *src_q = static_cast<const uint16_t *>(p.q.src) + t * p.q.src_stride;
  const uint16_t *src_k = static_cast<const uint16_t *>(p.k.src) + t * p.k.src_stride;
  const uint16_t *src_v = static_cast<const uint16_t *>(p.v.src) + t * p.v.src_stride;
  uint16_t *dst_q = static_cast<uint16_t *>(p.q.dst) + t * p.q.dst_stride;
  if constexpr (MODE == kRopeRows) k_dst = static_cast<uint16_t *>(p.k.dst) + t * p.k.dst_stride;
  auto src = [&](int h) {
    return h < hq ? src_q + h * D : h < hq + hk ? src_k + (h - hq) * D : src_v + (h - hq - hk) * D;
  };
  auto dst = [&](int h) {
    return h < hq ? dst_q + h * D : h < hq + hk ? k_dst + (h - hq) * D : v_dst + (h - hq - hk) * D;
  };
  // (checked build) both pieces of head h lie in their buffers
  auto inside = [&](int h, bool write) {
    const RopeRows &r = h < hq ? p.q : h < hq + hk ? p.k : p.v;
    const uint16_t *base = static_cast<const uint16_t *>(
        !write ? r.src : !APPEND || h < hq ? r.dst : h < hq + hk ? p.k_pool : p.v_pool);
    const size_t n = write && APPEND && h >= hq
                         ? static_cast<size_t>(p.num_blocks) * kDecodeBlock * r.heads * D
                         : rows_left(p.total_tokens, 0, write ? r.dst_stride : r.src_stride, r.heads, D);
    return in_bounds((write ? dst(h) : src(h)) - base, D, n, p.status);
  };

  const RopeUnit unit(u, p.rope.pairs, INTER);
  UnitAngles a{};
  constexpr int kFlight = 4;
  uint4 x[kFlight], y[kFlight];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int hh = h + i * p.head_lanes;
      x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
      if (hh < heads && inside(hh, false)) {
        x[i] = *reinterpret_cast<const uint4 *>(src(hh) + unit.o0);
        y[i] = *reinterpret_cast<const uint4 *>(src(hh) + unit.o1);
      }
    }
  };
  load(hl);  // in flight while the angles are formed
  auto angle = [&](int i) {
    const float2 cs = rope_cos_sin(
        rope_turns(checked_load(p.rope.inv_freq, u * 8 + i, p.rope.pairs, p.status)), pos);
    return make_float2(cs.x * p.rope.factor, (BACK ? -cs.y : cs.y) * p.rope.factor);
  };
  if (p.head_lanes == 1) {
    if (unit.turns) a.set(angle);
  } else {
    // The threads of a unit form its angles together: cosines at [0, 8), sines
    // at [8, 16) of a row of 20 floats (16-byte reads of 8 neighbouring rows
    // then fall on different banks).
    __shared__ __align__(16) float shared_angles[kRopeThreads / 2][20];
    float *row = shared_angles[threadIdx.x / (kUnits * p.head_lanes) * kUnits + u];
    if (unit.turns)
      for (int i = hl; i < 8; i += p.head_lanes) {
        const float2 cs = angle(i);
        row[i] = cs.x;
        row[8 + i] = cs.y;
      }
    __syncthreads();
    if (unit.turns) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = *reinterpret_cast<const float4 *>(row + 4 * i);
        const float4 s = *reinterpret_cast<const float4 *>(row + 8 + 4 * i);
        a.c[2 * i] = make_float2(c.x, c.y);
        a.c[2 * i + 1] = make_float2(c.z, c.w);
        a.s[2 * i] = make_float2(s.x, s.y);
        a.s[2 * i + 1] = make_float2(s.z, s.w);
      }
    }
  }
  for (int h = hl; h < heads;) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int hh = h + i * p.head_lanes;
      if (hh >= heads) break;
      if (unit.turns && hh < hq + hk) {
        float2 v[8];
        rotate_unit<INTER>(a, x[i], y[i], v);
        x[i] = pack_bf16x8(v);
        y[i] = pack_bf16x8(v + 4);
      }
      if (inside(hh, true)) {
        *reinterpret_cast<uint4 *>(dst(hh) + unit.o0) = x[i];
        *reinterpret_cast<uint4 *>(dst(hh) + unit.o1) = y[i];
      }
    }
    h += kFlight * p.head_lanes;
    if (h < heads) load(h);
  }
}

// Threads that share a unit's heads: as many as make kRopeWantThreads, and as
// leave each no more than kRopeMostHeads.  (A thread to itself for all heads
// forms its angles once and leaves few, long CTAs: 73 k tokens of 16 / 4 heads, two
// calls, 230 us against 227, 34.8 k of 32 / 8 heads into a cache 133 against 130; with
// too few threads 20 k tokens of 5 heads took 50 us instead of 21.)
constexpr long long kRopeWantThreads = 128 * 1024;
constexpr int kRopeMostHeads = 16;
template <int D>
inline int rope_head_lanes(long long rows, int heads) {
  int lanes = 1;
  while (lanes * 2 * (D / 16) <= kRopeThreads && 2 * lanes <= heads &&
         (rows * (D / 16) * lanes < kRopeWantThreads || heads > kRopeMostHeads * lanes))
    lanes *= 2;
  return lanes;
}

// CTAs for `tokens` tokens
template <int D>
inline unsigned rope_ctas(long long tokens, int head_lanes) {
  const int per = kRopeThreads / (D / 16 * head_lanes);
  return static_cast<unsigned>((tokens + per - 1) / per);
}

}  // namespace fa
