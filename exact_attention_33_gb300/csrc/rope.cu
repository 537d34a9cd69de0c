// rope.cu - rotary positions: queries and keys rotated in place or from rows
// to rows, and on the way into a bf16 paged cache.
//
// A head row of d values is d / 16 units of 16 values: two 16-byte pieces that
// hold 8 pairs (half layout: one piece of each half; interleaved: neighbours),
// or 16 values that pass through.  A thread owns one unit of one token: it
// forms the 8 angles once and walks over the token's heads with them, q's and
// k's (and copies v's), 4 rows in flight.  `head_lanes` threads share the
// heads of a unit; the host takes more of them the fewer tokens there are.
// Bound by HBM: 2 bytes read and 2 written for each value.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "checks.cuh"
#include "ptx.cuh"
#include "rope_common.cuh"
#include "rope_internal.h"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;

// The 8 pairs of a unit: cos and sin (times the factor), in two's.
struct UnitAngles {
  float2 c[4], s[4];
};

// One unit rotated in fp32.  INTER: word w is pair w; else word w of x holds
// the a's of pairs 2w and 2w + 1 and that of y their b's.
template <bool INTER>
__device__ __forceinline__ void rotate_unit(const UnitAngles &t, uint4 &x, uint4 &y) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (INTER) {
      // pairs w (of x) and 4 + w (of y)
      const float2 p = bf16x2_to_float2(a[w]), q = bf16x2_to_float2(b[w]);
      const float pc = w & 1 ? t.c[w / 2].y : t.c[w / 2].x, ps = w & 1 ? t.s[w / 2].y : t.s[w / 2].x;
      const float qc = w & 1 ? t.c[2 + w / 2].y : t.c[2 + w / 2].x;
      const float qs = w & 1 ? t.s[2 + w / 2].y : t.s[2 + w / 2].x;
      a[w] = pack_bf16x2(fmaf(p.x, pc, -(p.y * ps)), fmaf(p.x, ps, p.y * pc));
      b[w] = pack_bf16x2(fmaf(q.x, qc, -(q.y * qs)), fmaf(q.x, qs, q.y * qc));
    } else {
      const float2 u = bf16x2_to_float2(a[w]), v = bf16x2_to_float2(b[w]);
      const float2 ns = make_float2(-t.s[w].x, -t.s[w].y);
      const float2 r0 = ffma2(u, t.c[w], fmul2(v, ns));
      const float2 r1 = ffma2(u, t.s[w], fmul2(v, t.c[w]));
      a[w] = pack_bf16x2(r0.x, r0.y);
      b[w] = pack_bf16x2(r1.x, r1.y);
    }
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}

// Pieces [lo, hi) of the heads h0, h0 + step, ... of one token: rotated with
// `t` where `turn`, copied otherwise.  src and dst point to the token's first
// head; a piece's values start at o0 and at o1 of a head.  `extent` is what a
// buffer holds from those pointers on (checked build).
template <int D, bool INTER>
__device__ __forceinline__ void walk_heads(const uint16_t *src, uint16_t *dst, int h0, int heads,
                                           int step, int o0, int o1, bool turn,
                                           const UnitAngles &t, size_t src_extent,
                                           size_t dst_extent, unsigned int *status) {
  constexpr int kFlight = 4;
  for (int h = h0; h < heads; h += kFlight * step) {
    uint4 x[kFlight], y[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int hh = h + i * step;
      x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
      if (hh < heads && in_bounds(static_cast<size_t>(hh) * D + max(o0, o1), 8, src_extent, status)) {
        x[i] = *reinterpret_cast<const uint4 *>(src + hh * D + o0);
        y[i] = *reinterpret_cast<const uint4 *>(src + hh * D + o1);
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int hh = h + i * step;
      if (hh >= heads) break;
      if (turn) rotate_unit<INTER>(t, x[i], y[i]);
      if (in_bounds(static_cast<size_t>(hh) * D + max(o0, o1), 8, dst_extent, status)) {
        *reinterpret_cast<uint4 *>(dst + hh * D + o0) = x[i];
        *reinterpret_cast<uint4 *>(dst + hh * D + o1) = y[i];
      }
    }
  }
}

// What is left of [tokens, heads, D] rows from token t on, in elements.
__device__ __forceinline__ size_t rows_left(int tokens, int t, int64_t stride, int heads, int d) {
  return static_cast<size_t>(tokens - 1 - t) * stride + static_cast<size_t>(heads) * d;
}

}  // namespace

template <int D, bool INTER, bool BACK, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr int kUnits = D / 16;
  const int u = threadIdx.x % kUnits;
  const int hl = (threadIdx.x / kUnits) % p.head_lanes;
  const int tokens = kRopeThreads / (kUnits * p.head_lanes);  // of a CTA
  const long long mine =
      static_cast<long long>(blockIdx.x) * tokens + threadIdx.x / (kUnits * p.head_lanes);
  int t, pos;  // the row and its position
  uint16_t *k_dst = nullptr, *v_dst = nullptr;
  if constexpr (APPEND) {
    const int b = blockIdx.y;
    const bool report = blockIdx.x == 0 && threadIdx.x == 0;
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
    if (mine >= n) return;
    t = start + static_cast<int>(mine);
    pos = ctx - n + static_cast<int>(mine);
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
  } else {
    if (mine >= p.total_tokens) return;
    t = static_cast<int>(mine);
    pos = p.positions ? checked_load(p.positions, t, p.total_tokens, p.status) : t % p.seq_len;
  }

  const int pairs = p.rope.pairs;
  const bool turn = u < pairs / 8;
  // the unit's two pieces of a head
  const int o0 = turn && !INTER ? 8 * u : 16 * u;
  const int o1 = turn && !INTER ? pairs + 8 * u : 16 * u + 8;
  UnitAngles a{};
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 cs = rope_cos_sin(
          rope_turns(checked_load(p.rope.inv_freq, u * 8 + i, pairs, p.status)), pos);
      const float c = cs.x * p.rope.factor, s = (BACK ? -cs.y : cs.y) * p.rope.factor;
      if (i & 1)
        a.c[i / 2].y = c, a.s[i / 2].y = s;
      else
        a.c[i / 2].x = c, a.s[i / 2].x = s;
    }
  }
  auto rows = [&](const RopeRows &r) {
    if (r.src == nullptr) return;
    walk_heads<D, INTER>(static_cast<const uint16_t *>(r.src) + t * r.src_stride,
                         static_cast<uint16_t *>(r.dst) + t * r.dst_stride, hl, r.heads,
                         p.head_lanes, o0, o1, turn, a,
                         rows_left(p.total_tokens, t, r.src_stride, r.heads, D),
                         rows_left(p.total_tokens, t, r.dst_stride, r.heads, D), p.status);
  };
  rows(p.q);
  if constexpr (APPEND) {
    if (k_dst == nullptr) return;
    const size_t left = (static_cast<size_t>(p.num_blocks) * kDecodeBlock) * p.k.heads * D -
                        (k_dst - static_cast<uint16_t *>(p.k_pool));
    auto cache = [&](const RopeRows &r, uint16_t *dst, bool rotated) {
      walk_heads<D, INTER>(static_cast<const uint16_t *>(r.src) + t * r.src_stride, dst, hl, r.heads,
                           p.head_lanes, o0, o1, rotated, a,
                           rows_left(p.total_tokens, t, r.src_stride, r.heads, D), left, p.status);
    };
    cache(p.k, k_dst, turn);
    cache(p.v, v_dst, false);
  } else {
    rows(p.k);
  }
}

namespace {

template <int D, bool INTER, bool BACK, bool APPEND>
cudaError_t launch_rope_t(RopeParams p, cudaStream_t stream) {
  constexpr int kUnits = D / 16;
  const int heads = std::max(p.q.src ? p.q.heads : 0, p.k.heads);
  // Threads for the GPU: heads are shared among more of them until there are
  // enough, or every head has its own.
  const long long rows = APPEND ? static_cast<long long>(p.batch) * p.max_new : p.total_tokens;
  int lanes = 1;
  while (lanes * 2 * kUnits <= kRopeThreads && lanes < heads && rows * kUnits * lanes < 512 * 1024)
    lanes *= 2;
  p.head_lanes = lanes;
  const int tokens = kRopeThreads / (kUnits * lanes);
  const long long per = APPEND ? p.max_new : p.total_tokens;
  const dim3 grid(static_cast<unsigned>((per + tokens - 1) / tokens),
                  static_cast<unsigned>(APPEND ? p.batch : 1));
  rope_kernel<D, INTER, BACK, APPEND><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool BACK, bool APPEND>
cudaError_t launch_rope_d(const RopeParams &p, int d, bool interleaved, cudaStream_t stream) {
  if (d == 64)
    return interleaved ? launch_rope_t<64, true, BACK, APPEND>(p, stream)
                       : launch_rope_t<64, false, BACK, APPEND>(p, stream);
  return interleaved ? launch_rope_t<128, true, BACK, APPEND>(p, stream)
                     : launch_rope_t<128, false, BACK, APPEND>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int d, bool interleaved, bool back,
                        cudaStream_t stream) {
  return back ? launch_rope_d<true, false>(p, d, interleaved, stream)
              : launch_rope_d<false, false>(p, d, interleaved, stream);
}

cudaError_t launch_append_rope(const RopeParams &p, int d, bool interleaved, cudaStream_t stream) {
  return launch_rope_d<false, true>(p, d, interleaved, stream);
}

}  // namespace fa
