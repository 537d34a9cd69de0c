// decode_fp8.cu - paged GQA flash-decoding over a cache of e4m3 codes with a
// scale for each (16-token block, KV head), every key or a window with sinks.
//
// The plan of decode.cu: one warp per (sequence, KV head, split of the keys),
// blocks fetched with TMA into a ring of shared-memory stages, partial
// (m, l, o) states merged by decode_combine_kernel.  A step takes two blocks
// (32 tokens), since a block is half as large here.  With ks, vs the scales
// of token j's block and c = scale log2(e):
//   x_j = (q . code_j) ks c,  p_j = 2^(x_j - m),  l = sum p_j,
//   o = sum p_j vs code'_j,   out = o / l.
//   S^T [16 tokens x 4 heads x 2] += K [16 x 32 of d] [Qh | Ql]^T on e4m3
//     MMAs (fp32 sums), on the codes as they are; Q goes in as two e4m3 terms.
//     It is scaled per head by a power of two that puts its largest value at
//     2^7..2^8; Qh = e4m3(Q) takes its upper four significand bits and Ql =
//     e4m3(16 (Q - Qh)) the other four, exactly down to 2^-13 of the largest
//     value and to within 2^-21 of it below.  A head's terms are neighbouring
//     columns, so a thread holds both sums and adds them: s = S_h + S_l / 16.
//     Which of d's values stand in which k-slots is free as long as K and Q
//     agree, so a thread takes 32 (d = 64: 16) consecutive codes of a row:
//     whole 16-byte reads.  (With K's codes widened for fp16 MMAs instead,
//     twice as many at half the rate, the benchmark's batch took 544 us where
//     this takes 383.)
//   O^T [16 of d x 8 heads] += V^T P^T on fp16 MMAs: weights are rounded to 11
//     bits and V's codes widened exactly.  V's rows come through a transposing
//     16-bit ldmatrix, whose elements are pairs of codes: the two values of a
//     pair are accumulator rows g and g + 8, so row g of tile u is d = 16 u +
//     2 g, and row g + 8 the next one.  Two e4m3 terms of P would save the
//     widening, but lose weights below 2^-19 of the largest, which a long
//     context has enough of to matter.
// vs goes into the weights: o is kept relative to mo, a running reference of
// x_j + log2 vs, so the weights 2^(x_j + log2 vs - mo) stay in fp16's range
// whatever the scales (the largest at 2^12 to 2^14: 11 bits down to 2^-26 of it,
// multiples of 2^-36 below); the references move only when a maximum grows by more
// than kSlackLog2, which leaves the accumulators alone in most steps.
// Bound by HBM: half of decode.cu's bytes for the same products.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "cache_internal.h"
#include "checks.cuh"
#include "decode_common.cuh"
#include "fa_internal.h"
#include "launch.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kStepBlocks = 2;   // blocks of a step
constexpr int kF8Stages = 3;     // steps in flight per warp
// A weight is 2^kTopLog2 when its reference is fresh and at most 2^(kTopLog2 +
// kSlackLog2) = 2^14 before the reference moves (fp16 ends at 65504, and at
// 2^-24 below).
constexpr float kTopLog2 = 12.f, kSlackLog2 = 2.f;

template <int D>
struct DecodeF8Layout {
  static constexpr int kBlockBytes = kDecodeBlock * D;  // one KV head of one block
  static constexpr int kHalfBytes = kStepBlocks * kBlockBytes;  // K (or V) of a step
  static constexpr int kStageBytes = 2 * kHalfBytes;            // K then V
  static constexpr int kBar = kF8Stages * kStageBytes;
  static constexpr int kMisc = kBar + kF8Stages * 8;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kSmemAlloc = kBytes + 1024;
};

// Byte offset of 16-byte unit u of row t of a block (rows of D bytes in the
// swizzle of that width: 128 or 64).
template <int D>
__device__ __forceinline__ uint32_t f8_off(int t, int u) {
  if constexpr (D == 128) return t * 128 + ((u ^ (t & 7)) << 4);
  return t * 64 + ((u ^ ((t >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(32)
    decode_fp8_split_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const DecodeParams p,
                            const CacheScales sc) {
  using L = DecodeF8Layout<D>;
  constexpr int S = kF8Stages;
  constexpr int W = D / 16;       // words of a K row per thread (two to an MMA)
  constexpr int U = D / 16;       // 16-byte units of a V row, accumulator tiles
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x;
  const int quad = lane & 3, grp = lane >> 2;
  pdl_launch_dependents();

  // Without a window the block ids are read together with the context length
  // (one memory round trip); ids past the context are not used.
  const int lb0 = split * (p.split_tokens / kDecodeBlock);
  int my_blk = -1;
  auto read_block_id = [&](int lb) {
    const size_t tidx = static_cast<size_t>(b) * p.max_blocks_per_seq + lb;
    if (in_bounds(tidx, 1, static_cast<size_t>(p.batch) * p.max_blocks_per_seq, p.status))
      my_blk = p.block_table[tidx];
  };
  const bool windowed = p.window > 0;
  if (!windowed && lane < p.split_tokens / kDecodeBlock && lb0 + lane < p.max_blocks_per_seq)
    read_block_id(lb0 + lane);
  const int ctx = checked_load(p.ctx_lens, b, p.batch, p.status);
  if (ctx < 0 || ctx > p.max_ctx_len ||
      ctx > p.max_blocks_per_seq * static_cast<long long>(kDecodeBlock)) {
    if (split == 0 && kvh == 0 && lane == 0) raise_status(p.status, FA_DEV_BAD_CTX);
    return;
  }
  const WindowBlocks wb(ctx, windowed ? p.window : ctx, p.sinks);
  const int nblk = min(wb.nvb - lb0, p.split_tokens / kDecodeBlock);  // this split's, <= 32
  if (nblk <= 0) return;
  if (windowed && lane < nblk) read_block_id(wb.logical(lb0 + lane));
  const int G = p.group;
  // partial-state rows of the call: [batch, H, max_splits]
  const size_t part_rows = static_cast<size_t>(p.batch) * p.H * p.max_splits;
  const size_t part_row = static_cast<size_t>(b) * p.H + static_cast<size_t>(kvh) * G;

  if (__any_sync(0xffffffffu, lane < nblk && (my_blk < 0 || my_blk >= p.num_blocks))) {
    if (lane == 0) raise_status(p.status, FA_DEV_BAD_BLOCK);
    // a neutral partial state, so that the combine ignores this split
    for (int g = 0; g < G; ++g) {
      const size_t row = (part_row + g) * p.max_splits + split;
      if (!in_bounds(row, 1, part_rows, p.status)) continue;
      for (int c = lane; c < D; c += 32) p.o_part[row * D + c] = 0.f;
      if (lane == 0) {
        p.ml_part[row * 2 + 0] = -CUDART_INF_F;
        p.ml_part[row * 2 + 1] = 0.f;
      }
    }
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBar);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc);
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncwarp();

  const int steps = (nblk + kStepBlocks - 1) / kStepBlocks;
  int issued = 0;
  // lanes 0 .. 3 copy K and V of the step's two blocks (lane = 2 * block + v)
  auto issue = [&](int i) {
    const int st = i % S;
    const int in_step = min(kStepBlocks, nblk - i * kStepBlocks);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], in_step * 2 * L::kBlockBytes);
    __syncwarp();
    const int phys = __shfl_sync(0xffffffffu, my_blk, (i * kStepBlocks + (lane >> 1)) & 31);
    if (lane < 2 * in_step) {
      uint8_t *dst = smem + st * L::kStageBytes + (lane & 1) * L::kHalfBytes +
                     (lane >> 1) * L::kBlockBytes;
      tma_load_3d(dst, (lane & 1) ? &tm_v : &tm_k, &full[st], 0, kvh, phys * kDecodeBlock);
    }
    issued = i + 1;
  };
  for (int i = 0; i < min(S, steps); ++i) issue(i);

  // this lane's block's scales: ks times the softmax scale, log2 of vs
  float my_ks = 0.f, my_lv = 0.f;
  if (lane < nblk) {
    const size_t sidx = static_cast<size_t>(my_blk) * p.Hkv + kvh;
    const size_t n = static_cast<size_t>(p.num_blocks) * p.Hkv;
    my_ks = checked_load(sc.k, sidx, n, p.status) * p.scale_log2;
    my_lv = __log2f(checked_load(sc.v, sidx, n, p.status));
  }

  // Q^T fragments: columns 2 h and 2 h + 1 of N tile nt are the two terms of
  // query head kvh * G + 4 nt + h; word w of a thread holds d = 4 W quad + 4 w
  // .. + 3 of its column, as K's words do.
  uint32_t qf[NT][W];
  float cq[NT];  // 2^-e of the head of this thread's accumulator columns (head quad)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 4 + (grp >> 1);
    const bool valid =
        n < G && in_bounds((part_row + n) * D, D, static_cast<size_t>(p.batch) * p.H * D, p.status);
    const uint4 *qrow = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                        (part_row + (valid ? n : 0)) * D + 4 * W * quad);
    uint32_t raw[2 * W];
#pragma unroll
    for (int c = 0; c < W / 2; ++c) {
      const uint4 x = valid ? qrow[c] : make_uint4(0u, 0u, 0u, 0u);
      raw[4 * c] = x.x;
      raw[4 * c + 1] = x.y;
      raw[4 * c + 2] = x.z;
      raw[4 * c + 3] = x.w;
    }
    uint32_t top = 0;  // largest magnitude of the row, bf16 bits
#pragma unroll
    for (int c = 0; c < 2 * W; ++c)
      top = max(top, max(raw[c] & 0x7FFFu, (raw[c] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent that takes the row to [2^7, 2^8) (a row of zeros, or with an
    // infinity or NaN, stays as it is: e4m3 keeps NaN, and an infinite score
    // has no softmax, so infinities become NaN below)
    const int e = exponent_to_2_7(top);
    const float f0 = pow2_clamped(e / 2), f1 = pow2_clamped(e - e / 2);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 x0 = bf16x2_to_float2(raw[2 * w]), x1 = bf16x2_to_float2(raw[2 * w + 1]);
      const float a = x0.x * f0 * f1, b2 = x0.y * f0 * f1, c = x1.x * f0 * f1, d = x1.y * f0 * f1;
      uint32_t h = pack_e4m3x4(a, b2, c, d);
      if (grp & 1) {  // the second term
        const float2 h0 = e4m3x2_to_float2(h), h1 = e4m3x2_to_float2(h >> 16);
        h = pack_e4m3x4((a - h0.x) * 16.f, (b2 - h0.y) * 16.f, (c - h1.x) * 16.f,
                        (d - h1.y) * 16.f);
      }
      qf[nt][w] = (top >= 0x7F80u) ? 0x7F7F7F7Fu : h;
    }
    cq[nt] = pow2_exact(-__shfl_sync(0xffffffffu, e, quad * 8));
  }

  // O^T: columns 2 h and 2 h + 1 of tile np are heads h of S tiles 2 np and
  // 2 np + 1, so that the thread with a head's scores has its outputs too.
  constexpr int NP = (NT + 1) / 2;
  float acc[NP][U][4];
  float m[NT], mo[NT], l[NT];
#pragma unroll
  for (int np = 0; np < NP; ++np)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[np][u][x] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = mo[nt] = -CUDART_INF_F;
    l[nt] = 0.f;
  }

  bool ok = true;
  for (int i = 0; i < steps; ++i) {
    const int st = i % S;
    ok = mbar_wait(&full[st], (i / S) & 1, abort_flag, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t kb = smem_u32(smem + st * L::kStageBytes);
    const uint32_t vb = kb + L::kHalfBytes;

    float s[NT][kStepBlocks][4];
#pragma unroll
    for (int t = 0; t < kStepBlocks; ++t) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][t][x] = 0.f;
      // rows grp and grp + 8 of the block, 4 W codes each
      uint32_t lo[W], hi[W];
#pragma unroll
      for (int c = 0; c < W / 4; ++c) {
        const int u = quad * (W / 4) + c;
        const uint4 a = lds128(kb + t * L::kBlockBytes + f8_off<D>(grp, u));
        const uint4 d = lds128(kb + t * L::kBlockBytes + f8_off<D>(grp + 8, u));
        lo[4 * c] = a.x, lo[4 * c + 1] = a.y, lo[4 * c + 2] = a.z, lo[4 * c + 3] = a.w;
        hi[4 * c] = d.x, hi[4 * c + 1] = d.y, hi[4 * c + 2] = d.z, hi[4 * c + 3] = d.w;
      }
#pragma unroll
      for (int w = 0; w < W; w += 2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_m16n8k32_e4m3(s[nt][t], lo[w], hi[w], lo[w + 1], hi[w + 1], qf[nt][w],
                            qf[nt][w + 1]);
    }

    // Token masks of the step's blocks: slots past the context (all of them
    // for a block the step lacks) and, windowed, those between sinks and window.
    int n_valid[kStepBlocks], hid0[kStepBlocks], hid1[kStepBlocks];
    float ks[kStepBlocks], lv[kStepBlocks];
    bool masked = false;
#pragma unroll
    for (int t = 0; t < kStepBlocks; ++t) {
      const int vblk = i * kStepBlocks + t;
      const int base = wb.logical(lb0 + vblk) * kDecodeBlock;
      n_valid[t] = vblk < nblk ? min(kDecodeBlock, ctx - base) : 0;
      hid0[t] = windowed ? max(0, p.sinks - base) : 0;
      hid1[t] = windowed ? wb.lo - base : 0;
      masked = masked || n_valid[t] < kDecodeBlock || hid0[t] < hid1[t];
      ks[t] = __shfl_sync(0xffffffffu, my_ks, vblk & 31);
      lv[t] = __shfl_sync(0xffffffffu, my_lv, vblk & 31);
    }
    auto hidden = [&](int t, int tok) {
      return tok >= n_valid[t] || (tok >= hid0[t] && tok < hid1[t]);
    };
    // Softmax of head quad of each N tile over its tokens grp and grp + 8 of
    // each block (log2 units).
    float w[NT][kStepBlocks][2];  // weights times their block's scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[kStepBlocks][2];
      float top = -CUDART_INF_F, top_o = -CUDART_INF_F;
#pragma unroll
      for (int t = 0; t < kStepBlocks; ++t) {
        const float c = ks[t] * cq[nt];
        x[t][0] = fmaf(s[nt][t][1], 0.0625f, s[nt][t][0]) * c;
        x[t][1] = fmaf(s[nt][t][3], 0.0625f, s[nt][t][2]) * c;
        if (masked) {
          if (hidden(t, grp)) x[t][0] = -CUDART_INF_F;
          if (hidden(t, grp + 8)) x[t][1] = -CUDART_INF_F;
        }
        float mx = fmaxf(x[t][0], x[t][1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        top = fmaxf(top, mx);
        top_o = fmaxf(top_o, mx + lv[t]);
      }
      // references that a maximum has outgrown move to it (from -inf, where
      // nothing was seen, to the first one)
      const bool grow = top > m[nt] + kSlackLog2 || top_o > mo[nt] + kSlackLog2;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? fmaxf(m[nt], top) : m[nt];
        const float mo_new = grow ? fmaxf(mo[nt], top_o) : mo[nt];
        l[nt] *= (m[nt] == m_new) ? 1.f : ex2(m[nt] - m_new);
        const float alpha = (mo[nt] == mo_new) ? 1.f : ex2(mo[nt] - mo_new);
        m[nt] = m_new;
        mo[nt] = mo_new;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          acc[nt / 2][u][nt % 2] *= alpha;
          acc[nt / 2][u][2 + nt % 2] *= alpha;
        }
      }
      // (nothing seen yet: finite references, every weight is 0)
      const float m_use = (m[nt] == -CUDART_INF_F) ? 0.f : m[nt];
      const float mo_use = ((mo[nt] == -CUDART_INF_F) ? 0.f : mo[nt]) - kTopLog2;
#pragma unroll
      for (int t = 0; t < kStepBlocks; ++t) {
        l[nt] += ex2(x[t][0] - m_use) + ex2(x[t][1] - m_use);
        const float off = lv[t] - mo_use;
        w[nt][t][0] = ex2(x[t][0] + off);
        w[nt][t][1] = ex2(x[t][1] + off);
      }
    }
    // rows grp: tokens grp (grp + 8), columns the heads of two S tiles;
    // transposed: tokens 2 q and 2 q + 1 (+ 8) of column grp
    uint32_t pb[NP][kStepBlocks][2];
#pragma unroll
    for (int np = 0; np < NP; ++np)
#pragma unroll
      for (int t = 0; t < kStepBlocks; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          pb[np][t][x] = movmatrix_trans(
              pack_f16x2(w[2 * np][t][x], 2 * np + 1 < NT ? w[(2 * np + 1) % NT][t][x] : 0.f));
    // O^T += V^T P^T: matrix mi of the transposing load holds tokens
    // 8 mi .. + 7 of the step's 32, 16 values of d as pairs
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t vrow = vb + (mi >> 1) * L::kBlockBytes;
    const int vtok = mr + 8 * (mi & 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // r[mi]: codes (tok, d), (tok, d + 1), (tok + 1, d), (tok + 1, d + 1)
      uint32_t r[4];
      ldmatrix_x4_trans(vrow + f8_off<D>(vtok, u), r[0], r[1], r[2], r[3]);
      if (masked) {
        // never let a stale or hidden slot reach the accumulator
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int tok = 8 * (x & 1) + 2 * quad;
          r[x] &= (hidden(x >> 1, tok) ? 0u : 0x0000FFFFu) |
                  (hidden(x >> 1, tok + 1) ? 0u : 0xFFFF0000u);
        }
      }
#pragma unroll
      for (int t = 0; t < kStepBlocks; ++t) {
        // (tok, d), (tok + 1, d), then the same of d + 1
        const uint32_t y0 = __byte_perm(r[2 * t], 0, 0x3120);
        const uint32_t y1 = __byte_perm(r[2 * t + 1], 0, 0x3120);
        const uint32_t a0 = e4m3x2_to_f16x2(y0), a1 = e4m3x2_hi_to_f16x2(y0);
        const uint32_t a2 = e4m3x2_to_f16x2(y1), a3 = e4m3x2_hi_to_f16x2(y1);
#pragma unroll
        for (int np = 0; np < NP; ++np)
          mma_m16n8k16_f16(acc[np][u], a0, a1, a2, a3, pb[np][t][0], pb[np][t][1]);
      }
    }
    __syncwarp();
    if (i + S < steps) {
      if (lane < 2 * kStepBlocks) fence_proxy_async_smem();
      issue(i + S);
    }
  }

  if (!ok) {
    // drain copies still in flight before the CTA releases its shared memory
    if (lane == 0)
      for (int i = max(0, issued - S); i < issued; ++i)
        mbar_drain(&full[i % S], (i / S) & 1, p.status);
    __syncwarp();
    return;
  }
  // write the partial state of every query head of the group
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float lt = l[nt];
    lt += __shfl_xor_sync(0xffffffffu, lt, 4);
    lt += __shfl_xor_sync(0xffffffffu, lt, 8);
    lt += __shfl_xor_sync(0xffffffffu, lt, 16);
    const int g = nt * 4 + quad;
    if (g >= G) continue;
    const size_t row = (part_row + g) * p.max_splits + split;
    if (!in_bounds(row, 1, part_rows, p.status)) continue;
    if (grp == 0) {
      p.ml_part[row * 2 + 0] = split_max(m[nt], lt);
      p.ml_part[row * 2 + 1] = lt;
    }
    // o back from its own reference to m's
    const float f = (mo[nt] == -CUDART_INF_F) ? 0.f : exp2f(mo[nt] - m[nt] - kTopLog2);
    float2 *orow = reinterpret_cast<float2 *>(p.o_part + row * D);
#pragma unroll
    for (int u = 0; u < U; ++u)
      orow[u * 8 + grp] = make_float2(acc[nt / 2][u][nt % 2] * f, acc[nt / 2][u][2 + nt % 2] * f);
  }
}

template <int D, int NT>
static cudaError_t launch_decode_fp8_t(const CUtensorMap &tk, const CUtensorMap &tv,
                                       const DecodeParams &p, const CacheScales &sc,
                                       cudaStream_t stream) {
  using L = DecodeF8Layout<D>;
  auto kern = decode_fp8_split_kernel<D, NT>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = allow_smem(kern, L::kSmemAlloc, smem_set);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.max_splits, p.Hkv, p.batch), 32, L::kSmemAlloc, stream>>>(tk, tv, p, sc);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_decode_combine(p, D, stream) : e;
}

cudaError_t launch_decode_fp8(const CUtensorMap &tk, const CUtensorMap &tv, const DecodeParams &p,
                              const CacheScales &sc, int d, cudaStream_t stream) {
  const int nt = p.group <= 4 ? 1 : p.group <= 8 ? 2 : 4;  // N tiles of four heads
  if (d == 64) return nt == 1   ? launch_decode_fp8_t<64, 1>(tk, tv, p, sc, stream)
                      : nt == 2 ? launch_decode_fp8_t<64, 2>(tk, tv, p, sc, stream)
                                : launch_decode_fp8_t<64, 4>(tk, tv, p, sc, stream);
  return nt == 1   ? launch_decode_fp8_t<128, 1>(tk, tv, p, sc, stream)
         : nt == 2 ? launch_decode_fp8_t<128, 2>(tk, tv, p, sc, stream)
                   : launch_decode_fp8_t<128, 4>(tk, tv, p, sc, stream);
}

}  // namespace fa
