// decode_range.cuh - one warp's pass over a range of a sequence's keys in a bf16
// paged cache (decode.cu says how), shared by the decode kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "checks.cuh"
#include "decode_common.cuh"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {

// A warp's ring of STAGES blocks.
template <int D, int STAGES = kDecodeStages>
struct DecodeLayout {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kDecodeBlock * 128;   // 16 tokens x 64 bf16
  static constexpr int kBlockBytes = kChunks * kChunkBytes;  // one KV head of one block
  static constexpr int kStageBytes = 2 * kBlockBytes;        // K then V
  static constexpr int kBar = STAGES * kStageBytes;
  static constexpr int kMisc = kBar + STAGES * 8;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kSmemAlloc = kBytes + 1024;
};

// Byte offset of element (token, col) of a [16 x D] block staged with
// 128-byte swizzle as D/64 chunks of [16 rows][128 B].
__device__ __forceinline__ uint32_t swz_off(int token, int col) {
  const int chunk = col >> 6;
  const int unit = (col & 63) >> 3;  // 16-byte unit inside the 128-byte row
  return chunk * (kDecodeBlock * 128) + token * 128 + ((unit ^ (token & 7)) << 4);
}

// Keep the bf16 halves of x whose token is not hidden.
__device__ __forceinline__ uint32_t keep_tokens(uint32_t x, bool hide_lo, bool hide_hi) {
  return x & ((hide_lo ? 0u : 0x0000FFFFu) | (hide_hi ? 0u : 0xFFFF0000u));
}

// One warp's pass over a range of keys: the unnormalised O^T accumulator of
// the group's query heads (m16n8 accumulator layout: rows are the head
// dimension, columns the heads), the running maximum of each head (log2
// units) and each lane's share of the row sums.
template <int D, int NT>
struct WarpRange {
  float acc[NT][D / 16][4];
  float mcol[NT][2], lcol[NT][2];
};

constexpr int kRangeOk = 0, kRangeBadBlock = 1, kRangeFailed = 2;

// A converged warp streams keys [t0, t1) (at most kDecodeMaxSplitTokens) of
// sequence b and KV head kvh through its own ring of TMA stages at `smem`
// (DecodeLayout<D, STAGES>::kBytes, 1024-byte aligned) and leaves its state in st.
// Lane i holds the physical id of logical block t0 / 16 + i in my_blk (-1
// when it could not be read).  WIN: t0 and t1 count the keys of the blocks
// that the windowed query reads (wb), and the hidden ones among them are
// masked like those past the context of ctx keys.  Returns kRangeBadBlock (nothing loaded,
// status raised) when a block id of the range is outside the pool,
// kRangeFailed when a wait gave up (copies in flight are drained before it
// returns).
template <int D, int NT, bool WIN, int STAGES = kDecodeStages>
__device__ __forceinline__ int decode_range(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                            const DecodeParams &p, int b, int kvh, int t0, int t1,
                                            int my_blk, uint8_t *smem, WarpRange<D, NT> &st,
                                            const WindowBlocks &wb, int ctx) {
  using L = DecodeLayout<D, STAGES>;
  constexpr int S = STAGES;
  constexpr int KC = D / 16;  // 16-wide k chunks of the head dimension
  const int lane = threadIdx.x & 31;
  const int nblk = (t1 - t0 + kDecodeBlock - 1) / kDecodeBlock;  // <= 32
  const int G = p.group;

  const bool bad = lane < nblk && (my_blk < 0 || my_blk >= p.num_blocks);
  const size_t part_row = static_cast<size_t>(b) * p.H + static_cast<size_t>(kvh) * G;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) raise_status(p.status, FA_DEV_BAD_BLOCK);
    return kRangeBadBlock;
  }

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

  auto issue = [&](int st, int phys) {
    uint8_t *dst = smem + st * L::kStageBytes;
    mbar_arrive_expect_tx(&full[st], L::kStageBytes);
#pragma unroll
    for (int c = 0; c < L::kChunks; ++c) {
      tma_load_3d(dst + c * L::kChunkBytes, &tm_k, &full[st], c * 64, kvh, phys * kDecodeBlock);
      tma_load_3d(dst + L::kBlockBytes + c * L::kChunkBytes, &tm_v, &full[st], c * 64, kvh,
                  phys * kDecodeBlock);
    }
  };
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int phys = __shfl_sync(0xffffffffu, my_blk, i);
    if (lane == 0 && i < nblk) issue(i, phys);
  }

  // Q^T fragments (B operand): column n = query head kvh*G + n of the group.
  uint32_t qf[NT][KC][2];
  const int quad = lane & 3;
  const int grp = lane >> 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + grp;
    const bool valid =
        n < G && in_bounds((part_row + n) * D, D, static_cast<size_t>(p.batch) * p.H * D, p.status);
    const uint32_t *qrow = reinterpret_cast<const uint32_t *>(
        static_cast<const uint16_t *>(p.q) + (part_row + (valid ? n : 0)) * D);
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      qf[nt][kc][0] = valid ? qrow[(kc * 16 + 2 * quad) >> 1] : 0u;
      qf[nt][kc][1] = valid ? qrow[(kc * 16 + 8 + 2 * quad) >> 1] : 0u;
    }
  }

  float (&acc)[NT][KC][4] = st.acc;
  float (&mcol)[NT][2] = st.mcol;
  float (&lcol)[NT][2] = st.lcol;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < KC; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
    mcol[nt][0] = mcol[nt][1] = -CUDART_INF_F;
    lcol[nt][0] = lcol[nt][1] = 0.f;
  }
  const float sl2 = p.scale_log2;

  // ldmatrix row addresses: lane supplies row (lane & 7) of matrix (lane >> 3).
  const int mi = lane >> 3;
  const int mr = lane & 7;
  // K (non-transposed A operand): matrix mi covers tokens 8*(mi&1).., cols 8*(mi>>1)..
  const int k_tok = mr + 8 * (mi & 1);
  const int k_col = 8 * (mi >> 1);
  // V^T (transposed load): matrix mi covers tokens 8*(mi>>1).., cols 8*(mi&1)..
  const int v_tok = mr + 8 * (mi >> 1);
  const int v_col = 8 * (mi & 1);

  bool ok = true;
  for (int i = 0; i < nblk; ++i) {
    const int st = i % S;
    ok = mbar_wait(&full[st], (i / S) & 1, abort_flag, p.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t kb = smem_u32(smem + st * L::kStageBytes);
    const uint32_t vb = kb + L::kBlockBytes;
    const int base = WIN ? wb.logical(t0 / kDecodeBlock + i) * kDecodeBlock : t0 + i * kDecodeBlock;
    const int n_valid = min(kDecodeBlock, (WIN ? ctx : t1) - base);
    // windowed: tokens [hid0, hid1) of the block lie between sinks and window
    const int hid0 = WIN ? max(0, p.sinks - base) : 0;
    const int hid1 = WIN ? wb.lo - base : 0;
    const bool masked = n_valid < kDecodeBlock || (WIN && hid0 < hid1);
    auto hidden = [&](int tok) { return tok >= n_valid || (WIN && tok >= hid0 && tok < hid1); };

    // S^T = K Q^T
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
      uint32_t a0, a1, a2, a3;
      ldmatrix_x4(kb + swz_off(k_tok, kc * 16 + k_col), a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_m16n8k16_bf16(s[nt], a0, a1, a2, a3, qf[nt][kc][0], qf[nt][kc][1]);
    }
    // rows of the accumulator are tokens grp and grp + 8
    if (masked) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (hidden(grp)) s[nt][0] = s[nt][1] = -CUDART_INF_F;
        if (hidden(grp + 8)) s[nt][2] = s[nt][3] = -CUDART_INF_F;
      }
    }
    // column-wise (per query head) online softmax
    uint32_t pb0[NT], pb1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[4];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float mx = fmaxf(s[nt][cc], s[nt][2 + cc]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float m_new = fmaxf(mcol[nt][cc], mx * sl2);
        const float m_use = (m_new == -CUDART_INF_F) ? 0.f : m_new;
        const float alpha = ex2(mcol[nt][cc] - m_use);
        pv[cc] = ex2(fmaf(s[nt][cc], sl2, -m_use));
        pv[2 + cc] = ex2(fmaf(s[nt][2 + cc], sl2, -m_use));
        lcol[nt][cc] = lcol[nt][cc] * alpha + pv[cc] + pv[2 + cc];
        mcol[nt][cc] = m_new;
#pragma unroll
        for (int mt = 0; mt < KC; ++mt) {
          acc[nt][mt][cc] *= alpha;
          acc[nt][mt][2 + cc] *= alpha;
        }
      }
      pb0[nt] = movmatrix_trans(pack_bf16x2(pv[0], pv[1]));
      pb1[nt] = movmatrix_trans(pack_bf16x2(pv[2], pv[3]));
    }
    // O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < KC; ++mt) {
      uint32_t a0, a1, a2, a3;
      ldmatrix_x4_trans(vb + swz_off(v_tok, mt * 16 + v_col), a0, a1, a2, a3);
      if (masked) {
        // never let a stale slot past the context, or a hidden one, reach the accumulator
        a0 = keep_tokens(a0, hidden(2 * quad), hidden(2 * quad + 1));
        a1 = keep_tokens(a1, hidden(2 * quad), hidden(2 * quad + 1));
        a2 = keep_tokens(a2, hidden(8 + 2 * quad), hidden(9 + 2 * quad));
        a3 = keep_tokens(a3, hidden(8 + 2 * quad), hidden(9 + 2 * quad));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_m16n8k16_bf16(acc[nt][mt], a0, a1, a2, a3, pb0[nt], pb1[nt]);
    }
    __syncwarp();
    const int nxt = i + S;
    const int phys = __shfl_sync(0xffffffffu, my_blk, nxt & 31);
    if (lane == 0 && nxt < nblk) {
      fence_proxy_async_smem();
      issue(st, phys);
    }
  }

  if (ok) return kRangeOk;
    // drain copies still in flight before the CTA releases its shared memory
    if (lane == 0) {
      for (int i = 0; i < min(nblk, S); ++i) {
        const uint64_t tstart = globaltimer_ns();
        // the last load issued into stage i has phase ((last) / S) & 1
        int last = i;
        while (last + S < nblk) last += S;
        while (!mbar_try_wait(&full[i], (last / S) & 1)) {
          if (globaltimer_ns() - tstart > kWaitLimitNs) break;
        }
      }
    }
    __syncwarp();
  return kRangeFailed;
}

// Writes the partial states of the group's query heads, rows part_row, ... of
// [batch * H, max_splits], for split `split`.
template <int D, int NT>
__device__ __forceinline__ void store_range(const DecodeParams &p, size_t part_row, int split,
                                            const WarpRange<D, NT> &st) {
  constexpr int KC = D / 16;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const size_t part_rows = static_cast<size_t>(p.batch) * p.H * p.max_splits;
  const int quad = lane & 3;
  const int grp = lane >> 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
      float lt = st.lcol[nt][cc];
      lt += __shfl_xor_sync(0xffffffffu, lt, 4);
      lt += __shfl_xor_sync(0xffffffffu, lt, 8);
      lt += __shfl_xor_sync(0xffffffffu, lt, 16);
      const int g = nt * 8 + 2 * quad + cc;
      if (g < G) {
        const size_t row = (part_row + g) * p.max_splits + split;
        if (!in_bounds(row, 1, part_rows, p.status)) continue;
        if (grp == 0) {
          p.ml_part[row * 2 + 0] = split_max(st.mcol[nt][cc], lt);
          p.ml_part[row * 2 + 1] = lt;
        }
        float *orow = p.o_part + row * D;
#pragma unroll
        for (int mt = 0; mt < KC; ++mt) {
          orow[mt * 16 + grp] = st.acc[nt][mt][cc];
          orow[mt * 16 + 8 + grp] = st.acc[nt][mt][2 + cc];
        }
      }
    }
  }
}

// Leaves a neutral partial state, so that the combine ignores the split.
template <int D>
__device__ __forceinline__ void store_neutral(const DecodeParams &p, size_t part_row, int split) {
  const int lane = threadIdx.x & 31;
  const size_t part_rows = static_cast<size_t>(p.batch) * p.H * p.max_splits;
  for (int g = 0; g < p.group; ++g) {
    const size_t row = (part_row + g) * p.max_splits + split;
    if (!in_bounds(row, 1, part_rows, p.status)) continue;
    for (int c = lane; c < D; c += 32) p.o_part[row * D + c] = 0.f;
    if (lane == 0) {
      p.ml_part[row * 2 + 0] = -CUDART_INF_F;
      p.ml_part[row * 2 + 1] = 0.f;
    }
  }
}

}  // namespace fa
