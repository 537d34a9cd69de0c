// prefix.cu - single tokens over a prefix that the sequences of a group share,
// for sm_103a: the shared keys' part, and the combine with the own keys'
// (decode.cu).
//
// With one KV head's query heads of all sequences of a group as rows, n G
// rows meet the same keys, and what decode.cu reads n times is a matrix
// product over keys that are read once: S = Q K^T, p = 2^(s - m), o += p V with
// the running maximum and sums of the prefill kernel (prefill_kernel.cuh), and
// no row has a causal limit of its own but its context length.
//
// prefix_kernel: one CTA per SM, persistent.  The work is a line of key tiles
// (128 keys), group after group, KV head after KV head, pair of row tiles
// after pair; a CTA takes an equal stretch of it, that is one or more runs of
// key tiles over one pair of row tiles each, and leaves a partial state (m, l,
// o) for every row and run.
//   warps 0-7  softmax, one row a thread, two tiles of 128 rows
//   warp 8     MMA issuer: S_i = Q_i K^T, O_i += P_i V (tcgen05, TMEM)
//   warp 9     TMA of Q (a box of sequences x heads) and, block by block, K
//   warp 10    TMA of V
// A tile's rows are whole sequences, 128 / G of them with G heads each.
//
// prefix_combine_kernel: W warps per (sequence, query head) merge the partial
// states of its own keys and of the shared ones, as decode_combine_kernel.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "decode_common.cuh"
#include "fa_internal.h"
#include "launch.h"
#include "prefix_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kPrefixThreads = 352;
constexpr float kPrefixRescaleLog2 = 8.f;  // as the prefill kernel's

template <int D>
struct PrefixLayout {
  static constexpr int kChunks = D / 64;             // 64 bf16 columns, 128-byte rows
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;   // of K, and of V
  static constexpr int kQ = 0;                       // two tiles
  static constexpr int kK = 2 * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kOut = kV + kStages * kTileBytes;  // 32 rows x 128 bytes a softmax warp
  static constexpr int kBar = kOut + 8 * 32 * 128;
  // q_full, q_free, drain, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_done[2]
  static constexpr int kNumBars = 3 + 4 * kStages + 6;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kSmemAlloc = kBytes + 1024;
  static_assert(kSmemAlloc <= 232448, "prefix shared memory exceeds 227 KiB");
  static constexpr int kTmemO = 256;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using L = PrefixLayout<D>;
  constexpr int S = L::kStages;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  unsigned int *status = p.own.status;
  const int G = p.own.group;
  pdl_launch_dependents();

  // ---------------------------------------------------------------- work
  long long total;
  const int per = prefix_share(p, blockIdx.x == 0 && warp == 0, total);
  if (static_cast<long long>(blockIdx.x) * per >= total) return;  // the whole CTA
  int at = blockIdx.x * per;
  const int stop = static_cast<int>(min(total, static_cast<long long>(at) + per));

  // A run: key tiles [j0, j0 + n) of KV head kvh for the row tiles of the
  // sequences from seq0 on; rows[i] of tile i belong to the group.
  int kvh, j0, n, seq0, slot, lead, whole;
  int rows[2];
  auto load_run = [&]() {
    PrefixGroup g;
    long long start = 0;
    prefix_find(p, at, false, g, start);
    const int rel = at - static_cast<int>(start);
    const int unit = rel / g.tiles;
    j0 = rel - unit * g.tiles;
    n = min(g.tiles - j0, stop - at);
    kvh = unit / g.pairs;
    lead = g.a;
    whole = g.whole;
    seq0 = g.a + (unit - kvh * g.pairs) * 2 * p.seqs_per_tile;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      rows[i] = max(0, min(p.seqs_per_tile, g.e - seq0 - i * p.seqs_per_tile)) * G;
    slot = at / per - (at - j0) / per;
  };
  // k tiles, key tiles of tile 1 and runs so far, for the barriers' phases
  int tiles0 = 0, tiles1 = 0, turn = 0, turn1 = 0;
  auto next_run = [&]() -> bool {
    at += n;
    tiles0 += n;
    ++turn;
    if (rows[1] > 0) {
      tiles1 += n;
      ++turn1;
    }
    if (at >= stop) return false;
    load_run();
    return true;
  };
  load_run();

  // ------------------------------------------------------- shared memory
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::kBar);
  uint64_t *q_free = q_full + 1;
  uint64_t *drain = q_full + 2;
  uint64_t *k_full = q_full + 3;
  uint64_t *k_empty = k_full + S;
  uint64_t *v_full = k_empty + S;
  uint64_t *v_empty = v_full + S;
  uint64_t *s_full = v_empty + S;
  uint64_t *p_full = s_full + 2;
  uint64_t *o_done = p_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);

  if (warp == 9 && lane == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(drain, 1);
    for (int s = 0; s < S; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 9 || warp == 10) {
    // ------------------------------------------------------ copies
    // Lanes 0..7 hold a tile's 8 block ids; the ids of 4 tiles come with one
    // load, 4 tiles before they are needed.  A block past the prefix or outside
    // the pool is not copied: its rows are made 0 (what a stage held before
    // may be infinite, and 0 times that is NaN).
    constexpr int kTileBlocks = kPrefixTileKeys / kDecodeBlock;
    constexpr int kIdTiles = 32 / kTileBlocks;
    constexpr int kBlockRows = kDecodeBlock * 128;  // bytes of a block in one chunk
    const bool is_k = warp == 9;
    const CUtensorMap *map = is_k ? &tm_k : &tm_v;
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    uint8_t *stage0 = smem + (is_k ? L::kK : L::kV);
    int issued = 0, q_issued = 0;
    bool ok = true;
    do {
      auto fetch = [&](int w) -> int {
        const int j = w + lane / kTileBlocks;
        const int blk = (j0 + j) * kTileBlocks + lane % kTileBlocks;
        if (j >= n || blk * kDecodeBlock >= whole) return -1;
        const int id = checked_load(
            p.own.block_table, static_cast<size_t>(lead) * p.own.max_blocks_per_seq + blk,
            static_cast<size_t>(p.own.batch) * p.own.max_blocks_per_seq, status);
        if (id >= 0 && id < p.own.num_blocks) return id;
        if (is_k) raise_status(status, FA_DEV_BAD_BLOCK);
        return -1;
      };
      int cur = fetch(0), nxt = fetch(kIdTiles);
      auto load = [&](int j) -> bool {
        if (j > 0 && j % kIdTiles == 0) {
          cur = nxt;
          nxt = fetch(j + kIdTiles);
        }
        const int x = tiles0 + j, st = x % S;
        if (x >= S && !mbar_wait_warp(&empty[st], ((x / S) - 1) & 1, abort_flag, status)) return false;
        uint8_t *stage = stage0 + st * L::kTileBytes;
        // lane = block * chunks + chunk issues that copy
        const int id = __shfl_sync(0xffffffffu, cur,
                                   (j % kIdTiles) * kTileBlocks + (lane / L::kChunks) % kTileBlocks);
        uint8_t *dst = stage + (lane % L::kChunks) * L::kChunkBytes + lane / L::kChunks * kBlockRows;
        const bool mine = lane < kTileBlocks * L::kChunks;
        const unsigned live = __ballot_sync(0xffffffffu, mine && id >= 0);
        if (mine && id < 0) {
          for (int t = 0; t < kBlockRows / 16; ++t)
            reinterpret_cast<uint4 *>(dst)[t] = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(live) * kBlockRows);
        __syncwarp();
        if (mine && id >= 0)
          tma_load_3d(dst, map, &full[st], (lane % L::kChunks) * 64, kvh, id * kDecodeBlock);
        issued = x + 1;
        return true;
      };
      ok = load(0);
      if (is_k && ok) {
        // Q's place is free once the last run's S products have read it
        if (turn > 0) ok = mbar_wait_warp(q_free, (turn - 1) & 1, abort_flag, status);
        if (ok && lane == 0) {
          const int tiles = rows[1] > 0 ? 2 : 1;
          mbar_arrive_expect_tx(q_full, tiles * p.seqs_per_tile * G * 128 * L::kChunks);
          for (int i = 0; i < tiles; ++i)
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(smem + L::kQ + i * L::kTileBytes + c * L::kChunkBytes, &tm_q, q_full, c * 64,
                          kvh * G, seq0 + i * p.seqs_per_tile);
        }
        if (ok) q_issued = turn + 1;
      }
      for (int j = 1; ok && j < n; ++j) ok = load(j);
    } while (ok && next_run());
    if (lane == 0) {  // no copy outlives the CTA
      if (is_k && q_issued > 0) mbar_drain(q_full, (q_issued - 1) & 1, status);
      for (int x = max(0, issued - S); x < issued; ++x) mbar_drain(&full[x % S], (x / S) & 1, status);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------ MMA issuer
    constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
    const uint32_t q_base = smem_u32(smem + L::kQ);
    const uint32_t k_base = smem_u32(smem + L::kK);
    const uint32_t v_base = smem_u32(smem + L::kV);
    auto issue_s = [&](int i, int st) {
      if (elect_one()) {
        const uint64_t a0 = sdesc_swz<128>(q_base + i * L::kTileBytes, 16, 1024);
        const uint64_t b0 = sdesc_swz<128>(k_base + st * L::kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>((kk / 4 * L::kChunkBytes + kk % 4 * 32) >> 4);
          mma_ss(tmem + i * 128, a0 + off, b0 + off, kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[i]);
      }
      __syncwarp();
    };
    auto issue_o = [&](int i, int st, int j) {
      if (elect_one()) {
        const uint64_t b0 = sdesc_swz<128>(v_base + st * L::kTileBytes, L::kChunkBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + L::kTmemO + i * D, tmem + i * 128 + kk * 8,
                 b0 + static_cast<uint64_t>((kk * 16 * 128) >> 4), kIdescO,
                 (j > 0 || kk > 0) ? 1u : 0u);
        if (j == n - 1) mma_commit(&o_done[i]);
      }
      __syncwarp();
    };
    // Per key tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1), as the prefill kernel.
    bool ok = true;
    do {
      const bool two = rows[1] > 0;
      auto wait_k = [&](int x) {
        const bool done = mbar_wait_warp(&k_full[x % S], (x / S) & 1, abort_flag, status);
        tc_fence_after();
        return done;
      };
      ok = mbar_wait_warp(q_full, turn & 1, abort_flag, status) && wait_k(tiles0);
      if (!ok) break;
      issue_s(0, tiles0 % S);
      if (two) issue_s(1, tiles0 % S);
      mma_commit_elect(&k_empty[tiles0 % S]);
      if (n == 1) mma_commit_elect(q_free);
      int j = 0;
      for (; j < n; ++j) {
        const int x = tiles0 + j;
        if (!mbar_wait_warp(&v_full[x % S], (x / S) & 1, abort_flag, status)) break;
        if (!mbar_wait_warp(&p_full[0], x & 1, abort_flag, status)) break;
        tc_fence_after();
        issue_o(0, x % S, j);
        if (j + 1 < n) {
          if (!wait_k(x + 1)) break;
          issue_s(0, (x + 1) % S);
        }
        if (two) {
          if (!mbar_wait_warp(&p_full[1], (tiles1 + j) & 1, abort_flag, status)) break;
          tc_fence_after();
          issue_o(1, x % S, j);
        }
        mma_commit_elect(&v_empty[x % S]);
        if (j + 1 < n) {
          if (two) issue_s(1, (x + 1) % S);
          mma_commit_elect(&k_empty[(x + 1) % S]);
          if (j + 2 == n) mma_commit_elect(q_free);  // the run's last S products are issued
        }
      }
      ok = j == n;
    } while (ok && next_run());
    // everything issued must finish before TMEM is released
    mma_commit_elect(drain);
    mbar_drain(drain, 0, status);
  } else {
    // ------------------------------------------------------ softmax
    const int i = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + i * 128 + lane_off;
    const uint32_t tO = tmem + L::kTmemO + i * D + lane_off;
    uint8_t *out_stage = smem + L::kOut + warp * 32 * 128;
    const float sl2 = p.own.scale_log2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    bool ok = true;
    do {
      if (rows[i] == 0) continue;
      const int t0 = i == 0 ? tiles0 : tiles1;
      // rows behind the group's last sequence take part in the products and are
      // not written; a warp of them alone only keeps the barriers going
      const bool live = row < rows[i];
      const bool warp_live = (warp & 3) * 32 < rows[i];
      const int seq = seq0 + i * p.seqs_per_tile + row / G;
      const int head = kvh * G + row % G;
      int limit = whole;
      if (live) limit = min(whole, prefix_ctx(p, seq, whole, false));
      float m_ref = -CUDART_INF_F, l = 0.f, l_exact = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = mbar_wait_warp(&s_full[i], (t0 + j) & 1, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          uint32_t sr[128];
          tmem_ld128_wait(tS, sr);
          const int nvis = limit - (j0 + j) * kPrefixTileKeys;
          if (__any_sync(0xffffffffu, nvis < kPrefixTileKeys)) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= nvis) sr[c] = 0xff800000u;  // -inf
          }
          auto f = [&](int c) { return __uint_as_float(sr[c]); };
          float mx0 = f(0), mx1 = f(1), mx2 = f(2), mx3 = f(3);
#pragma unroll
          for (int c = 4; c < 124; c += 8) {
            mx0 = fmax3(mx0, f(c), f(c + 1));
            mx1 = fmax3(mx1, f(c + 2), f(c + 3));
            mx2 = fmax3(mx2, f(c + 4), f(c + 5));
            mx3 = fmax3(mx3, f(c + 6), f(c + 7));
          }
          mx0 = fmax3(mx0, f(124), f(125));
          mx1 = fmax3(mx1, f(126), f(127));
          const float m_new = fmaxf(m_ref, fmax3(mx0, mx1, fmaxf(mx2, mx3)) * sl2);
          // the reference moves only when the maximum grows by more than 2^8
          // (p stays below that); false while nothing visible has been seen
          const bool grow = m_new > m_ref + kPrefixRescaleLog2;
          float alpha = 1.f;
          if (grow) {
            alpha = ex2(m_ref - m_new);  // 0 on the first visible tile
            m_ref = m_new;
          }
          const float m_use = (m_ref == -CUDART_INF_F) ? 0.f : m_ref;
          const float2 negm = make_float2(-m_use, -m_use);
          // l sums the bf16 weights that the product multiplies (o / l is a mean
          // with consistent weights), l_exact the fp32 ones (for the log-sum-exp)
          float2 rs0 = make_float2(0.f, 0.f), rs1 = rs0, re0 = rs0, re1 = rs0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const int e = half * 64 + 2 * c;
              const float2 x0 = ffma2(
                  make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl2x2, negm);
              const float2 x1 = ffma2(
                  make_float2(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])), sl2x2, negm);
              const float2 p0 = make_float2(ex2(x0.x), ex2(x0.y));
              const float2 p1 = make_float2(ex2(x1.x), ex2(x1.y));
              pk[c] = pack_bf16x2(p0.x, p0.y);
              pk[c + 1] = pack_bf16x2(p1.x, p1.y);
              re0 = fadd2(re0, p0);
              re1 = fadd2(re1, p1);
              add_bf16x2_to(rs0, pk[c]);
              add_bf16x2_to(rs1, pk[c + 1]);
            }
            tmem_st32(tS + half * 32, pk);
          }
          const float2 rs = fadd2(rs0, rs1), re = fadd2(re0, re1);
          l = l * alpha + (rs.x + rs.y);
          l_exact = l_exact * alpha + (re.x + re.y);
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_wait(tO + c * 32, o);
#pragma unroll
              for (int t = 0; t < 32; t += 2) {
                const float2 v =
                    fmul2(make_float2(__uint_as_float(o[t]), __uint_as_float(o[t + 1])), a2);
                o[t] = __float_as_uint(v.x);
                o[t + 1] = __float_as_uint(v.y);
              }
              tmem_st32(tO + c * 32, o);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[i]);
      }
      // ---------------------------------------------------- partial state
      if (ok) ok = mbar_wait_warp(&o_done[i], (i == 0 ? turn : turn1) & 1, abort_flag, status);
      if (!ok || !warp_live) continue;
      tc_fence_after();
      const size_t n_rows = static_cast<size_t>(p.own.batch) * p.own.H * p.max_slots;
      const size_t mine = (static_cast<size_t>(seq) * p.own.H + head) * p.max_slots + slot;
      if (live && in_bounds(mine, 1, n_rows, status))
        p.pml_part[mine] = make_float4(split_max(m_ref, l), l, l_exact, 0.f);
      // 32 columns at a time: each thread's row through shared memory (16-byte
      // unit u of row r at u ^ (r % 8)), then 8 lanes write a row's 128 bytes
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32_wait(tO + c * 32, o);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<uint4 *>(out_stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
              make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        __syncwarp();
#pragma unroll
        for (int r4 = 0; r4 < 8; ++r4) {
          const int r = r4 * 4 + lane / 8, u = lane % 8;
          const uint4 v =
              *reinterpret_cast<const uint4 *>(out_stage + r * 128 + ((u ^ (r & 7)) << 4));
          const size_t to = __shfl_sync(0xffffffffu, mine, r) * D + c * 32 + u * 4;
          if ((warp & 3) * 32 + r < rows[i] && in_bounds(to, 4, n_rows * D, status))
            *reinterpret_cast<uint4 *>(p.po_part + to) = v;
        }
        __syncwarp();
      }
      // the next run's products overwrite O once this warp's next p_full arrives
      tc_fence_before();
    } while (ok && next_run());
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ combine

namespace {

constexpr int kPrefixCombineWarps = 4;

}  // namespace

// A CTA per (sequence, query head).  Its warps find the maximum of all states
// together, take every fourth state each, and are added through shared memory.
template <int D>
__global__ void __launch_bounds__(32 * kPrefixCombineWarps)
    prefix_combine_kernel(const PrefixParams p) {
  constexpr int W = kPrefixCombineWarps;
  constexpr int E = D / 32;
  __shared__ float s_acc[W][D];
  __shared__ float s_l[W], s_lx[W], s_m[W];
  const DecodeParams &o = p.own;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / o.H, h = blockIdx.x - b * o.H;
  // the plan of the shared keys, and this row's place in it
  PrefixGroup g{};
  long long start = 0, total;
  const int per = prefix_share(p, false, total);
  const bool grouped = prefix_find(p, b, true, g, start) && total > 0;
  const int whole = grouped ? g.whole : 0;
  const int ctx = prefix_ctx(p, b, whole, blockIdx.x % o.H == 0 && threadIdx.x == 0);
  int shared = 0;  // partial states over shared keys
  if (whole > 0 && ctx > 0) {
    const int first = static_cast<int>(start) +
                      (h / o.group * g.pairs + (b - g.a) / (2 * p.seqs_per_tile)) * g.tiles;
    shared = (first + g.tiles - 1) / per - first / per + 1;
  }
  const int own = (max(0, ctx - whole) + o.split_tokens - 1) / o.split_tokens;
  const int ns = own + shared;
  pdl_wait_primary();  // both kernels' partial states are complete from here on
  const bool publisher = blockIdx.x == 0 && threadIdx.x == 0;
  const unsigned int call_bits = publisher ? call_status_bits(o.call) : 0u;
  // this kernel's own (checked-build) index errors go to the device word only
  unsigned int *status = o.dev_status;
  const size_t n_own = static_cast<size_t>(o.batch) * o.H * o.max_splits;
  const size_t n_shared = static_cast<size_t>(o.batch) * o.H * p.max_slots;
  const size_t own0 = static_cast<size_t>(blockIdx.x) * o.max_splits;
  const size_t shared0 = static_cast<size_t>(blockIdx.x) * p.max_slots;
  // (m, l, l_exact) of state i
  auto state = [&](int i) -> float3 {
    if (i < own) {
      if (!in_bounds(own0 + i, 1, n_own, status)) return make_float3(-CUDART_INF_F, 0.f, 0.f);
      const float2 x = reinterpret_cast<const float2 *>(o.ml_part)[own0 + i];
      return make_float3(x.x, x.y, x.y);
    }
    if (!in_bounds(shared0 + i - own, 1, n_shared, status))
      return make_float3(-CUDART_INF_F, 0.f, 0.f);
    const float4 x = p.pml_part[shared0 + i - own];
    return make_float3(x.x, x.y, x.z);
  };
  float M = -CUDART_INF_F;
  for (int i = threadIdx.x; i < ns; i += 32 * W) M = fmaxf(M, state(i).x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w]);

  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float L = 0.f, Lx = 0.f;
  if (M != -CUDART_INF_F) {
    constexpr int U = 4;
    for (int i0 = warp; i0 < ns; i0 += U * W) {
      float3 st[U];
      float v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * W;
        st[u] = i < ns ? state(i) : make_float3(-CUDART_INF_F, 0.f, 0.f);
        const size_t row = i < own ? own0 + i : shared0 + i - own;
        const float *src = (i < own ? o.o_part : p.po_part) + row * D + lane * E;
        const bool there = i < ns && in_bounds(row, 1, i < own ? n_own : n_shared, status);
        if constexpr (E == 4) {
          const float4 x = there ? *reinterpret_cast<const float4 *>(src) : make_float4(0, 0, 0, 0);
          v[u][0] = x.x;
          v[u][1 % E] = x.y;
          v[u][2 % E] = x.z;
          v[u][3 % E] = x.w;
        } else {
          const float2 x = there ? *reinterpret_cast<const float2 *>(src) : make_float2(0, 0);
          v[u][0] = x.x;
          v[u][1 % E] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // an empty state is passed over, whatever its o holds
        const bool live = st[u].x != -CUDART_INF_F;
        const float w = ex2(st[u].x - M);
        L = live ? fmaf(w, st[u].y, L) : L;
        Lx = live ? fmaf(w, st[u].z, Lx) : Lx;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = live ? fmaf(w, v[u][e], acc[e]) : acc[e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    s_l[warp] = L;
    s_lx[warp] = Lx;
  }
  __syncthreads();
  if (warp != 0) return;
  L = Lx = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    L += s_l[w];
    Lx += s_lx[w];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += s_acc[w][lane * E + e];
    acc[e] = t;
  }
  const float inv = (L == 0.f) ? 0.f : 1.f / L;
  const size_t at = static_cast<size_t>(blockIdx.x) * D + lane * E;
  uint16_t *dst = static_cast<uint16_t *>(o.out) + at;
  if (in_bounds(at, E, static_cast<size_t>(o.batch) * o.H * D, status)) {
    if constexpr (E == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1 % E] * inv),
                                                   pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1 % E] * inv);
  }
  if (lane == 0 && o.lse != nullptr &&
      in_bounds(blockIdx.x, 1, static_cast<size_t>(o.batch) * o.H, status))
    o.lse[blockIdx.x] = (Lx == 0.f) ? -CUDART_INF_F : (M + __log2f(Lx)) * 0.69314718055994530942f;
  if (publisher) publish_call_status(o.call, call_bits, o.dev_status);
}

// ------------------------------------------------------------------ launch

// a kernel launched as a programmatic dependent of the one before it
template <typename Kernel, typename... Args>
static cudaError_t launch_dependent(Kernel kern, dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_decode_own(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                              int d, cudaStream_t stream);

template <int D>
static cudaError_t launch_prefix_d(const CUtensorMap &tq, const CUtensorMap &tk,
                                   const CUtensorMap &tv, const PrefixParams &p,
                                   cudaStream_t stream) {
  using L = PrefixLayout<D>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = allow_smem(prefix_kernel<D>, L::kSmemAlloc, smem_set);
  if (e != cudaSuccess) return e;
  prefix_kernel<D><<<p.ctas, kPrefixThreads, L::kSmemAlloc, stream>>>(tq, tk, tv, p);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_decode_own(tk, tv, p, D, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(prefix_combine_kernel<D>, dim3(static_cast<unsigned>(p.own.batch * p.own.H)),
                          dim3(32 * kPrefixCombineWarps), 0, stream, p);
}

cudaError_t launch_prefix(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const PrefixParams &p, int d, cudaStream_t stream) {
  return d == 64 ? launch_prefix_d<64>(tq, tk, tv, p, stream)
                 : launch_prefix_d<128>(tq, tk, tv, p, stream);
}

}  // namespace fa
