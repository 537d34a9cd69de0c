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
// prefix_kernel: one CTA per SM, persistent.  A CTA takes a KV head and a
// stretch of the call's key tiles (128 keys; prefix_internal.h), that is one or
// more runs of key tiles over one pair of row tiles each, and leaves a partial
// state (m, l, o) for every row and run.
//   warps 0-7  softmax, one row a thread, in two streams of four warps
//   warp 8     MMA issuer: S_i = Q_i K^T, O_i += P_i V (tcgen05, TMEM)
//   warp 9     TMA of Q (a box of sequences x heads) and, block by block, K
//   warp 10    TMA of V
// A tile's rows are whole sequences, 128 / G of them with G heads each.  With
// two row tiles stream i is row tile i over every key tile.  A run with one
// row tile would have one stream wait for its own products in turn; there
// stream i takes the key tiles j0 + i, j0 + i + 2, ... of the same rows, and the
// two states are merged as they leave TMEM.
//
// The own keys' CTAs, launched as programmatic dependents, run on the SMs that it
// leaves to them (prefix_plan) and on its own as its CTAs end.
//
// prefix_combine_kernel: one, two or four warps per (sequence, query head) merge
// the states of its own keys and of the shared ones, as decode_combine_kernel.
//
// What bounds it: with many rows the loop over key tiles, 3200 cycles each for
// two row tiles of d = 128, of which the products are 2048 (the rest the issuer
// waits, most for P: 394), 1024 rows and 16384 keys of 8 KV heads 85 us on 96
// SMs; with few rows the feed, 5.2 TB/s.  A call has 9 us before its first product
// (plan 3.4, block ids 1.3, ring 4) and 5 to 7 behind its last in the combine.
// 64 sequences over 8192 shared keys and 1 to 1024 of their own, 32 / 8 heads: 41 us
// where the ordinary call takes 216; 256 over 16384 and 1 to 512: 95 and 1537.
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
  static constexpr int kStates = kV + kStages * kTileBytes;  // 3 x 128 floats
  static constexpr int kBar = kStates + 3 * 128 * 4;
  // q_full, q_free, drain, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_done[2]
  static constexpr int kNumBars = 3 + 4 * kStages + 6;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kSave = kMisc + 16;  // 12 ints for each of 8 softmax warps
  static constexpr int kBytes = kSave + 8 * 12 * 4;
  static constexpr int kTmemO = 256;
};

// named_bar_sync of `count` threads that tells all of them whether any says so.
__device__ __forceinline__ bool named_bar_any(int id, int count, bool x) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, %3, q;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(static_cast<int>(x)), "r"(id), "r"(count)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0,
                                            int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(c4)
      : "memory");
}

// 8 floats to a 32-byte aligned address: a whole sector
__device__ __forceinline__ void store8(float *to, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The first of the sequences [a, e) that has all of `whole` shared keys, or else the
// longest, and how many of them it has (a converged warp).
__device__ __noinline__ int2 find_lead(const PrefixParams &p, int a, int e, int whole) {
  int lead = a, held = 0;
  for (int b0 = a; held < whole && b0 < e; b0 += 32) {
    const int b = b0 + static_cast<int>(threadIdx.x & 31);
    const int keys = b < e ? min(whole, prefix_ctx(p, b, whole, false)) : 0;
    const int most = __reduce_max_sync(0xffffffffu, keys);
    if (most > held) {
      held = most;
      lead = b0 + __ffs(__ballot_sync(0xffffffffu, keys == most)) - 1;
    }
  }
  return make_int2(lead, held);
}

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
  PrefixSums sums;
  PrefixGroup g{};
  const PrefixFirst first = prefix_first(p);
  prefix_walk<kPrefixNone>(p, 0, blockIdx.x == 0 && warp == 0, g, &sums, 0, &first);
  const PrefixPlan plan = prefix_plan(p, sums, first);
  const int my_team = blockIdx.x / p.team_heads;
  if (static_cast<long long>(my_team) * plan.per >= plan.total) return;  // the whole CTA
  int at = my_team * plan.per;
  int stop = static_cast<int>(min(static_cast<long long>(plan.total),
                                  static_cast<long long>(at) + plan.per));

  // A run: key tiles [j0, j0 + n) of KV head kvh for the row tiles of the
  // sequences from seq0 on; rows0 and rows1 of the two belong to the group.
  int kvh, j0, n, seq0, slot, whole;
  int rows0, rows1;
  auto load_run = [&](int team, int per, bool apart) {
    prefix_walk<kPrefixByTile>(p, at, false, g, nullptr, apart ? per : 0);
    const int rel = at - g.start;
    const int unit = rel / g.span;
    j0 = rel - unit * g.span;
    n = min(g.tiles - j0, stop - at);
    const int round = p.head_rounds > 1 ? unit / g.pairs : 0;
    kvh = round * p.team_heads + blockIdx.x - team * p.team_heads;
    whole = g.whole;
    seq0 = g.a + (unit - round * g.pairs) * 2 * p.seqs_per_tile;
    rows0 = min(p.seqs_per_tile, g.e - seq0) * G;
    rows1 = max(0, min(p.seqs_per_tile, g.e - seq0 - p.seqs_per_tile)) * G;
    slot = team - (at - j0) / per;
  };
  // (what later runs want of the plan waits in shared memory: registers are short)
  extern __shared__ __align__(1024) uint8_t smem[];
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMisc);
  // Key tiles and runs so far, and those of each stream, for the barriers' phases.
  int tiles = 0, turn = 0;
  int tiles_0 = 0, tiles_1 = 0, turns_0 = 0, turns_1 = 0;
  // key tiles of stream i in this run; those and its runs before
  auto stream_tiles = [&](int i) { return rows1 > 0 ? n : (n + 1 - i) / 2; };
  auto tiles_of = [&](int i) { return i ? tiles_1 : tiles_0; };
  auto turns_of = [&](int i) { return i ? turns_1 : turns_0; };
  auto next_run = [&]() -> bool {
    at += n;
    tiles += n;
    ++turn;
    tiles_0 += stream_tiles(0);
    tiles_1 += stream_tiles(1);
    ++turns_0;
    turns_1 += stream_tiles(1) > 0 ? 1 : 0;
    if (at >= stop) return false;
    load_run(misc[2], misc[3], false);
    return true;
  };
  load_run(my_team, plan.per, plan.apart);
  if (plan.apart) stop = at;  // no other run

  // ------------------------------------------------------- shared memory
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) raise_status(status, FA_DEV_SMEM_ALIGN);
    return;
  }
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
  volatile int *abort_flag = misc + 1;

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
    misc[2] = my_team;
    misc[3] = plan.per;
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
    // load, 4 tiles before they are needed.  A block past the held keys or outside
    // the pool is not copied: its rows are made 0 (what a stage held before
    // may be infinite, and 0 times that is NaN).
    constexpr int kTileBlocks = kPrefixTileKeys / kDecodeBlock;
    constexpr int kIdTiles = 32 / kTileBlocks;
    constexpr int kBlockBytes = kDecodeBlock * D * 2;
    const bool is_k = warp == 9;
    const CUtensorMap *map = is_k ? &tm_k : &tm_v;
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    uint8_t *stage0 = smem + (is_k ? L::kK : L::kV);
    int issued = 0, q_issued = 0;
    unsigned zeros = 0;  // stages whose place for this lane's block holds zeros
    bool ok = true;
    do {
      // The table row to read the blocks through: a sequence's row holds its own
      // keys' blocks and no more, so the first of the group that has all shared
      // keys, or the longest if none has (`held` of them; nobody sees the others).
      // That is mostly the first of all, whose ids come while its length is looked
      // at.  (-1: an id that no pool has, -2: no block wanted)
      int lead = g.a, held = whole;
      auto fetch = [&](int w) -> int {
        const int j = w + lane / kTileBlocks;
        const int blk = (j0 + j) * kTileBlocks + lane % kTileBlocks;
        if (j >= n || blk * kDecodeBlock >= held) return -2;
        return max(-1, checked_load(
            p.own.block_table, static_cast<size_t>(lead) * p.own.max_blocks_per_seq + blk,
            static_cast<size_t>(p.own.batch) * p.own.max_blocks_per_seq, status));
      };
      const int lead_ctx = prefix_ctx(p, lead, whole, false);
      int cur = fetch(0), nxt = fetch(kIdTiles);
      if (lead_ctx < whole) {
        const int2 found = find_lead(p, g.a, g.e, whole);
        lead = found.x;
        held = found.y;
        cur = fetch(0);
        nxt = fetch(kIdTiles);
      }
      auto load = [&](int j) -> bool {
        if (j > 0 && j % kIdTiles == 0) {
          cur = nxt;
          nxt = fetch(j + kIdTiles);
        }
        const int x = tiles + j, st = x % S;
        if (x >= S && !mbar_wait_warp(&empty[st], ((x / S) - 1) & 1, abort_flag, status)) return false;
        uint8_t *stage = stage0 + st * L::kTileBytes;
        // lane = block issues that copy
        const int id = __shfl_sync(0xffffffffu, cur, (j % kIdTiles) * kTileBlocks + lane % kTileBlocks);
        uint8_t *dst = stage + lane * kBlockBytes;
        const bool mine = lane < kTileBlocks, there = mine && id >= 0 && id < p.own.num_blocks;
        const unsigned live = __ballot_sync(0xffffffffu, there);
        if (mine && !there) {
          if (is_k && id != -2) raise_status(status, FA_DEV_BAD_BLOCK);
          if ((zeros >> st & 1u) == 0u) {
            for (int t = 0; t < kBlockBytes / 16; ++t)
              reinterpret_cast<uint4 *>(dst)[t] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
          zeros |= 1u << st;
        } else {
          zeros &= ~(1u << st);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(live) * kBlockBytes);
        __syncwarp();
        if (there)
          tma_load_5d(dst, map, &full[st], 0, 0, 0, id * (kDecodeBlock / 8), kvh);
        issued = x + 1;
        return true;
      };
      ok = load(0);
      if (is_k && ok) {
        // Q's place is free once the last run's S products have read it
        if (turn > 0) ok = mbar_wait_warp(q_free, (turn - 1) & 1, abort_flag, status);
        if (ok && lane == 0) {
          const int loads = rows1 > 0 ? 2 : 1;
          mbar_arrive_expect_tx(q_full, loads * p.seqs_per_tile * G * 128 * L::kChunks);
          for (int i = 0; i < loads; ++i)
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
    // S of stream i: row tile `tile` over the K stage st
    auto issue_s = [&](int i, int tile, int st) {
      if (elect_one()) {
        const uint64_t a0 = sdesc_swz<128>(q_base + tile * L::kTileBytes, 16, 1024);
        const uint64_t b0 = sdesc_swz<128>(k_base + st * L::kTileBytes, 16, L::kChunks * 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t a_off = static_cast<uint64_t>((kk / 4 * L::kChunkBytes + kk % 4 * 32) >> 4);
          const uint64_t b_off = static_cast<uint64_t>((kk / 4 * 1024 + kk % 4 * 32) >> 4);
          mma_ss(tmem + i * 128, a0 + a_off, b0 + b_off, kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[i]);
      }
      __syncwarp();
    };
    // O of stream i, its first or last key tile of the run
    auto issue_o = [&](int i, int st, bool first, bool last) {
      if (elect_one()) {
        const uint64_t b0 = sdesc_swz<128>(v_base + st * L::kTileBytes, 1024, L::kChunks * 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + L::kTmemO + i * D, tmem + i * 128 + kk * 8,
                 b0 + static_cast<uint64_t>((kk * kDecodeBlock * D * 2) >> 4), kIdescO,
                 (!first || kk > 0) ? 1u : 0u);
        if (last) mma_commit(&o_done[i]);
      }
      __syncwarp();
    };
    auto wait_k = [&](int x) {
      const bool done = mbar_wait_warp(&k_full[x % S], (x / S) & 1, abort_flag, status);
      tc_fence_after();
      return done;
    };
    // V(x) and P of stream i, its t-th key tile
    auto wait_p = [&](int i, int t) {
      const bool done = mbar_wait_warp(&p_full[i], (tiles_of(i) + t) & 1, abort_flag, status);
      tc_fence_after();
      return done;
    };
    auto wait_v = [&](int x) {
      return mbar_wait_warp(&v_full[x % S], (x / S) & 1, abort_flag, status);
    };
    bool ok = true;
    do {
      ok = mbar_wait_warp(q_full, turn & 1, abort_flag, status) && wait_k(tiles);
      if (!ok) break;
      int j = 0;
      if (rows1 > 0) {
        // Per key tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1), as the prefill kernel.
        issue_s(0, 0, tiles % S);
        issue_s(1, 1, tiles % S);
        mma_commit_elect(&k_empty[tiles % S]);
        if (n == 1) mma_commit_elect(q_free);
        for (; j < n; ++j) {
          const int x = tiles + j;
          if (!wait_v(x) || !wait_p(0, j)) break;
          issue_o(0, x % S, j == 0, j == n - 1);
          if (j + 1 < n) {
            if (!wait_k(x + 1)) break;
            issue_s(0, 0, (x + 1) % S);
          }
          if (!wait_p(1, j)) break;
          issue_o(1, x % S, j == 0, j == n - 1);
          mma_commit_elect(&v_empty[x % S]);
          if (j + 1 < n) {
            issue_s(1, 1, (x + 1) % S);
            mma_commit_elect(&k_empty[(x + 1) % S]);
            if (j + 2 == n) mma_commit_elect(q_free);  // the run's last S products are issued
          }
        }
      } else {
        // One row tile: key tile j is stream j % 2's, two of them under way.
        issue_s(0, 0, tiles % S);
        mma_commit_elect(&k_empty[tiles % S]);
        if (n > 1) {
          ok = wait_k(tiles + 1);
          if (!ok) break;
          issue_s(1, 0, (tiles + 1) % S);
          mma_commit_elect(&k_empty[(tiles + 1) % S]);
        }
        if (n <= 2) mma_commit_elect(q_free);
        for (; j < n; ++j) {
          const int x = tiles + j;
          if (!wait_v(x) || !wait_p(j & 1, j / 2)) break;
          issue_o(j & 1, x % S, j < 2, j + 2 >= n);
          mma_commit_elect(&v_empty[x % S]);
          if (j + 2 < n) {
            if (!wait_k(x + 2)) break;
            issue_s(j & 1, 0, (x + 2) % S);
            mma_commit_elect(&k_empty[(x + 2) % S]);
            if (j + 3 == n) mma_commit_elect(q_free);
          }
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
    const float sl2 = p.own.scale_log2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    volatile int *save = reinterpret_cast<volatile int *>(smem + L::kSave) + warp * 12;
    bool ok = true;
    do {
      bool two = rows1 > 0;
      const int count = stream_tiles(i);   // its key tiles: j, j + 1 or j + 2, ...
      const int step = two ? kPrefixTileKeys : 2 * kPrefixTileKeys;
      int tile = two ? i : 0;              // row tile
      int tile_rows = tile ? rows1 : rows0;
      // rows behind the group's last sequence take part in the products and are
      // not written; a warp of them alone only keeps the barriers going
      const bool warp_live = (warp & 3) * 32 < tile_rows;
      int nvis = whole;  // visible keys from the stream's next tile on
      if (row < tile_rows)
        nvis = min(whole, prefix_ctx(p, seq0 + tile * p.seqs_per_tile + row / G, whole, false));
      nvis -= (j0 + (two ? 0 : i)) * kPrefixTileKeys;
      unsigned phase = tiles_of(i) & 1;
      // what the loop does not need waits in shared memory (with it in registers
      // the scores do not fit)
      if (lane == 0) {
        const int keep[12] = {at, stop, n, seq0, slot, kvh, rows0, rows1, tiles_0, tiles_1, turns_0, turns_1};
#pragma unroll
        for (int x = 0; x < 12; ++x) save[x] = keep[x];
      }
      __syncwarp();
      float m_ref = -CUDART_INF_F, l = 0.f, l_exact = 0.f;
      for (int t = 0; t < count; ++t) {
        ok = mbar_wait_warp(&s_full[i], phase, abort_flag, status);
        if (!ok) break;
        phase ^= 1u;
        tc_fence_after();
        if (warp_live) {
          uint32_t sr[128];
          tmem_ld128_wait(tS, sr);
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
          if (t > 0 && __any_sync(0xffffffffu, grow)) {
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_wait(tO + c * 32, o);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 v =
                    fmul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2);
                o[e] = __float_as_uint(v.x);
                o[e + 1] = __float_as_uint(v.y);
              }
              tmem_st32(tO + c * 32, o);
            }
          }
          tmem_wait_st();
        }
        nvis -= step;
        tc_fence_before();
        mbar_arrive(&p_full[i]);
      }
      at = save[0], stop = save[1], n = save[2], seq0 = save[3], slot = save[4], kvh = save[5];
      rows0 = save[6], rows1 = save[7], tiles_0 = save[8], tiles_1 = save[9];
      turns_0 = save[10], turns_1 = save[11];
      __syncwarp();
      two = rows1 > 0;
      tile = two ? i : 0;
      tile_rows = tile ? rows1 : rows0;
      const bool live = row < tile_rows;
      const int seq = seq0 + tile * p.seqs_per_tile + row / G;
      const int head = kvh * G + row % G;
      // ---------------------------------------------------- partial state
      // Stream i of two row tiles writes its tile.  With one row tile each
      // stream writes half of the columns, from both streams' O, and stream 0
      // the sums.  Every thread of the streams comes to every barrier here, and
      // they agree on whether a wait gave up: a stream alone would wait for ever.
      if (ok && stream_tiles(i) > 0) ok = mbar_wait_warp(&o_done[i], turns_of(i) & 1, abort_flag, status);
      const size_t n_rows = static_cast<size_t>(p.own.batch) * p.own.H * p.max_slots;
      const size_t to = (static_cast<size_t>(seq) * p.own.H + head) * p.max_slots + slot;
      const bool write = live && in_bounds(to, 1, n_rows, status);
      float m = split_max(m_ref, l);
      float w0 = 1.f, w1 = 0.f;  // weights of O_i and of the other stream's
      const bool other = !two && stream_tiles(1 - i) > 0;
      // row r's maxima at [r] and [128 + r]; stream 1's sums replace the first,
      // which only its own thread reads, and follow at [256 + r]
      float *state = reinterpret_cast<float *>(smem + L::kStates) + row;
      if (!two) {
        state[i * 128] = m;
        named_bar_sync(1, 256);
        if (ok && other)
          ok = mbar_wait_warp(&o_done[1 - i], turns_of(1 - i) & 1, abort_flag, status);
        const float m1 = state[(1 - i) * 128];
        const float top = fmaxf(m, m1);
        w0 = m == -CUDART_INF_F ? 0.f : ex2(m - top);
        w1 = m1 == -CUDART_INF_F ? 0.f : ex2(m1 - top);
        l = w0 == 0.f ? 0.f : w0 * l;
        l_exact = w0 == 0.f ? 0.f : w0 * l_exact;
        m = top;
        if (i == 1) {
          state[0] = l;
          state[256] = l_exact;
        }
      }
      if (ok && warp_live) {
        tc_fence_after();
        const uint32_t tOther = tmem + L::kTmemO + (1 - i) * D + lane_off;
        const int c0 = two ? 0 : i * (D / 64), c1 = two ? D / 32 : c0 + D / 64;
        for (int c = c0; c < c1; ++c) {
          uint32_t o[32];
          tmem_ld32_wait(tO + c * 32, o);
          if (!two) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = w0 == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * w0);
            if (other) {
              uint32_t o1[32];
              tmem_ld32_wait(tOther + c * 32, o1);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (w1 != 0.f)
                  o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
            }
          }
          if (write)
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              const float v[8] = {__uint_as_float(o[e]),     __uint_as_float(o[e + 1]),
                                  __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]),
                                  __uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]),
                                  __uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])};
              store8(p.po_part + to * D + c * 32 + e, v);
            }
        }
      }
      // the next run's products overwrite O once both streams are past this
      tc_fence_before();
      ok = !named_bar_any(1, 256, !ok);
      if (!two && i == 0) {
        l += state[0];
        l_exact += state[256];
      }
      if (ok && write && (two || i == 0)) p.pml_part[to] = make_float4(m, l, l_exact, 0.f);
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

constexpr int kPrefixCombineWarps = 4;  // of a CTA
// on an SM: 72 registers a thread.  (8, with 64, spill a few, and what they spill
// comes from HBM: 1 to 2 us of a call.  6 take two more at the largest batch.)
constexpr int kPrefixCombineCtas = 7;

// E consecutive bf16 values from element `at` on of an array of n.
template <int E>
__device__ __forceinline__ void load_bf16(const void *base, size_t at, size_t n, unsigned int *status,
                                          float (&v)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
  if (!in_bounds(at, E, n, status)) return;
  const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + at);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 x = bf16x2_to_float2(src[e / 2]);
    v[e] = x.x;
    v[e + 1] = x.y;
  }
}

// Rows [row0, row0 + rows) of one sequence over all its keys, one after the other,
// through its own table row: writes the output alone.  (A converged warp, E values
// of the head a lane.)
template <int E>
__device__ __noinline__ void sum_rows(const PrefixParams &p, int row0, int rows) {
  constexpr int D = 32 * E, U = 4;
  const DecodeParams &o = p.own;
  unsigned int *status = o.dev_status;
  const int lane = threadIdx.x & 31, b = row0 / o.H;
  const int ctx = checked_load(o.ctx_lens, b, o.batch, status);
  const size_t n_pool = static_cast<size_t>(o.num_blocks) * kDecodeBlock * o.Hkv * D;
  const size_t n_out = static_cast<size_t>(o.batch) * o.H * D;
  const size_t token = static_cast<size_t>(o.Hkv) * D;  // elements from key to key of a block
  for (int row = row0; row < row0 + rows; ++row) {
    const size_t mine = static_cast<size_t>(row) * D + lane * E;
    const size_t head = static_cast<size_t>((row - b * o.H) / o.group) * D + lane * E;
    float q[E], acc[E], m = -CUDART_INF_F, l = 0.f;
    load_bf16<E>(o.q, mine, n_out, status, q);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int t = 0; t < ctx; t += U) {  // U keys of one block
      const int id = checked_load(
          o.block_table, static_cast<size_t>(b) * o.max_blocks_per_seq + t / kDecodeBlock,
          static_cast<size_t>(o.batch) * o.max_blocks_per_seq, status);
      if (id < 0 || id >= o.num_blocks) {
        if (lane == 0) raise_status(o.dev_status, FA_DEV_BAD_BLOCK);
        break;
      }
      const size_t at =
          (static_cast<size_t>(id) * kDecodeBlock + t % kDecodeBlock) * token + head;
      float s[U], v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float k[E];
        load_bf16<E>(p.k_pool, at + u * token, n_pool, status, k);
        load_bf16<E>(p.v_pool, at + u * token, n_pool, status, v[u]);
        s[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s[u] = fmaf(q[e], k[e], s[u]);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
        s[u] = t + u < ctx ? s[u] * o.scale_log2 : -CUDART_INF_F;
        top = fmaxf(top, s[u]);
      }
      const float ref = top == -CUDART_INF_F ? 0.f : top, alpha = ex2(m - ref);
      m = top;
      l *= alpha;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u >= ctx) break;
        const float w = ex2(s[u] - ref);
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (!in_bounds(mine, E, n_out, status)) continue;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(o.out) + mine);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

}  // namespace

// W warps per (sequence, query head) row, 4 / W rows a CTA; warp w of a row takes
// states w, w + W, ..., a lane each for the maxima and weights, eight o rows per
// memory round trip.  The CTAs are there before the states are and read the plan
// meanwhile, so a call takes no more of them than the GPU holds at once: with
// W = 1 a warp takes `rows` rows of a sequence, one after the other.
template <int D, int W>
__global__ void __launch_bounds__(32 * kPrefixCombineWarps, kPrefixCombineCtas)
    prefix_combine_kernel(const PrefixParams p, const int rows) {
  constexpr int E = D / 32;
  constexpr int U = 8;
  constexpr int R = kPrefixCombineWarps / W;
  __shared__ float s_acc[kPrefixCombineWarps][D];
  __shared__ float s_l[kPrefixCombineWarps], s_lx[kPrefixCombineWarps], s_m[kPrefixCombineWarps];
  const DecodeParams &o = p.own;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = warp % W, r0 = warp - w;
  const int row0 = (blockIdx.x * R + warp / W) * rows;
  const bool live = row0 < o.batch * o.H;  // (a CTA's last rows may lie past the end)
  const int b = live ? row0 / o.H : 0;
  // the plan of the shared keys, and this sequence's place in it
  PrefixSums sums;
  PrefixGroup g{};
  const PrefixFirst firsts = prefix_first(p);
  if (!prefix_walk<kPrefixBySeq>(p, b, false, g, &sums, 0, &firsts)) g = PrefixGroup{};
  const PrefixPlan plan = p.alone ? PrefixPlan{0, 1, true} : prefix_plan(p, sums, firsts);
  const int per = plan.per;
  const int ctx = prefix_ctx(p, b, g.whole, false);  // (decode_own.cu reports)
  const int own = (max(0, ctx - prefix_own_from(p, g)) + o.split_tokens - 1) / o.split_tokens;
  // A sequence that ends inside the shared keys meets the values behind its own with
  // weight 0 in the products, and 0 times an infinity or a NaN is a NaN: then its
  // rows are summed again over its own keys alone.  That takes 0.25 us a key (8000
  // keys 2 ms), and no cache of finite values comes there.  (That the code is there
  // moved calls of 41 to 97 us by 0 to 1.2 us, in line or out of it, here or in the
  // own keys' kernel, as any change of what comes through a cold L2 does.)
  const bool ends_inside = !p.alone && live && ctx < g.whole;
  bool again = false;
  // this kernel's own (checked-build) index errors go to the device word only
  unsigned int *status = o.dev_status;
  const size_t n_own = static_cast<size_t>(o.batch) * o.H * o.max_splits;
  const size_t n_shared = static_cast<size_t>(o.batch) * o.H * p.max_slots;
  pdl_wait_primary();  // both kernels' partial states are complete from here on
  const bool publisher = blockIdx.x == 0 && threadIdx.x == 0;
  const unsigned int call_bits = publisher ? call_status_bits(o.call) : 0u;
  for (int row = row0; row < row0 + rows; ++row) {
    int shared = 0;  // partial states over shared keys
    if (g.tiles > 0 && ctx > 0 && !p.alone) {
      const int round = (row - b * o.H) / o.group / p.team_heads;
      const int first =
          g.start + (round * g.pairs + (b - g.a) / (2 * p.seqs_per_tile)) * g.tiles;
      shared = plan.apart ? (g.tiles + per - 1) / per
                          : (first + g.tiles - 1) / per - first / per + 1;
    }
    const int ns = live ? own + shared : 0;
    const size_t own0 = static_cast<size_t>(row) * o.max_splits;
    const size_t shared0 = static_cast<size_t>(row) * p.max_slots;
    // (m, l, l_exact) of state i, the neutral one past the last
    auto state = [&](int i) -> float3 {
      if (i < own && i < ns && in_bounds(own0 + i, 1, n_own, status)) {
        const float2 x = reinterpret_cast<const float2 *>(o.ml_part)[own0 + i];
        return make_float3(x.x, x.y, x.y);
      }
      if (i >= own && i < ns && in_bounds(shared0 + i - own, 1, n_shared, status)) {
        const float4 x = p.pml_part[shared0 + i - own];
        return make_float3(x.x, x.y, x.z);
      }
      return make_float3(-CUDART_INF_F, 0.f, 0.f);
    };
    // o of U states from the t-th of this warp on (states w + W t); own_o + i D is
    // o of state i, from `own` on shared_o + i D
    const float *own_o = o.o_part + own0 * D + lane * E;
    const float *shared_o = p.po_part + shared0 * D - own * D + lane * E;
    float v[U][E];
    auto load = [&](int t) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (t + u) * W + w;
        const bool there = i < ns && (i < own ? in_bounds(own0 + i, 1, n_own, status)
                                              : in_bounds(shared0 + i - own, 1, n_shared, status));
        const float *src = (i < own ? own_o : shared_o) + i * D;
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
    };
    load(0);
    float3 st = state(lane * W + w);  // of this warp's first 32 states
    float M = st.x;
    for (int i = (lane + 32) * W + w; i < ns; i += 32 * W) M = fmaxf(M, state(i).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if constexpr (W > 1) {
      if (lane == 0) s_m[warp] = M;
      __syncthreads();
#pragma unroll
      for (int x = 0; x < W; ++x) M = fmaxf(M, s_m[r0 + x]);
    }

    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float L = 0.f, Lx = 0.f;  // this lane's states'
    float weight = 0.f;       // this lane's state's
    for (int t = 0; t * W + w < ns; t += U) {
      if (t % 32 == 0) {
        if (t > 0) st = state((t + lane) * W + w);
        // an empty state has weight 0 and is passed over, whatever its o holds
        weight = st.x == -CUDART_INF_F ? 0.f : ex2(st.x - M);
        if (weight != 0.f) {
          L = fmaf(weight, st.y, L);
          Lx = fmaf(weight, st.z, Lx);
        }
      }
      if (t > 0) load(t);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wu = __shfl_sync(0xffffffffu, weight, (t + u) & 31);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = wu != 0.f ? fmaf(wu, v[u][e], acc[e]) : acc[e];
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      L += __shfl_xor_sync(0xffffffffu, L, x);
      Lx += __shfl_xor_sync(0xffffffffu, Lx, x);
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
      if (lane == 0) {
        s_l[warp] = L;
        s_lx[warp] = Lx;
      }
      __syncthreads();
      if (w != 0) break;  // (one row)
      L = Lx = 0.f;
#pragma unroll
      for (int x = 0; x < W; ++x) {
        L += s_l[r0 + x];
        Lx += s_lx[r0 + x];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[e] = 0.f;
#pragma unroll
        for (int x = 0; x < W; ++x) acc[e] += s_acc[r0 + x][lane * E + e];
      }
    }
    if (ends_inside) {
#pragma unroll
      for (int e = 0; e < E; ++e) again = again || !(fabsf(acc[e]) < CUDART_INF_F);
    }
    const float inv = (L == 0.f) ? 0.f : 1.f / L;
    const size_t at = static_cast<size_t>(row) * D + lane * E;
    uint16_t *dst = static_cast<uint16_t *>(o.out) + at;
    if (live && in_bounds(at, E, static_cast<size_t>(o.batch) * o.H * D, status)) {
      if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1 % E] * inv),
                                                     pack_bf16x2(acc[2 % E] * inv, acc[3 % E] * inv));
      else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1 % E] * inv);
    }
    if (live && lane == 0 && o.lse != nullptr &&
        in_bounds(row, 1, static_cast<size_t>(o.batch) * o.H, status))
      o.lse[row] = (Lx == 0.f) ? -CUDART_INF_F : (M + __log2f(Lx)) * 0.69314718055994530942f;
  }
  if (__any_sync(0xffffffffu, again)) sum_rows<E>(p, row0, rows);
  if (publisher) publish_call_status(o.call, call_bits, o.dev_status);
}

// ------------------------------------------------------------------ launch

cudaError_t launch_decode_own(const CUtensorMap &tk, const CUtensorMap &tv, const PrefixParams &p,
                              int d, cudaStream_t stream);

template <int D>
static cudaError_t launch_prefix_d(const PrefixMaps &m, const PrefixParams &p,
                                   cudaStream_t stream) {
  using L = PrefixLayout<D>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = allow_smem(prefix_kernel<D>, L::kBytes, smem_set);
  if (e != cudaSuccess) return e;
  if (!p.alone) {
    prefix_kernel<D><<<p.ctas, kPrefixThreads, L::kBytes, stream>>>(m.q, m.k_tile, m.v_tile, p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = launch_decode_own(m.k, m.v, p, D, stream);
  if (e != cudaSuccess) return e;
  // as many warps a row, and then as few rows a warp, as the GPU holds at once
  const int rows = p.own.batch * p.own.H, ctas = p.ctas * kPrefixCombineCtas;
  const dim3 block(32 * kPrefixCombineWarps);
  if (rows <= ctas)
    return launch_dependent(prefix_combine_kernel<D, 4>, dim3(static_cast<unsigned>(rows)), block, 0,
                            stream, p, 1);
  if (rows <= 2 * ctas)
    return launch_dependent(prefix_combine_kernel<D, 2>,
                            dim3(static_cast<unsigned>((rows + 1) / 2)), block, 0, stream, p, 1);
  int each = 1;
  while (rows > 4LL * each * ctas && p.own.H % (2 * each) == 0) each *= 2;
  return launch_dependent(prefix_combine_kernel<D, 1>,
                          dim3(static_cast<unsigned>((rows / each + 3) / 4)), block, 0, stream, p,
                          each);
}

cudaError_t launch_prefix(const PrefixMaps &m, const PrefixParams &p, int d, cudaStream_t stream) {
  return d == 64 ? launch_prefix_d<64>(m, p, stream) : launch_prefix_d<128>(m, p, stream);
}

}  // namespace fa
