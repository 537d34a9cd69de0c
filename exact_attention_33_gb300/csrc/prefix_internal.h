// prefix_internal.h - what the kernels of a decode call over shared prefixes
// have in common: their parameters, and the plan that every CTA reads off the
// groups by itself.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "checks.cuh"
#include "fa_internal.h"

namespace fa {

constexpr int kPrefixTileKeys = 128;

struct PrefixParams {
  // The own keys' decode call.  block_table, ctx_lens, q, the status words and
  // the sizes serve all kernels; max_ctx_len is the table's reach, o_part and
  // ml_part are the own keys' partial states [batch, H, max_splits].
  DecodeParams own;
  const int32_t *cu_groups;    // [num_groups + 1]
  const int32_t *prefix_lens;  // [num_groups]
  int num_groups;
  int max_prefix, max_own;     // keys; max_own counts the prefix's last part block
  int alone;                   // every key as a sequence's own (small calls)
  int seqs_per_tile;           // sequences whose group of heads fills a 128-row tile
  int ctas;                    // CTAs that share the prefix work at most (one an SM)
  int team_heads, head_rounds; // KV heads that a team does at a time, and how often
  int teams;                   // at most
  // What decides how many do: ns of a key tile with two row tiles and with one,
  // before and after them, between two runs, and of the partial states that each
  // CTA adds; bytes of a cache block (all KV heads); bytes a ns that the own keys' CTAs read
  // at most, and on an SM that is left to them.
  float tile_ns2, tile_ns1, fixed_ns, run_ns, state_ns;
  float block_bytes, max_rate, max_rate_inv, free_rate;
  int max_slots;               // partial states of a row over shared keys
  float *po_part;              // fp32 [batch, H, max_slots, d]
  float4 *pml_part;            // [batch, H, max_slots]: m (log2 units), l, l_exact, 0
  const void *k_pool, *v_pool; // bf16 [num_blocks, 16, Hkv, d]
};

// The maps of Q, of the pools as the own keys' kernel copies them (a block's
// tokens x 64 values) and as the shared keys' one does (a block's whole rows).
struct PrefixMaps {
  CUtensorMap q, k, v, k_tile, v_tile;
};

// The work is a line of key tiles, group after group and, in a group, pair of
// row tiles after pair.  Teams of team_heads CTAs share it out in equal
// stretches; a team's CTAs do the same stretch for a KV head each, so that the
// heads of a token, which lie side by side in the pools, are read together.
// (More KV heads than CTAs: a group's pairs come head_rounds times, with other
// heads each time.)  Where it pays, a pair's place in the line is rounded up to
// whole stretches, so that none goes on into another pair (PrefixPlan::apart).
//
// One group: its sequences [a, e), the keys of its shared blocks, and the work
// of it: `pairs` CTA loads of query rows (two tiles), `tiles` key tiles each,
// `span` of the line; `start` of the line lies before it.
struct PrefixGroup {
  int a, e, whole, pairs, tiles;
  int span, start;
  bool bad;  // outside the batch or of negative size (and empty here)
};

__device__ __forceinline__ PrefixGroup prefix_group(const PrefixParams &p, int g, bool report) {
  PrefixGroup r{};
  if (g >= p.num_groups) return r;
  unsigned int *status = p.own.status;
  const int a = checked_load(p.cu_groups, g, p.num_groups + 1, status);
  const int e = checked_load(p.cu_groups, g + 1, p.num_groups + 1, status);
  const int n = checked_load(p.prefix_lens, g, p.num_groups, status);
  if (a < 0 || e < a || e > p.own.batch) {
    if (report) raise_status(status, FA_DEV_BAD_SEQLEN);
    r.bad = true;
    return r;
  }
  r.a = a;
  r.e = e;
  if (n < 0 || n > p.max_prefix ||
      n > p.own.max_blocks_per_seq * static_cast<long long>(kDecodeBlock)) {
    if (report) raise_status(status, FA_DEV_BAD_CTX);
    return r;
  }
  r.whole = n / kDecodeBlock * kDecodeBlock;
  r.tiles = (r.whole + kPrefixTileKeys - 1) / kPrefixTileKeys;
  r.pairs = (e - a + 2 * p.seqs_per_tile - 1) / (2 * p.seqs_per_tile);
  return r;
}

// The line's length, and how it is shared: team t takes key tiles [t per, (t +
// 1) per) of `total`; `apart`: a pair's key tiles begin at a multiple of `per`.
// (Whatever the arrays hold, the line's length without gaps is an int: the host
// sees to that.  With gaps it is at most per times the teams.)
struct PrefixPlan {
  int total, per;
  bool apart;
};

// What the search is for: the group of a sequence, or of a key tile.
constexpr int kPrefixNone = 0, kPrefixBySeq = 1, kPrefixByTile = 2;

// Keys of the batch's sequences (of a large batch's every `skip`-th), four a lane:
// loaded before the walk over the groups, whose loads they then do not wait for.
constexpr int kPrefixFirst = 4;
struct PrefixFirst {
  int keys[kPrefixFirst];
};
__device__ __forceinline__ int prefix_skip(const PrefixParams &p) {
  return (p.own.batch + 32 * kPrefixFirst - 1) / (32 * kPrefixFirst);
}
__device__ __forceinline__ PrefixFirst prefix_first(const PrefixParams &p) {
  const int lane = threadIdx.x & 31, skip = prefix_skip(p);
  PrefixFirst f;
#pragma unroll
  for (int i = 0; i < kPrefixFirst; ++i) {
    const int b = (lane + 32 * i) * skip;
    f.keys[i] = b < p.own.batch ? checked_load(p.own.ctx_lens, b, p.own.batch, p.own.status) : 0;
  }
  return f;
}

// Walks over the groups, 32 at a time (all lanes of a converged warp).  Finds
// the group that `what` and `key` ask for, into `found`; false if there is none.
// Sums the work; key tiles of pairs with two row tiles and with one and the shared
// blocks are this lane's groups' alone; with `first`, `covered` is the blocks that
// this lane's of those sequences share.  Of the first 32 groups lane l keeps the l-th
// one's pairs and their key tiles.  `apart`: 0, or the stretch that pairs are rounded
// up to.
struct PrefixSums {
  int total;
  int tiles2, tiles1;
  long long blocks;
  int covered;
  int pairs, tiles;
};
template <int WHAT>
__device__ __forceinline__ bool prefix_walk(const PrefixParams &p, int key, bool report,
                                            PrefixGroup &found, PrefixSums *sums, int apart = 0,
                                            const PrefixFirst *first = nullptr) {
  const int lane = threadIdx.x & 31;
  int base = 0, reached = 0;  // of the groups before these: their work, their largest end
  bool hit = false, falls = false;
  if (sums) *sums = {};
  for (int g0 = 0; g0 < p.num_groups && !(hit && !sums); g0 += 32) {
    PrefixGroup r = prefix_group(p, g0 + lane, report);
    int end = g0 + lane < p.num_groups ? r.e : 0x7fffffff;  // the largest up to this group's
    // A group begins where the one before it ends, so groups in order do not
    // overlap.  Behind one that is not, a group that begins inside an earlier one is
    // passed over too: both would write their sequences' states.
    falls = falls || __any_sync(0xffffffffu, r.bad);
    if (falls) {
      end = max(reached, end);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(0xffffffffu, end, o));
      int before = __shfl_up_sync(0xffffffffu, end, 1);
      if (lane == 0) before = reached;
      if (r.a < before && r.a < r.e) {
        if (report) raise_status(p.own.status, FA_DEV_BAD_SEQLEN);
        r = PrefixGroup{};
      }
    }
    reached = __shfl_sync(0xffffffffu, end, min(31, p.num_groups - 1 - g0));
    r.span = apart > 0 ? (r.tiles + apart - 1) / apart * apart : r.tiles;
    const int work = r.span * r.pairs * p.head_rounds;
    int incl = work;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    r.start = base + incl - work;
    if (WHAT != kPrefixNone && !hit) {
      const unsigned at = __ballot_sync(
          0xffffffffu, WHAT == kPrefixBySeq ? (r.a <= key && key < r.e)
                                            : (work > 0 && key < r.start + work));
      if (at != 0u) {
        const int l = __ffs(at) - 1;
        found.a = __shfl_sync(0xffffffffu, r.a, l);
        found.e = __shfl_sync(0xffffffffu, r.e, l);
        found.whole = __shfl_sync(0xffffffffu, r.whole, l);
        found.pairs = __shfl_sync(0xffffffffu, r.pairs, l);
        found.tiles = __shfl_sync(0xffffffffu, r.tiles, l);
        found.span = __shfl_sync(0xffffffffu, r.span, l);
        found.start = __shfl_sync(0xffffffffu, r.start, l);
        hit = true;
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (sums) {
      // pairs with two row tiles take longer than a single one
      const int n = r.e - r.a, single = n <= (2 * r.pairs - 1) * p.seqs_per_tile ? 1 : 0;
      sums->tiles2 += r.tiles * (r.pairs - single);
      sums->tiles1 += r.tiles * single;
      sums->blocks += n > 0 ? r.whole / kDecodeBlock : 0;
      if (first) {
        // (rolled: what is fetched to run once costs more than the loop)
        const int skip = prefix_skip(p);
#pragma unroll 1
        for (int i = 0; i < kPrefixFirst && 32 * i * skip < reached; ++i) {
          const int b = (lane + 32 * i) * skip;
          const int keys = i < 2 ? (i == 0 ? first->keys[0] : first->keys[1])
                                  : (i == 2 ? first->keys[2] : first->keys[3]);
          int l = 0;  // the first group that ends behind b
          if (p.num_groups > 1)
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1)
              if (__shfl_sync(0xffffffffu, end, l + o - 1) <= b) l += o;
          const int a = __shfl_sync(0xffffffffu, r.a, l), e = __shfl_sync(0xffffffffu, r.e, l);
          const int whole = __shfl_sync(0xffffffffu, r.whole, l);
          if (a <= b && b < e) sums->covered += min(max(0, keys), whole) / kDecodeBlock;
        }
      }
      if (g0 == 0) {
        sums->pairs = r.pairs * p.head_rounds;
        sums->tiles = r.tiles;
      }
    }
  }
  if (sums) sums->total = base;
  return hit;
}

// 1 / x, to 2^-23, the same in every kernel
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The plan of a call, the same in every warp that asks (integers, and fp32
// operations that no compiler contracts, without divisions: a call waits for it).  The own keys' CTAs read while this
// work computes, on the SMs that it leaves to them and then on all of them; it
// takes as many as let both end first.  (64 sequences over 8192 keys, 1 to
// 1024 of their own: 48 SMs 47 us, 64 SMs 42, 88 SMs 47, 128 SMs 49; 256 over 16384
// keys, 1 to 512 of their own: 64 SMs 136 us, 96 SMs 98, 128 SMs 110, 152 SMs 125.)
//
// A stretch that goes from one pair to the next has two runs, and the MMAs rest
// between them until O has left, Q has come and the first weights are there: 8
// us that the other teams do not have.  Pairs set apart have no such stretch, but
// their last ones are shorter; the same estimate decides.
__device__ __forceinline__ PrefixPlan prefix_plan(const PrefixParams &p, const PrefixSums &s,
                                                  const PrefixFirst &f) {
  const int lane = threadIdx.x & 31;
  const int total = max(0, s.total), teams = p.teams;
  if (total <= teams) return {total, 1, false};
  // blocks of their own that the sequences read
  int mine = -s.covered;
#pragma unroll
  for (int i = 0; i < kPrefixFirst; ++i) mine += max(0, f.keys[i]) / kDecodeBlock;
  // (cut off at 2^25 a lane: such a call is bound by its bytes whatever the plan)
  constexpr long long kMost = 1 << 25;
  const int own_blocks = __reduce_add_sync(0xffffffffu, min(1 << 25, mine));
  const int once = __reduce_add_sync(0xffffffffu, static_cast<int>(min(kMost, s.blocks)));
  const int tiles2 = __reduce_add_sync(0xffffffffu, s.tiles2);
  const int tiles1 = __reduce_add_sync(0xffffffffu, s.tiles1);
  // lane l tries stretches of 1 to 4 times what all teams would take
  const int least = (total - 1) / teams + 1;
  int per = static_cast<int>(min(static_cast<long long>(total), least + 3LL * least * lane / 32));
  // ... and, pairs set apart, the least that cuts none into more parts
  int parts = 0, even = 1;
  if (p.num_groups <= 32)
    for (int g = 0; g < p.num_groups; ++g) {
      const int tiles = __shfl_sync(0xffffffffu, s.tiles, g);
      const int pairs = __shfl_sync(0xffffffffu, s.pairs, g);
      if (tiles > 0 && pairs > 0) {
        const int n = (tiles - 1) / per + 1;
        parts += n * pairs;
        even = max(even, (tiles - 1) / n + 1);
      }
    }
  const float own_bytes = __fmul_rn(__fmul_rn(static_cast<float>(own_blocks), p.block_bytes),
                                    static_cast<float>(prefix_skip(p)));
  const float all_bytes = __fadd_rn(own_bytes, __fmul_rn(static_cast<float>(once), p.block_bytes));
  const float tiles = __fadd_rn(static_cast<float>(tiles2), static_cast<float>(tiles1));
  const float tile_ns = __fmul_rn(__fadd_rn(__fmul_rn(static_cast<float>(tiles2), p.tile_ns2),
                                            __fmul_rn(static_cast<float>(tiles1), p.tile_ns1)),
                                  rcp_approx(tiles));
  // ns of the call with stretches of `x` on n SMs, `more` beside what CTAs take anyway
  auto estimate = [&](int x, int n, float more) {
    // (without an SM of their own they come after this work)
    const float rate = fminf(p.max_rate, __fmul_rn(static_cast<float>(p.ctas - n), p.free_rate));
    const float mine = __fadd_rn(more, __fmul_rn(static_cast<float>(x), tile_ns));
    // what they have not read by the end of this work they read on every SM
    const float rest = fmaxf(0.f, __fadd_rn(own_bytes, -__fmul_rn(rate, mine)));
    const float t = fmaxf(__fmul_rn(all_bytes, p.max_rate_inv),
                          __fadd_rn(mine, __fmul_rn(rest, p.max_rate_inv)));
    return static_cast<unsigned>(
        fminf(__fadd_rn(t, __fmul_rn(static_cast<float>(n), p.state_ns)), 1.3e8f));
  };
  const unsigned line = estimate(per, ((total - 1) / per + 1) * p.team_heads,
                                 __fadd_rn(p.fixed_ns, p.run_ns));
  const unsigned apart = parts > 0 && parts <= teams
                             ? estimate(even, parts * p.team_heads, p.fixed_ns)
                             : 0xffffffffu;
  const unsigned best =
      __reduce_min_sync(0xffffffffu, (min(apart, line) << 5) | static_cast<unsigned>(lane));
  const int l = best & 31;
  const bool is_apart = __shfl_sync(0xffffffffu, apart <= line ? 1 : 0, l) != 0;
  per = __shfl_sync(0xffffffffu, is_apart ? even : per, l);
  if (!is_apart) return {total, per, false};
  const int parts_of_all = __reduce_add_sync(
      0xffffffffu, s.tiles > 0 ? ((s.tiles - 1) / per + 1) * s.pairs : 0);
  return {parts_of_all * per, per, true};
}

// The first key that a sequence of a group reads on its own.
__device__ __forceinline__ int prefix_own_from(const PrefixParams &p, const PrefixGroup &g) {
  return p.alone ? 0 : g.whole;
}

// Keys of sequence b, 0 where ctx_lens breaks a rule (`whole` of them shared).
__device__ __forceinline__ int prefix_ctx(const PrefixParams &p, int b, int whole, bool report) {
  const int ctx = checked_load(p.own.ctx_lens, b, p.own.batch, p.own.status);
  if (ctx >= 0 && ctx <= p.own.max_blocks_per_seq * static_cast<long long>(kDecodeBlock) &&
      ctx - static_cast<long long>(whole) <= p.max_own)
    return ctx;
  if (report) raise_status(p.own.status, FA_DEV_BAD_CTX);
  return 0;
}

// Launches a kernel as a programmatic dependent of the one before it on the
// stream.
template <typename Kernel, typename... Args>
inline cudaError_t launch_dependent(Kernel kern, dim3 grid, dim3 block, size_t smem,
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

}  // namespace fa
