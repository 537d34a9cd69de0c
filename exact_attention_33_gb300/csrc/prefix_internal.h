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
  // What decides how many do: ns of a key tile with two row tiles and with one,
  // before and after them, and of the partial states that each CTA adds; bytes
  // a key (all KV heads); bytes a ns that the own keys' CTAs read at most, and on
  // an SM that is left to them.
  float tile_ns2, tile_ns1, fixed_ns, state_ns;
  float key_bytes, max_rate, free_rate;
  int max_slots;               // partial states of a row over shared keys
  float *po_part;              // fp32 [batch, H, max_slots, d]
  float4 *pml_part;            // [batch, H, max_slots]: m (log2 units), l, l_exact, 0
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
// heads each time.)
//
// One group: its sequences [a, e), the keys of its shared blocks, and the work
// of it: `pairs` CTA loads of query rows (two tiles), `tiles` key tiles each;
// `start` key tiles lie before it in the line.
struct PrefixGroup {
  int a, e, whole, pairs, tiles;
  int start;
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
// 1) per) of `total`.  (Whatever the arrays hold, it is an int: the host sees to
// that.)
struct PrefixPlan {
  int total, per;
};

// What the search is for: the group of a sequence, or of a key tile.
constexpr int kPrefixNone = 0, kPrefixBySeq = 1, kPrefixByTile = 2;

// Walks over the groups, 32 at a time (all lanes of a converged warp).  Finds
// the group that `what` and `key` ask for, into `found`; false if there is none.
// Sums the work, its cost in ns of one SM, and the keys that sequences share.
struct PrefixSums {
  int total;
  float cost;
  long long shared_keys;
};
template <int WHAT>
__device__ __forceinline__ bool prefix_walk(const PrefixParams &p, int key, bool report,
                                            PrefixGroup &found, PrefixSums *sums) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  bool hit = false;
  if (sums) *sums = {0, 0.f, 0};
  for (int g0 = 0; g0 < p.num_groups && !(hit && !sums); g0 += 32) {
    PrefixGroup r = prefix_group(p, g0 + lane, report);
    const int work = r.tiles * r.pairs * p.head_rounds;
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
        found.start = __shfl_sync(0xffffffffu, r.start, l);
        hit = true;
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (sums) {
      // pairs with two row tiles take longer than a single one
      const int n = r.e - r.a, single = n > 0 && (n - 1) / p.seqs_per_tile % 2 == 0 ? 1 : 0;
      const float tiles = static_cast<float>(r.tiles * p.own.Hkv);
      sums->cost = __fadd_rn(
          sums->cost, __fmul_rn(tiles, __fadd_rn(__fmul_rn(static_cast<float>(r.pairs - single),
                                                           p.tile_ns2),
                                                 __fmul_rn(static_cast<float>(single), p.tile_ns1))));
      sums->shared_keys += static_cast<long long>(r.whole) * n;
    }
  }
  if (sums) sums->total = base;
  return hit;
}

// The plan of a call, the same in every warp that asks (integers, and fp32
// operations that no compiler contracts).  The own keys' CTAs read while this
// work computes, on the SMs that it leaves to them and then on all of them; it
// takes as many as let both end first.  (64 sequences over 8192 keys, 300 to
// 1000 of their own: 64 SMs 42 us, 86 SMs 46, 128 SMs 47; 256 over 16384 keys:
// 120 SMs 107 us, 152 SMs 124.)
__device__ __forceinline__ PrefixPlan prefix_plan(const PrefixParams &p, const PrefixSums &s) {
  const int lane = threadIdx.x & 31;
  if (s.total <= p.ctas / p.team_heads) return {max(0, s.total), 1};
  float cost = s.cost;
  // keys of all sequences, from every `skip`-th of a large batch
  const int skip = (p.own.batch + 1023) / 1024;
  long long keys = 0;
  for (int b = lane * skip; b < p.own.batch; b += 32 * skip)
    keys += max(0, checked_load(p.own.ctx_lens, b, p.own.batch, p.own.status));
  keys *= skip;
  float shared = static_cast<float>(s.shared_keys);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    cost = __fadd_rn(cost, __shfl_xor_sync(0xffffffffu, cost, o));
    shared = __fadd_rn(shared, __shfl_xor_sync(0xffffffffu, shared, o));
    keys += __shfl_xor_sync(0xffffffffu, keys, o);
  }
  // lane l tries whole teams of ctas - l ctas / 40 SMs
  const int n = max(1, (p.ctas - lane * p.ctas / 40) / p.team_heads) * p.team_heads;
  const float own_bytes =
      __fmul_rn(fmaxf(0.f, __fadd_rn(static_cast<float>(keys), -shared)), p.key_bytes);
  // (without an SM of their own they come after this work)
  const float rate = fminf(p.max_rate, __fmul_rn(static_cast<float>(p.ctas - n), p.free_rate));
  const float mine = __fadd_rn(p.fixed_ns, __fdiv_rn(cost, static_cast<float>(n)));
  const float all = __fdiv_rn(own_bytes, p.max_rate);
  // what they have not read by the end of this work they read on every SM
  const float rest = fmaxf(0.f, __fadd_rn(own_bytes, -__fmul_rn(rate, mine)));
  const float t = __fadd_rn(fmaxf(all, __fadd_rn(mine, __fdiv_rn(rest, p.max_rate))),
                            __fmul_rn(static_cast<float>(n), p.state_ns));
  const unsigned best = __reduce_min_sync(
      0xffffffffu, (static_cast<unsigned>(fminf(t, 1.3e8f)) << 5) | static_cast<unsigned>(lane));
  const int teams = __shfl_sync(0xffffffffu, n / p.team_heads, best & 31);
  const int total = max(0, s.total);
  return {total, max(1, (total + teams - 1) / teams)};
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
