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
  int seqs_per_tile;           // sequences whose group of heads fills a 128-row tile
  int ctas;                    // CTAs that share the prefix work
  int max_slots;               // partial states of a row over shared keys
  float *po_part;              // fp32 [batch, H, max_slots, d]
  float4 *pml_part;            // [batch, H, max_slots]: m (log2 units), l, l_exact, 0
};

// One group: its sequences [a, e), the keys of its shared blocks, and the work
// of it: `pairs` CTA loads of query rows (two tiles) of each KV head, `tiles`
// key tiles each.
struct PrefixGroup {
  int a, e, whole, pairs, tiles;
  long long work;  // key tiles over all pairs and KV heads
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
  r.work = static_cast<long long>(r.tiles) * r.pairs * p.own.Hkv;
  return r;
}

// The group that holds key tile `pos` of the call's work (all groups' one
// after the other), or, with by_seq, the sequence `pos`; its work starts at
// `start`.  All lanes of a converged warp; false if there is none.
__device__ __forceinline__ bool prefix_find(const PrefixParams &p, long long pos, bool by_seq,
                                            PrefixGroup &found, long long &start) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
    const PrefixGroup r = prefix_group(p, g0 + lane, false);
    long long incl = r.work;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(
        0xffffffffu, by_seq ? (r.a <= pos && pos < r.e) : pos < base + incl);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      found.a = __shfl_sync(0xffffffffu, r.a, l);
      found.e = __shfl_sync(0xffffffffu, r.e, l);
      found.whole = __shfl_sync(0xffffffffu, r.whole, l);
      found.pairs = __shfl_sync(0xffffffffu, r.pairs, l);
      found.tiles = __shfl_sync(0xffffffffu, r.tiles, l);
      found.work = __shfl_sync(0xffffffffu, r.work, l);
      start = base + __shfl_sync(0xffffffffu, incl - r.work, l);
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Key tiles of a CTA's share: CTA c takes tiles [c per, (c + 1) per) of the
// call's work.  0 without work (and where groups that overlap against the
// rules add up to more than an int).  All lanes of a converged warp.
__device__ __forceinline__ int prefix_share(const PrefixParams &p, bool report, long long &total) {
  total = 0;
  for (int g = threadIdx.x & 31; g < p.num_groups; g += 32) total += prefix_group(p, g, report).work;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (total > 0x7fffffffLL) total = 0;
  return static_cast<int>((total + p.ctas - 1) / p.ctas);
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

}  // namespace fa
