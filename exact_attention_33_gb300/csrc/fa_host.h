// fa_host.h - host helpers of the C ABI: tensor maps, argument rules and
// workspace layouts, shared by fa_api.cu and fa_cache_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "fa_internal.h"

namespace fa {

// Device address of the sticky status word of the current device (fa_api.cu).
unsigned int *status_ptr();

constexpr float kLog2e = 1.4426950408889634f;

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Tensor [outer][rows][heads][d] (d innermost) of bf16 (or one-byte, or
// fp32) elements as a 4-D TMA map with dims {d, heads, rows, outer}; each
// copy moves a box of one swizzled row of swz_bytes per (head, row): {64, 1,
// box_rows, 1} bf16 values with the 128-byte swizzle, or, for e4m3 rows of
// d = 64, {64, 1, box_rows, 1} bytes with the 64-byte swizzle.
// Out-of-range rows read as zero and are not stored.
inline int make_map(CUtensorMap *map, const void *base, int d, int heads, long long rows,
             long long outer, int box_rows, int elem_bytes = 2, int swz_bytes = 128) {
  auto fn = encode_fn();
  if (fn == nullptr) return FA_ERR_CUDA;
  const cuuint64_t eb = static_cast<cuuint64_t>(elem_bytes);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * eb,
                                 static_cast<cuuint64_t>(heads) * d * eb,
                                 static_cast<cuuint64_t>(rows) * heads * d * eb};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(swz_bytes / elem_bytes), 1,
                             static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType dt = elem_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : elem_bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUresult r = fn(map, dt, 4, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swz_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// Swizzled row bytes of the prefill kernels for e4m3 rows of d values.
inline int fp8_swz(int d) { return d < 128 ? d : 128; }

// Paged pool [num_blocks * block_size tokens][Hkv][d] of bf16 values or e4m3
// codes as a 3-D map; each copy moves one swizzled row per token, {64, 1,
// box_rows} bf16 values (a whole 16-token block, or one token row), or {d, 1,
// box_rows} codes with the 128- or 64-byte swizzle, or without one.
inline int make_pool_map(CUtensorMap *map, const void *base, int d, int heads, long long tokens,
                  int box_rows = kDecodeBlock, int elem_bytes = 2, bool swizzled = true) {
  auto fn = encode_fn();
  if (fn == nullptr) return FA_ERR_CUDA;
  const cuuint64_t eb = static_cast<cuuint64_t>(elem_bytes);
  const int swz = std::min(128, d * elem_bytes);  // bytes of a swizzled row
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * eb,
                                 static_cast<cuuint64_t>(heads) * d * eb};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(swz / elem_bytes), 1,
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map,
                  elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !swizzled   ? CU_TENSOR_MAP_SWIZZLE_NONE
                  : swz == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                              : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// The keys a causal query sees: all up to its own (window 0), or the last
// `window` of them and the first `sinks` keys of the sequence.
struct WindowSpec {
  int window = 0;
  int sinks = 0;
};

// The window arguments of a call, checked.
inline bool window_ok(int window, int sinks) { return window >= 1 && sinks >= 0; }

// No sequence is longer than `longest` keys: a longer window or more sinks
// than that see the same keys (and positions less a window stay in int).
inline WindowSpec clamp_window(WindowSpec w, int longest) {
  if (w.window > 0) w.window = std::min(w.window, std::max(1, longest));
  w.sinks = std::min(w.sinks, std::max(0, longest));
  return w;
}

inline bool scale_ok(float s) { return std::isfinite(s) && s > 0.f; }

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Keys per split of the decode kernel.  Large splits keep the partial-state
// traffic small; the split shrinks (down to 64 keys) while the number of
// (sequence, KV head, split) work items would not fill kDecodeWaveCtas split
// CTAs per SM (about two waves of seven resident CTAs).
#ifndef FA_DECODE_WAVE_CTAS
#define FA_DECODE_WAVE_CTAS 14
#endif
constexpr int kDecodeWaveCtas = FA_DECODE_WAVE_CTAS;
constexpr int kDecodeMinSplitTokens = 64;
// Work items that a decode call wants at least.
inline long long decode_want_items() {
  int sms = sm_count();
  if (sms <= 0) sms = 148;
  return static_cast<long long>(kDecodeWaveCtas) * sms;
}
inline int decode_split_tokens(int batch, int Hkv, int max_ctx_len) {
  const long long want = decode_want_items();
  int split = kDecodeMaxSplitTokens;
  while (split > kDecodeMinSplitTokens) {
    const long long items = static_cast<long long>(batch) * Hkv *
                            ((static_cast<long long>(max_ctx_len) + split - 1) / split);
    if (items >= want) break;
    split >>= 1;
  }
  return split;
}

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Context lengths above this are refused (the split arithmetic stays in int).
constexpr int kMaxCtxLen = 0x7fffffff - kDecodeMaxSplitTokens;

// Heads per group of the prefill CTA order: the largest divisor of H that is
// at most 8 (consecutive heads, so GQA heads sharing a KV head stay together).
inline int prefill_head_group(int H) {
  for (int g = 8; g > 1; --g)
    if (H % g == 0) return g;
  return 1;
}

// Splits of the split-KV prefill: about 1.7 CTAs per SM (rounded down), at
// most 16 splits and at most one split per key tile.  Every extra split costs
// an fp32 partial tile per query tile and its share of the combine; on
// B1 H4 N8192 causal (128 work items on 152 SMs) 2 splits ran at 924 TFLOP/s
// against 796 for 3 and 640 unsplit, and from 256 work items up the unsplit
// kernel was fastest.
inline int prefill_num_splits(int B, int H, int N, int requested) {
  const long long pairs = (N + kPrefillRowsPerCta - 1) / kPrefillRowsPerCta;
  const int tiles = (N + kPrefillBN - 1) / kPrefillBN;
  int s = requested;
  if (s <= 0) {
    int sms = sm_count();
    if (sms <= 0) sms = 148;
    const long long base = std::max(1LL, pairs * B * H);
    s = static_cast<int>(std::min(16LL, (17LL * sms) / (10LL * base)));
  }
  return std::max(1, std::min({s, 16, std::max(1, tiles)}));
}

struct SplitWs {
  int splits;
  size_t o_bytes, ml_bytes;
};

// Split-KV workspace: control block, fp32 partial o tiles, (m, l, l_exact).
inline SplitWs split_ws(int B, int H, int N, int d, int requested) {
  SplitWs w;
  w.splits = prefill_num_splits(B, H, N, requested);
  const size_t rows = static_cast<size_t>(w.splits) * B * N * H;
  w.o_bytes = round_up(rows * d * sizeof(float), 256);
  w.ml_bytes = round_up(rows * 4 * sizeof(float), 256);
  return w;
}

inline size_t split_ws_bytes(const SplitWs &w) { return FA_WORKSPACE_HEADER_BYTES + w.o_bytes + w.ml_bytes; }

// Keys of the cache blocks that a decode call reads at most: every one up to
// max_ctx_len, or whole blocks of the sinks and of the window (whose first
// and last keys may lie anywhere in their blocks).
inline int window_keys(WindowSpec w, int max_ctx_len) {
  if (w.window == 0) return max_ctx_len;
  auto blocks = [](long long keys) { return (keys + kDecodeBlock - 1) / kDecodeBlock; };
  const long long read = blocks(w.sinks) + blocks(w.window + kDecodeBlock - 1LL);
  return static_cast<int>(std::min<long long>(max_ctx_len, read * kDecodeBlock));
}

struct DecodeWs {
  int split_tokens;
  int max_splits;
  size_t o_bytes;
  size_t ml_bytes;
};

// Decode workspace: control block, fp32 partial o rows, (m, l) pairs.
inline DecodeWs decode_ws(int batch, int H, int Hkv, int d, int max_ctx_len) {
  DecodeWs w;
  w.split_tokens = decode_split_tokens(batch, Hkv, max_ctx_len);
  w.max_splits = static_cast<int>(std::max(
      1LL, (static_cast<long long>(max_ctx_len) + w.split_tokens - 1) / w.split_tokens));
  const size_t rows = static_cast<size_t>(batch) * H * w.max_splits;
  w.o_bytes = round_up(rows * d * sizeof(float), 256);
  w.ml_bytes = round_up(rows * 2 * sizeof(float), 256);
  return w;
}

// Workspace bytes that every decode call of at most `batch` sequences of at most
// max_ctx_len keys fits into.  The split size falls as the batch or the context
// does, so what a call needs rises with neither.  Its splits of one head are at
// most ceil(keys / 512) of each sequence or, where they are shorter than that,
// at most ceil(keys / 64) of each, and all of them (on every KV head) fewer than
// twice the wanted items, because splits of twice the size were fewer than those.
inline size_t decode_ws_bound(int batch, int H, int Hkv, int d, int max_ctx_len) {
  auto splits = [&](int tokens) {
    return batch * std::max(1LL, (static_cast<long long>(max_ctx_len) + tokens - 1) / tokens);
  };
  const long long rows =
      H * std::max(splits(kDecodeMaxSplitTokens),
                   std::min(splits(kDecodeMinSplitTokens), 2 * decode_want_items() / Hkv));
  return round_up(static_cast<size_t>(rows) * d * sizeof(float), 256) +
         round_up(static_cast<size_t>(rows) * 2 * sizeof(float), 256);
}

}  // namespace fa
