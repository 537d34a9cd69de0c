// fa_prefix_api.cu - the C ABI of decoding over shared prefixes
// (include/fa_prefix.h): argument validation, tensor maps and dispatch, as
// fa_api.cu for fa.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa_prefix.h"
#include "fa_host.h"
#include "prefix_internal.h"

namespace fa {

cudaError_t launch_prefix(const PrefixMaps &m, const PrefixParams &p, int d, cudaStream_t stream);

namespace {

// Twice the ordinary work items: sequences' own keys mostly stay well below
// max_own_len, and a call of few rounds of CTAs waits for the last of them.
constexpr int kOwnItems = 2;

// Calls that read less than this (K and V of every sequence up to its largest
// length) take every key as its sequence's own: two kernels instead of three,
// and the shared blocks come from L2.  Measured with 32 / 8 heads of d = 128, us
// as own keys and as shared ones: 3 sequences over 1001 keys (two heads of 64)
// 9 and 14, 8 over 1024 keys (36 MB) 14.4 and 16.0, 4 over 4096 (68 MB) 18.5 and
// 19.2, 16 over 1024 (71 MB) 18.5 and 17.2, 8 over 4096 (136 MB) 27 and 21.
constexpr long long kAloneBytes = 64LL << 20;

// Most keys of a sequence.
int longest(int max_prefix, int max_own) { return max_prefix + max_own + kDecodeBlock - 1; }

bool prefix_alone(int batch, int Hkv, int d, int max_prefix, int max_own) {
  return static_cast<long long>(batch) * longest(max_prefix, max_own) <=
         kAloneBytes / (4LL * Hkv * d);
}

// Bytes of the partial states that such calls of at most this batch and these
// lengths need: a call of b sequences of c keys each, b c <= keys, has at most
// ceil(c / 512) states of each head and sequence, or, where its splits are
// shorter, fewer than twice the wanted items and at most ceil(c / 64) of each.
size_t alone_bound(int batch, int H, int Hkv, int d, int max_prefix, int max_own, int times) {
  const long long keys = std::min(static_cast<long long>(batch) * longest(max_prefix, max_own),
                                  kAloneBytes / (4LL * Hkv * d));
  const long long rows =
      H * std::max(keys / kDecodeMaxSplitTokens + batch,
                   std::min(keys / kDecodeMinSplitTokens + batch, 2 * decode_want_items(times) / Hkv));
  return round_up(static_cast<size_t>(rows) * d * sizeof(float), 256) +
         round_up(static_cast<size_t>(rows) * 2 * sizeof(float), 256);
}

struct PrefixWs {
  int max_slots;
  size_t o_bytes, ml_bytes;
  size_t bytes() const { return o_bytes + ml_bytes; }
};

int prefix_ctas() {
  const int sms = sm_count();
  return sms > 0 ? sms : 148;
}

// positions stay in int
bool lengths_ok(int max_prefix, int max_own) {
  return static_cast<long long>(max_prefix) + max_own <= kMaxCtxLen - kDecodeBlock;
}

// KV heads of a team: the most that divide Hkv and find CTAs.
int team_heads(int Hkv) {
  int h = std::min(Hkv, prefix_ctas());
  while (Hkv % h != 0) --h;
  return h;
}

// Partial states over shared keys.  A run of a CTA is at least one key tile,
// and a team's share of the line at least the teams' part of one group's tiles,
// so a row meets at most as many shares of them as there are teams, and two cut
// ones.
PrefixWs prefix_ws(int batch, int H, int Hkv, int d, int max_prefix) {
  PrefixWs w;
  const int tiles = (max_prefix / kDecodeBlock * kDecodeBlock + kPrefixTileKeys - 1) / kPrefixTileKeys;
  w.max_slots = std::max(1, std::min(tiles, prefix_ctas() / team_heads(Hkv) + 2));
  const size_t rows = static_cast<size_t>(batch) * H * w.max_slots;
  w.o_bytes = round_up(rows * d * sizeof(float), 256);
  w.ml_bytes = round_up(rows * 4 * sizeof(float), 256);
  return w;
}

// The tensor map of Q [batch, H, d] for boxes of `seqs` sequences x the heads
// of one KV group x 64 values.
int make_q_map(CUtensorMap *map, const void *q, int batch, int H, int group, int d, int seqs) {
  auto fn = encode_fn();
  if (fn == nullptr) return FA_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(H) * d * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(seqs)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// A pool's tensor map for whole blocks of one KV head: 16 tokens' rows of d bf16
// values go to shared memory as 128-byte swizzled rows, 8 tokens x 64 values at
// a time, the 64-value chunks of 8 tokens one behind the other.  (One copy of 4
// KB a block: what a copy costs the copy engine does not shrink with it.)
int make_block_map(CUtensorMap *map, const void *pool, int d, int Hkv, long long tokens) {
  auto fn = encode_fn();
  if (fn == nullptr) return FA_ERR_CUDA;
  const cuuint64_t row = static_cast<cuuint64_t>(Hkv) * d * 2;
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(d / 64),
                              static_cast<cuuint64_t>(tokens / 8), static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(d / 64), kDecodeBlock / 8, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(pool), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_decode_prefix_workspace_size(int batch, int H, int Hkv, int d, int max_prefix_len,
                                       int max_own_len, int block_size) {
  if (batch < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || max_prefix_len < 0 || max_own_len < 0)
    return 0;
  if ((d != 64 && d != 128) || block_size != kDecodeBlock) return 0;
  if (!lengths_ok(max_prefix_len, max_own_len)) return 0;
  const PrefixWs w = prefix_ws(batch, H, Hkv, d, max_prefix_len);
  return FA_WORKSPACE_HEADER_BYTES +
         std::max(alone_bound(batch, H, Hkv, d, max_prefix_len, max_own_len, kOwnItems),
                  w.bytes() + decode_ws_bound(batch, H, Hkv, d, max_own_len + kDecodeBlock - 1,
                                              kOwnItems));
}

int fa_decode_paged_prefix(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *ctx_lens, const int32_t *cu_groups,
                           const int32_t *prefix_lens, int num_groups, int max_prefix_len,
                           int max_own_len, int batch, int H, int Hkv, int d, int block_size,
                           int num_blocks, float scale, void *out, float *lse, void *workspace,
                           size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !block_table || !ctx_lens || !out) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16))
    return FA_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(ctx_lens, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID_ARG;
  if (num_groups < 0 || (num_groups > 0 && (!cu_groups || !prefix_lens || !aligned(cu_groups, 4) ||
                                            !aligned(prefix_lens, 4))))
    return FA_ERR_INVALID_ARG;
  if (batch < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || num_blocks < 1 || max_blocks_per_seq < 1 ||
      max_prefix_len < 0 || max_own_len < 0)
    return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (block_size != kDecodeBlock) return FA_ERR_UNSUPPORTED;
  if (H / Hkv > 16) return FA_ERR_UNSUPPORTED;
  const long long reach = static_cast<long long>(max_blocks_per_seq) * block_size;
  if (reach < std::max(max_prefix_len, max_own_len)) return FA_ERR_INVALID_ARG;
  if (!lengths_ok(max_prefix_len, max_own_len)) return FA_ERR_UNSUPPORTED;
  if (batch > 65535 || Hkv > 65535 || static_cast<long long>(batch) * H > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (batch == 0) return FA_OK;
  const int group = H / Hkv, seqs = kPrefillBM / group;
  // Key tiles are counted in int, whatever groups the arrays name: those that stand
  // do not overlap, so they have at most a batch's worth of pairs of row tiles each,
  // and all of them one batch's worth and a pair for each group of some sequences.
  // (Every CTA walks over all groups, hence their limit.)
  const long long tiles = (max_prefix_len + kPrefixTileKeys - 1LL) / kPrefixTileKeys;
  const long long pairs = (batch + 2LL * seqs - 1) / (2 * seqs);
  const long long all_pairs =
      std::min(num_groups * pairs, pairs + std::min<long long>(num_groups, batch));
  if (num_groups > 65535 || tiles * Hkv * all_pairs > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const int max_own = max_own_len + kDecodeBlock - 1;
  const bool alone = prefix_alone(batch, Hkv, d, max_prefix_len, max_own_len);
  const DecodeWs w = decode_ws(
      batch, H, Hkv, d,
      alone ? static_cast<int>(std::min<long long>(reach, longest(max_prefix_len, max_own_len)))
            : max_own,
      kOwnItems);
  if (static_cast<long long>(w.max_splits) * Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const PrefixWs s = alone ? PrefixWs{1, 0, 0} : prefix_ws(batch, H, Hkv, d, max_prefix_len);
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < FA_WORKSPACE_HEADER_BYTES + w.o_bytes + w.ml_bytes + s.bytes())
    return FA_ERR_WORKSPACE;
  CallStatus *call = static_cast<CallStatus *>(workspace);
  uint8_t *parts = static_cast<uint8_t *>(workspace) + FA_WORKSPACE_HEADER_BYTES;

  PrefixMaps m{};
  const long long tokens = static_cast<long long>(num_blocks) * block_size;
  int rc = make_pool_map(&m.k, k_pool, d, Hkv, tokens);
  if (rc == FA_OK) rc = make_pool_map(&m.v, v_pool, d, Hkv, tokens);
  if (!alone) {
    if (rc == FA_OK) rc = make_q_map(&m.q, q, batch, H, group, d, seqs);
    if (rc == FA_OK) rc = make_block_map(&m.k_tile, k_pool, d, Hkv, tokens);
    if (rc == FA_OK) rc = make_block_map(&m.v_tile, v_pool, d, Hkv, tokens);
  }
  if (rc != FA_OK) return rc;

  PrefixParams p{};
  p.own.dev_status = status_ptr();
  if (p.own.dev_status == nullptr) return FA_ERR_CUDA;
  p.own.status = &call->acc;
  p.own.call = call;
  p.own.q = q;
  p.own.block_table = block_table;
  p.own.ctx_lens = ctx_lens;
  p.own.o_part = reinterpret_cast<float *>(parts);
  p.own.ml_part = reinterpret_cast<float *>(parts + w.o_bytes);
  p.own.out = out;
  p.own.lse = lse;
  p.own.batch = batch;
  p.own.H = H;
  p.own.Hkv = Hkv;
  p.own.group = group;
  p.own.max_blocks_per_seq = max_blocks_per_seq;
  p.own.max_ctx_len = static_cast<int>(std::min<long long>(reach, 0x7fffffff));
  p.own.num_blocks = num_blocks;
  p.own.split_tokens = w.split_tokens;
  p.own.max_splits = w.max_splits;
  p.own.scale_log2 = scale * kLog2e;
  p.cu_groups = cu_groups;
  p.prefix_lens = prefix_lens;
  p.num_groups = num_groups;
  p.max_prefix = max_prefix_len;
  p.max_own = max_own;
  p.alone = alone;
  p.seqs_per_tile = seqs;
  p.ctas = prefix_ctas();
  p.team_heads = team_heads(Hkv);
  p.head_rounds = Hkv / p.team_heads;
  p.teams = p.ctas / p.team_heads;
  // What prefix_plan's estimate is made of: ns of a key tile of 128 with two row
  // tiles and with one, before a CTA's first product and after its last, between two
  // runs, and what one more CTA costs the others; bytes a ns that the own keys' CTAs
  // read on an SM that is left to them while the others work, and all at most.  All
  // ten are fits, no times of anything by themselves (a key tile with two row tiles
  // takes 1.65 us in a long run without own keys): of 53 batches (d = 64 and 128, 1 to
  // 16 heads a group, 1 to 20 groups, own keys from none to twice the shared ones,
  // idle slots) every stretch was timed.  The ones chosen so take 1.6% longer than the
  // best, 15% at worst (4 unlike groups, d = 64); batches that were left out of the fit
  // do nearly as well.  The constants before, taken at three batches of one shape,
  // chose ones that take 6.2% longer, 38% at worst.
  p.tile_ns2 = d == 128 ? 2600.f : 1500.f;
  p.tile_ns1 = d == 128 ? 2600.f : 930.f;
  p.fixed_ns = 6900.f;
  p.run_ns = 5300.f;
  p.state_ns = d == 128 ? 160.f : 39.f;
  p.block_bytes = 4.f * kDecodeBlock * d * Hkv;
  p.max_rate = 5600.f;
  p.max_rate_inv = 1.f / p.max_rate;
  p.free_rate = 51.f;
  p.max_slots = s.max_slots;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.po_part = reinterpret_cast<float *>(parts + w.o_bytes + w.ml_bytes);
  p.pml_part = reinterpret_cast<float4 *>(parts + w.o_bytes + w.ml_bytes + s.o_bytes);
  return launch_prefix(m, p, d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
