// fa_cache_api.cu - the C ABI of the 8-bit paged cache (include/fa_kvcache.h):
// argument validation, tensor maps and dispatch, as fa_api.cu for fa.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa_kvcache.h"
#include "cache_internal.h"
#include "fa_host.h"

namespace fa {

cudaError_t launch_cache_append(const AppendParams &p, int d, cudaStream_t stream);
cudaError_t launch_decode_fp8(const CUtensorMap &tk, const CUtensorMap &tv, const DecodeParams &p,
                              const CacheScales &sc, int d, cudaStream_t stream);

cudaError_t launch_prefill_fp8cache(const CUtensorMap &tq, const CUtensorMap &tk,
                                    const CUtensorMap &tv, const CUtensorMap &to,
                                    const PrefillParams &p, int d, bool head_pairs, int grid,
                                    cudaStream_t stream);

namespace {

// window and sinks of a cache call: none, or a window with or without sinks
bool cache_window_ok(int window, int sinks) {
  return (window == 0 && sinks == 0) || (window >= 1 && sinks >= 0);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_append_fp8(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                        void *k_pool, void *v_pool, float *k_scale, float *v_scale,
                        const int32_t *block_table, int max_blocks_per_seq,
                        const int32_t *ctx_lens, const int32_t *cu_seqlens, int batch,
                        int total_tokens, int max_new, int Hkv, int d, int block_size,
                        int num_blocks, fa_stream_t stream) {
  if (!k || !v || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || !ctx_lens ||
      !cu_seqlens)
    return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
      !aligned(ctx_lens, 4) || !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  if (batch < 0 || total_tokens < 0 || max_new < 0 || Hkv < 1 || num_blocks < 1 ||
      max_blocks_per_seq < 1)
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (block_size != kDecodeBlock) return FA_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(Hkv) * d;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return FA_ERR_INVALID_ARG;
  if (batch > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (batch == 0 || total_tokens == 0 || max_new == 0) return FA_OK;
  max_new = std::min(max_new, total_tokens);
  if ((max_new / kDecodeBlock + 2LL) * Hkv * 2 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;

  AppendParams p{};
  p.status = status_ptr();
  if (p.status == nullptr) return FA_ERR_CUDA;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.cu_seqlens = cu_seqlens;
  p.batch = batch;
  p.total_tokens = total_tokens;
  p.max_new = max_new;
  p.Hkv = Hkv;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return launch_cache_append(p, d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_decode_paged_fp8(const void *q, const void *k_pool, const void *v_pool,
                        const float *k_scale, const float *v_scale, const int32_t *block_table,
                        int max_blocks_per_seq, const int32_t *ctx_lens, int max_ctx_len,
                        int batch, int H, int Hkv, int d, int block_size, int num_blocks,
                        float scale, int window, int sinks, void *out, float *lse,
                        void *workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || !ctx_lens || !out)
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
      !aligned(ctx_lens, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID_ARG;
  if (batch < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || num_blocks < 1 ||
      max_blocks_per_seq < 1 || max_ctx_len < 0)
    return FA_ERR_INVALID_ARG;
  if (!cache_window_ok(window, sinks)) return FA_ERR_INVALID_ARG;
  if (max_ctx_len > kMaxCtxLen) return FA_ERR_UNSUPPORTED;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (block_size != kDecodeBlock) return FA_ERR_UNSUPPORTED;
  if (H / Hkv > 16) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_ctx_len)
    return FA_ERR_INVALID_ARG;
  if (batch > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (batch == 0) return FA_OK;
  const WindowSpec win = clamp_window({window, sinks}, max_ctx_len);
  const DecodeWs w = decode_ws(batch, H, Hkv, d, window_keys(win, max_ctx_len));
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < FA_WORKSPACE_HEADER_BYTES + w.o_bytes + w.ml_bytes)
    return FA_ERR_WORKSPACE;
  CallStatus *call = static_cast<CallStatus *>(workspace);
  uint8_t *parts = static_cast<uint8_t *>(workspace) + FA_WORKSPACE_HEADER_BYTES;

  CUtensorMap tk, tv;
  const long long tokens = static_cast<long long>(num_blocks) * block_size;
  int rc = make_pool_map(&tk, k_pool, d, Hkv, tokens, kDecodeBlock, 1);
  if (rc == FA_OK) rc = make_pool_map(&tv, v_pool, d, Hkv, tokens, kDecodeBlock, 1);
  if (rc != FA_OK) return rc;

  DecodeParams p{};
  p.dev_status = status_ptr();
  if (p.dev_status == nullptr) return FA_ERR_CUDA;
  p.status = &call->acc;
  p.call = call;
  p.q = q;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.o_part = reinterpret_cast<float *>(parts);
  p.ml_part = reinterpret_cast<float *>(parts + w.o_bytes);
  p.out = out;
  p.lse = lse;
  p.batch = batch;
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_ctx_len = max_ctx_len;
  p.num_blocks = num_blocks;
  p.split_tokens = w.split_tokens;
  p.max_splits = w.max_splits;
  p.scale_log2 = scale * kLog2e;
  p.window = win.window;
  p.sinks = win.sinks;
  return launch_decode_fp8(tk, tv, p, {k_scale, v_scale}, d,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_fwd_paged_fp8(const void *q, const void *k_pool, const void *v_pool, const float *k_scale,
                     const float *v_scale, const int32_t *block_table, int max_blocks_per_seq,
                     const int32_t *ctx_lens, const int32_t *cu_seqlens_q, int batch, int total_q,
                     int max_seqlen_q, int max_ctx_len, int H, int Hkv, int d, int block_size,
                     int num_blocks, float scale, int window, int sinks, void *out, float *lse,
                     fa_stream_t stream) {
  if (!q || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || !ctx_lens ||
      !cu_seqlens_q || !out)
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
      !aligned(ctx_lens, 4) || !aligned(cu_seqlens_q, 4) || (lse && !aligned(lse, 4)))
    return FA_ERR_INVALID_ARG;
  if (batch < 0 || total_q < 0 || max_seqlen_q < 0 || max_ctx_len < 0 || H < 1 || Hkv < 1 ||
      H % Hkv != 0 || num_blocks < 1 || max_blocks_per_seq < 1)
    return FA_ERR_INVALID_ARG;
  if (!cache_window_ok(window, sinks)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (block_size != kDecodeBlock) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks_per_seq) * block_size < max_ctx_len)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return FA_OK;
  max_seqlen_q = std::min(max_seqlen_q, total_q);
  const bool head_pairs = (H / Hkv) % 2 == 0;
  const int rows = head_pairs ? kPrefillBM : kPrefillRowsPerCta;  // query rows per work item
  const long long pairs = (max_seqlen_q + rows - 1) / rows;
  const long long grid = pairs * batch * (head_pairs ? H / 2 : H);
  if (grid > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(total_q) * H * d * 2 >= (1LL << 40)) return FA_ERR_UNSUPPORTED;

  CUtensorMap tq, tk, tv, to;
  const long long tokens = static_cast<long long>(num_blocks) * block_size;
  int rc = make_map(&tq, q, d, H, total_q, 1, kPrefillBM);
  // (K's codes are MMA operands; V's are read by the widening warps: rows as they are)
  if (rc == FA_OK) rc = make_pool_map(&tk, k_pool, d, Hkv, tokens, kDecodeBlock, 1);
  if (rc == FA_OK) rc = make_pool_map(&tv, v_pool, d, Hkv, tokens, kDecodeBlock, 1, false);
  if (rc == FA_OK) rc = make_map(&to, out, d, H, total_q, 1, kPrefillBM);
  if (rc != FA_OK) return rc;

  PrefillParams p{};
  p.status = status_ptr();
  if (p.status == nullptr) return FA_ERR_CUDA;
  p.out = out;
  p.lse = lse;
  p.cu_seqlens = cu_seqlens_q;
  p.B = batch;
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.head_group = head_pairs ? 2 * prefill_head_group(H / 2) : prefill_head_group(H);
  p.N = total_q;
  p.max_pairs = static_cast<int>(pairs);
  p.total_tokens = total_q;
  p.scale_log2 = scale * kLog2e;
  p.v_descale = 1.f;
  p.causal = 1;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_ctx_len = max_ctx_len;
  p.num_blocks = num_blocks;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  // without a window: one that reaches over any context
  const WindowSpec win =
      clamp_window({window == 0 ? std::max(1, max_ctx_len) : window, sinks}, max_ctx_len);
  p.window = win.window;
  p.sinks = win.sinks;
  return launch_prefill_fp8cache(tq, tk, tv, to, p, d, head_pairs, static_cast<int>(grid),
                                 reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
