// fa_rope_api.cu - the C ABI of the rotary calls (include/fa_rope.h): argument
// validation and dispatch, as fa_api.cu for fa.h.
#include <cuda_runtime.h>

#include "../../include/fa_rope.h"
#include "cache_internal.h"
#include "fa_host.h"
#include "rope_internal.h"

namespace fa {

cudaError_t launch_rope(const RopeParams &p, int d, bool interleaved, bool back,
                        cudaStream_t stream);
cudaError_t launch_append_rope(const RopeParams &p, int d, bool interleaved, cudaStream_t stream);
cudaError_t launch_cache_append_rope(const AppendParams &p, const RopeParams &rp, float grow, int d,
                                     bool interleaved, cudaStream_t stream);

namespace {

// rows of `heads` heads of d values: addresses, and strides that hold them
bool rows_ok(const RopeRows &r, int d) {
  const int64_t row = static_cast<int64_t>(r.heads) * d;
  return r.src && r.dst && aligned(r.src, 16) && aligned(r.dst, 16) && r.src_stride >= row &&
         r.dst_stride >= row && r.src_stride % 8 == 0 && r.dst_stride % 8 == 0 &&
         (r.src != r.dst || r.src_stride == r.dst_stride);
}

int rope_ok(const RopeSpec &s, int rot_dim, int d) {
  if (!s.inv_freq || !aligned(s.inv_freq, 8) || rot_dim < 1 || rot_dim > d || !scale_ok(s.factor))
    return FA_ERR_INVALID_ARG;
  return rot_dim % 16 == 0 ? FA_OK : FA_ERR_UNSUPPORTED;
}

int rope(RopeParams p, int rot_dim, int interleaved, int d, bool back, fa_stream_t stream) {
  if (p.total_tokens < 0 || p.q.heads < 1 || p.k.heads < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!rows_ok(p.q, d) || (p.k.heads > 0 && !rows_ok(p.k, d))) return FA_ERR_INVALID_ARG;
  if (p.positions ? !aligned(p.positions, 4) : p.seq_len < 1) return FA_ERR_INVALID_ARG;
  const int rc = rope_ok(p.rope, rot_dim, d);
  if (rc != FA_OK) return rc;
  if (p.q.heads > 65535 || p.k.heads > 65535) return FA_ERR_UNSUPPORTED;
  if (p.total_tokens == 0) return FA_OK;
  if (p.k.heads == 0) p.k.src = nullptr;
  p.status = status_ptr();
  if (p.status == nullptr) return FA_ERR_CUDA;
  return launch_rope(p, d, interleaved != 0, back, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// What the two writes' checks share; `run` is false where there is nothing to do.
int append_ok(const RopeRows &q, const RopeRows &k, const RopeRows &v, const RopeSpec &s,
              int rot_dim, const void *k_pool, const void *v_pool, const int32_t *block_table,
              int max_blocks_per_seq, const int32_t *ctx_lens, const int32_t *cu_seqlens, int batch,
              int total_tokens, int max_new, int d, int block_size, int num_blocks, bool &run) {
  run = false;
  if (!k.src || !v.src || !k_pool || !v_pool || !block_table || !ctx_lens || !cu_seqlens)
    return FA_ERR_INVALID_ARG;
  if (!aligned(k.src, 16) || !aligned(v.src, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return FA_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  if (batch < 0 || total_tokens < 0 || max_new < 0 || k.heads < 1 || num_blocks < 1 ||
      max_blocks_per_seq < 1)
    return FA_ERR_INVALID_ARG;
  if ((q.src == nullptr) != (q.dst == nullptr) || (q.src && q.heads < 1)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (block_size != kDecodeBlock) return FA_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(k.heads) * d;
  if (k.src_stride < row || v.src_stride < row || k.src_stride % 8 != 0 || v.src_stride % 8 != 0)
    return FA_ERR_INVALID_ARG;
  if (q.src && !rows_ok(q, d)) return FA_ERR_INVALID_ARG;
  if (rot_dim != 0 || s.inv_freq) {
    const int rc = rope_ok(s, rot_dim, d);
    if (rc != FA_OK) return rc;
  }
  if (batch > 65535 || k.heads > 65535 || (q.src && q.heads > 65535)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  run = batch > 0 && total_tokens > 0 && max_new > 0;
  return FA_OK;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_rope(const void *q, const void *k, int64_t q_stride, int64_t k_stride, void *q_out,
            void *k_out, int64_t q_out_stride, int64_t k_out_stride, const double *inv_freq,
            int rot_dim, float factor, int interleaved, const int32_t *positions, int seq_len,
            int total_tokens, int H, int Hkv, int d, fa_stream_t stream) {
  RopeParams p{};
  p.rope = {inv_freq, rot_dim / 2, factor};
  p.q = {q, q_out, q_stride, q_out_stride, H};
  p.k = {k, k_out, k_stride, k_out_stride, Hkv};
  p.positions = positions;
  p.seq_len = seq_len;
  p.total_tokens = total_tokens;
  return rope(p, rot_dim, interleaved, d, false, stream);
}

int fa_rope_bwd(const void *dq, const void *dk, int64_t dq_stride, int64_t dk_stride, void *dq_out,
                void *dk_out, int64_t dq_out_stride, int64_t dk_out_stride, const double *inv_freq,
                int rot_dim, float factor, int interleaved, const int32_t *positions, int seq_len,
                int total_tokens, int H, int Hkv, int d, fa_stream_t stream) {
  RopeParams p{};
  p.rope = {inv_freq, rot_dim / 2, factor};
  p.q = {dq, dq_out, dq_stride, dq_out_stride, H};
  p.k = {dk, dk_out, dk_stride, dk_out_stride, Hkv};
  p.positions = positions;
  p.seq_len = seq_len;
  p.total_tokens = total_tokens;
  return rope(p, rot_dim, interleaved, d, true, stream);
}

int fa_cache_append_rope(const void *q, const void *k, const void *v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, void *q_out, int64_t q_out_stride,
                         const double *inv_freq, int rot_dim, float factor, int interleaved,
                         void *k_pool, void *v_pool, const int32_t *block_table,
                         int max_blocks_per_seq, const int32_t *ctx_lens,
                         const int32_t *cu_seqlens, int batch, int total_tokens, int max_new,
                         int H, int Hkv, int d, int block_size, int num_blocks,
                         fa_stream_t stream) {
  RopeParams p{};
  p.rope = {inv_freq, rot_dim / 2, factor};
  p.q = {q, q_out, q_stride, q_out_stride, H};
  p.k = {k, nullptr, k_stride, 0, Hkv};
  p.v = {v, nullptr, v_stride, 0, Hkv};
  bool run;
  const int rc = append_ok(p.q, p.k, p.v, p.rope, rot_dim, k_pool, v_pool, block_table,
                           max_blocks_per_seq, ctx_lens, cu_seqlens, batch, total_tokens, max_new,
                           d, block_size, num_blocks, run);
  if (rc != FA_OK || !run) return rc;
  p.status = status_ptr();
  if (p.status == nullptr) return FA_ERR_CUDA;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.cu_seqlens = cu_seqlens;
  p.batch = batch;
  p.total_tokens = total_tokens;
  p.max_new = std::min(max_new, total_tokens);
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  return launch_append_rope(p, d, interleaved != 0, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_cache_append_rope_fp8(const void *q, const void *k, const void *v, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, void *q_out,
                             int64_t q_out_stride, const double *inv_freq, int rot_dim,
                             float factor, int interleaved, void *k_pool, void *v_pool,
                             float *k_scale, float *v_scale, const int32_t *block_table,
                             int max_blocks_per_seq, const int32_t *ctx_lens,
                             const int32_t *cu_seqlens, int batch, int total_tokens, int max_new,
                             int H, int Hkv, int d, int block_size, int num_blocks,
                             fa_stream_t stream) {
  RopeParams r{};
  r.rope = {inv_freq, rot_dim / 2, factor};
  r.q = {q, q_out, q_stride, q_out_stride, H};
  const RopeRows kr = {k, nullptr, k_stride, 0, Hkv}, vr = {v, nullptr, v_stride, 0, Hkv};
  if (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !inv_freq)
    return FA_ERR_INVALID_ARG;
  bool run;
  const int rc = append_ok(r.q, kr, vr, r.rope, rot_dim, k_pool, v_pool, block_table,
                           max_blocks_per_seq, ctx_lens, cu_seqlens, batch, total_tokens, max_new,
                           d, block_size, num_blocks, run);
  if (rc != FA_OK || !run) return rc;
  max_new = std::min(max_new, total_tokens);
  if ((max_new / kDecodeBlock + 6LL) * (Hkv * 2 + 8) + max_new > 0x7fffffffLL)
    return FA_ERR_UNSUPPORTED;
  // what a rotated key may grow by
  const float grow = std::max(1.f, static_cast<float>(1.4142135623730951 * factor));
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
  r.status = p.status;
  r.ctx_lens = ctx_lens;
  r.cu_seqlens = cu_seqlens;
  r.batch = batch;
  r.total_tokens = total_tokens;
  r.max_new = max_new;
  r.max_blocks_per_seq = max_blocks_per_seq;
  return launch_cache_append_rope(p, r, grow, d, interleaved != 0,
                                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

}  // extern "C"
