// prefill.cu - instantiations and launches of the prefill kernel for every
// unwindowed layout, and the split-KV combine.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "fa_internal.h"
#include "prefill_kernel.cuh"
#include "ptx.cuh"
#include "checks.cuh"

namespace fa {

// ------------------------------------------------------------------ split combine
// One warp per (batch, row, head) merges the partial states of the splits
// with the rescaling of the explainer page's "Show the maths":
// M = max m_s, o = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s,
// lse = (M + log2 sum 2^(m_s - M) l_exact_s) ln 2.
template <int D>
__global__ void __launch_bounds__(128) prefill_split_combine_kernel(const PrefillParams p) {
  pdl_wait_primary();  // the split grid's partial states are complete from here on
  // The split grid has raised all its status bits: one thread reads them
  // here and publishes them as the call's status when its row is done.
  const bool publisher = blockIdx.x == 0 && threadIdx.x == 0 && p.call != nullptr;
  const unsigned int call_bits = publisher ? call_status_bits(p.call) : 0u;
  // this kernel's own (checked-build) index errors go to the device word only
  unsigned int *status = p.call != nullptr ? p.dev_status : p.status;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const size_t rows = static_cast<size_t>(p.B) * p.N * p.H;
  const size_t gw = static_cast<size_t>(blockIdx.x) * 4 + warp;
  if (gw >= rows) return;
  const size_t bn = gw / p.H;  // b * N + n
  const int h = static_cast<int>(gw % p.H);
  const size_t stride = static_cast<size_t>(p.B) * p.N * p.H;  // between splits
  const size_t parts = static_cast<size_t>(p.num_splits) * stride;  // partial rows
  // (m, l, l_exact) of split s for this row (the neutral state if the index
  // fails a check of the checked build)
  auto ml = [&](int sp) -> float4 {
    const size_t idx = sp * stride + gw;
    return in_bounds(idx, 1, parts, status) ? reinterpret_cast<const float4 *>(p.ml_part)[idx]
                                              : make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
  };
  // M = max over the splits, one split per lane (at most 16 splits)
  float M = (lane < p.num_splits) ? ml(lane).x : -CUDART_INF_F;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float Ls = 0.f, Le = 0.f;
  // Split s adds 2^(m_s - M) (l_s, l_exact_s, o_s), four splits per memory
  // round trip; a split without keys for this row (m_s = -inf) is passed
  // over by a select, so its o_s slot never reaches the output.
  if (M != -CUDART_INF_F) {
    auto add = [&](const float4 st, const float (&v)[E]) {
      const bool live = st.x != -CUDART_INF_F;
      const float w = ex2(st.x - M);
      Ls = live ? fmaf(w, st.y, Ls) : Ls;
      Le = live ? fmaf(w, st.z, Le) : Le;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = live ? fmaf(w, v[e], acc[e]) : acc[e];
    };
    auto load_o = [&](int sp, float (&v)[E]) {
      const size_t idx = (sp * stride + gw) * D + lane * E;
      const bool in = in_bounds(idx, E, parts * D, status);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = in ? p.o_part[idx + e] : 0.f;
    };
    constexpr int U = 4;
    int sp = 0;
    for (; sp + U <= p.num_splits; sp += U) {
      float4 st[U];
      float v[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        st[u] = ml(sp + u);
        load_o(sp + u, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add(st[u], v[u]);
    }
    for (; sp < p.num_splits; ++sp) {
      float v[E];
      load_o(sp, v);
      add(ml(sp), v);
    }
  }
  const float inv = (Ls > 0.f) ? 1.f / Ls : 0.f;
  uint16_t *dst = static_cast<uint16_t *>(p.out) + gw * D + lane * E;
  if (in_bounds(gw * D + lane * E, E, rows * D, status)) {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
  const size_t b = bn / p.N, n = bn % p.N;
  const size_t lse_idx = (b * p.H + h) * p.N + n;
  if (lane == 0 && p.lse != nullptr && in_bounds(lse_idx, 1, rows, status))
    p.lse[lse_idx] = (Le > 0.f) ? (M + __log2f(Le)) * 0.69314718055994530942f : -CUDART_INF_F;
  if (publisher) publish_call_status(p.call, call_bits, p.dev_status);
}

cudaError_t launch_prefill_split_combine(const PrefillParams &p, int d, cudaStream_t stream) {
  const size_t rows = static_cast<size_t>(p.B) * p.N * p.H;
  // launched as a programmatic dependent of the split grid on the same stream
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (d == 64) return cudaLaunchKernelEx(&cfg, prefill_split_combine_kernel<64>, p);
  return cudaLaunchKernelEx(&cfg, prefill_split_combine_kernel<128>, p);
}

// Publishes the status of a split-KV call that ran the plain kernel alone
// (one split), once that kernel has completed.
__global__ void __launch_bounds__(32) call_status_kernel(CallStatus *call, unsigned int *dev) {
  if (threadIdx.x == 0) publish_call_status(call, call_status_bits(call), dev);
}

cudaError_t launch_call_status(CallStatus *call, unsigned int *dev, cudaStream_t stream) {
  call_status_kernel<<<1, 32, 0, stream>>>(call, dev);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ launch

template <int D, int KIND, int QT = 2>
static cudaError_t launch_prefill_k(const CUtensorMap &tq, const CUtensorMap &tk,
                                    const CUtensorMap &tv, const CUtensorMap &tv1,
                                    const CUtensorMap &to, const PrefillParams &p, bool causal,
                                    int grid, cudaStream_t stream) {
  return causal ? launch_prefill_t<D, true, KIND, false, QT>(tq, tk, tv, tv1, to, p, grid, stream)
                : launch_prefill_t<D, false, KIND, false, QT>(tq, tk, tv, tv1, to, p, grid, stream);
}

// FP8 prefill, d = 64 or 128: dense batches and packed sequences (row pairs
// or head pairs); `to` is the bf16 output map (used at d = 128).
template <int D, int KIND>
static cudaError_t launch_prefill_fp8_k(const CUtensorMap &tq, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &to,
                                        const PrefillParams &p, bool causal, int grid,
                                        cudaStream_t stream) {
  return causal ? launch_prefill_t<D, true, KIND, true>(tq, tk, tv, tv, to, p, grid, stream)
                : launch_prefill_t<D, false, KIND, true>(tq, tk, tv, tv, to, p, grid, stream);
}

template <int D>
static cudaError_t launch_prefill_fp8_d(const CUtensorMap &tq, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &to,
                                        const PrefillParams &p, bool causal, int grid,
                                        cudaStream_t stream, int kind) {
  if (kind == kKindVarlen)
    return launch_prefill_fp8_k<D, kKindVarlen>(tq, tk, tv, to, p, causal, grid, stream);
  if (kind == kKindVarlenHeads)
    return launch_prefill_fp8_k<D, kKindVarlenHeads>(tq, tk, tv, to, p, causal, grid, stream);
  return launch_prefill_fp8_k<D, kKindDense>(tq, tk, tv, to, p, causal, grid, stream);
}

cudaError_t launch_prefill_fp8(const CUtensorMap &tq, const CUtensorMap &tk,
                               const CUtensorMap &tv, const CUtensorMap &to,
                               const PrefillParams &p, bool causal, int grid,
                               cudaStream_t stream, int kind, int d) {
  return d == 64 ? launch_prefill_fp8_d<64>(tq, tk, tv, to, p, causal, grid, stream, kind)
                 : launch_prefill_fp8_d<128>(tq, tk, tv, to, p, causal, grid, stream, kind);
}

cudaError_t launch_prefill(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const CUtensorMap &tv1, const CUtensorMap &to, const PrefillParams &p,
                           int d, bool causal, int kind, int grid, cudaStream_t stream,
                           int qtiles) {
  if (kind == kKindVarlen && qtiles == 1)
    return d == 64 ? launch_prefill_k<64, kKindVarlen, 1>(tq, tk, tv, tv1, to, p, causal, grid, stream)
                   : launch_prefill_k<128, kKindVarlen, 1>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (d == 64) {
    if (kind == kKindDense)
      return launch_prefill_k<64, kKindDense>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    if (kind == kKindVarlen)
      return launch_prefill_k<64, kKindVarlen>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    if (kind == kKindVarlenHeads)
      return launch_prefill_k<64, kKindVarlenHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    if (kind == kKindDenseHeads)
      return launch_prefill_k<64, kKindDenseHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    if (kind == kKindDenseSplit)
      return launch_prefill_k<64, kKindDenseSplit>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    if (kind == kKindPagedHeads)
      return launch_prefill_k<64, kKindPagedHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
    return launch_prefill_k<64, kKindPaged>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  }
  if (kind == kKindDense)
    return launch_prefill_k<128, kKindDense>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (kind == kKindVarlen)
    return launch_prefill_k<128, kKindVarlen>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (kind == kKindVarlenHeads)
    return launch_prefill_k<128, kKindVarlenHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (kind == kKindDenseHeads)
    return launch_prefill_k<128, kKindDenseHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (kind == kKindDenseSplit)
    return launch_prefill_k<128, kKindDenseSplit>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  if (kind == kKindPagedHeads)
    return launch_prefill_k<128, kKindPagedHeads>(tq, tk, tv, tv1, to, p, causal, grid, stream);
  return launch_prefill_k<128, kKindPaged>(tq, tk, tv, tv1, to, p, causal, grid, stream);
}

}  // namespace fa
