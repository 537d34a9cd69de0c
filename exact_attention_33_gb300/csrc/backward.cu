// backward.cu - launches of the backward kernels without a window.
#include "backward_kernel.cuh"

namespace fa {

cudaError_t launch_bwd(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                       const CUtensorMap &tv, const BwdParams &p, int d, bool causal,
                       cudaStream_t stream) {
  if (p.cu_seqlens != nullptr)
    return d == 64 ? launch_bwd_d<64, true>(tq, tdo, tk, tv, p, causal, stream)
                   : launch_bwd_d<128, true>(tq, tdo, tk, tv, p, causal, stream);
  return d == 64 ? launch_bwd_d<64, false>(tq, tdo, tk, tv, p, causal, stream)
                 : launch_bwd_d<128, false>(tq, tdo, tk, tv, p, causal, stream);
}

}  // namespace fa
