// backward_window.cu - launches of the windowed backward kernels.
#include "backward_kernel.cuh"

namespace fa {

cudaError_t launch_bwd_window(const CUtensorMap &tq, const CUtensorMap &tdo, const CUtensorMap &tk,
                              const CUtensorMap &tv, const BwdParams &p, int d,
                              cudaStream_t stream) {
  if (p.cu_seqlens != nullptr)
    return d == 64 ? launch_bwd_d<64, true, true>(tq, tdo, tk, tv, p, true, stream)
                   : launch_bwd_d<128, true, true>(tq, tdo, tk, tv, p, true, stream);
  return d == 64 ? launch_bwd_d<64, false, true>(tq, tdo, tk, tv, p, true, stream)
                 : launch_bwd_d<128, false, true>(tq, tdo, tk, tv, p, true, stream);
}

}  // namespace fa
