// backward_window.cu - launches of the windowed backward kernels: the row sums D
// = sum_j P_ij dP_ij, then dK / dV = sums of P^T dO and scale dS^T Q, then dQ =
// scale dS K with dS = P (dP - D), over the tiles that the window and the sinks
// leave.  Nine products where five are the gradient's, so that no kernel adds into
// another's results.  16 packed documents of up to 4096 rows, 16 / 4 heads of
// d = 128, window 512, 16 sinks take 1.0 ms with the forward pass, 474 TFLOP/s of
// the seven products that forward and gradient cannot do without.  No pipe is
// full: the tensor pipe is busy 43 to 48% of the cycles (23 to 25% at d = 64), the
// issue slots 29 to 36% (35 to 40%), the exponential's unit 12 to 26%.  Each step
// waits in turn for scores, weights, dP and dS, mostly for loads from TMEM.
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
