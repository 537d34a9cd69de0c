// prefill_window.cu - windowed instantiations of the prefill kernel: a query
// at position i sees key j <= i when j > i - window or j < sinks.  A CTA
// streams the key tiles of the sinks and those from the window of its first
// row to its diagonal, so the work grows with N (window + sinks) instead of
// N^2.  Only the first window tile, the diagonal tile and the last sink tile
// hold masked scores.  32 packed prompts of 64 to 4096 rows, 16 / 4 heads of
// d = 128, window 1024, 4 sinks: 547 us, 892 TFLOP/s of visible scores.  No pipe
// is full (8 sequences of 2048, window 512: tensor 38%, issue slots 49% of the
// cycles): a tile's softmax waits for its scores and its products for the weights,
// and the masked halves of the edge tiles and what a CTA spends around a few key
// tiles come on top.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "prefill_kernel.cuh"

namespace fa {

// A head-pair item of a short window is a few key tiles long, and what a CTA
// spends before and after them (set-up, the first copies, the epilogue) a
// quarter of its time.  Persistent CTAs, one an SM, take the items in turn, and
// the next item's copies and first products run beside the last softmax and the
// epilogue.  They take fixed shares, and long items level out badly.  (One-tile
// CTAs, two an SM, overlap already: persistent ones took 5 to 17% longer.)  The
// rule asks for the caller's bound on the lengths to be some windows; one limit
// serves both head sizes, though at d = 64 it leaves 5% of window 2048.  In us,
// one CTA an item / persistent (32 / 8 heads, N = 16384, B = 1; the last two 16 / 4
// heads, B = 8):
//   d    window 512   1024        2048        4096        N 2048, 512  N 2048, 1024
//   128  187 / 165    261 / 246   400 / 400   658 / 687   98 / 93      119 / 121
//   64   160 / 138    222 / 202   341 / 325   558 / 556   83 / 78      101 / 101
// Items that are not alike and bounds that are loose gain as well (16 / 4 heads,
// d = 128, windows 128, 512, 1024): 32 sequences of 64 to 4096 226 / 193, 312 /
// 287, 404 / 406; 64 of 256 to 512 with a bound of 16384 111 / 97, 119 / 105, 119 /
// 105; one of 16384 and 200 of 1 to 256, whose grid of one CTA an item is mostly
// empty, 1365 / 614, 1393 / 644, 1432 / 689.
constexpr int kPersistentKeys = 1536;

template <int D>
static cudaError_t launch_prefill_window_d(const CUtensorMap &tq, const CUtensorMap &tk,
                                           const CUtensorMap &tv, const CUtensorMap &tv1,
                                           const CUtensorMap &to, const PrefillParams &p, int kind,
                                           int grid, int longest, cudaStream_t stream) {
  const long long reach =
      static_cast<long long>(std::min(p.window, longest)) + std::min(p.sinks, longest);
  const bool persistent = grid > p.prefetch_ahead && reach <= kPersistentKeys &&
                          3 * reach <= static_cast<long long>(p.max_pairs) * kPrefillBM;
  switch (kind) {
    case kKindDenseHeads:
      return persistent
                 ? launch_prefill_t<D, true, kKindDenseHeads, false, 2, true, false, true>(
                       tq, tk, tv, tv1, to, p, grid, stream)
                 : launch_prefill_t<D, true, kKindDenseHeads, false, 2, true>(tq, tk, tv, tv1, to, p,
                                                                             grid, stream);
    case kKindVarlenHeads:
      return persistent
                 ? launch_prefill_t<D, true, kKindVarlenHeads, false, 2, true, false, true>(
                       tq, tk, tv, tv1, to, p, grid, stream)
                 : launch_prefill_t<D, true, kKindVarlenHeads, false, 2, true>(tq, tk, tv, tv1, to, p,
                                                                              grid, stream);
    case kKindPagedHeads:
      return launch_prefill_t<D, true, kKindPagedHeads, false, 2, true>(tq, tk, tv, tv1, to, p, grid,
                                                                       stream);
    case kKindDense:
      return launch_prefill_t<D, true, kKindDense, false, 1, true>(tq, tk, tv, tv1, to, p, grid,
                                                                  stream);
    case kKindVarlen:
      return launch_prefill_t<D, true, kKindVarlen, false, 1, true>(tq, tk, tv, tv1, to, p, grid,
                                                                   stream);
    default:
      return launch_prefill_t<D, true, kKindPaged, false, 1, true>(tq, tk, tv, tv1, to, p, grid,
                                                                  stream);
  }
}

// Head-pair kinds run two heads of a KV group over the same 128 rows per CTA;
// the others one query tile per CTA, so that every tile of a CTA has the same
// key tiles.  longest: the caller's bound on the sequences' keys.
cudaError_t launch_prefill_window(const CUtensorMap &tq, const CUtensorMap &tk,
                                  const CUtensorMap &tv, const CUtensorMap &tv1,
                                  const CUtensorMap &to, const PrefillParams &p, int d, int kind,
                                  int grid, int longest, cudaStream_t stream) {
  return d == 64 ? launch_prefill_window_d<64>(tq, tk, tv, tv1, to, p, kind, grid, longest, stream)
                 : launch_prefill_window_d<128>(tq, tk, tv, tv1, to, p, kind, grid, longest, stream);
}

}  // namespace fa
