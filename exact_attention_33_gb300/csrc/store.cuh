// store.cuh - tiles held in registers, a row per lane, to rows of bf16 in memory.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fa {

// Writes one half (D / 2 columns) of the 128 rows of a tile as bf16 times
// `mul`: lane l holds its row's half, fp32 from TMEM in v (32 columns per
// v[c]).  Row by row (one row per lane) a warp's 16-byte stores would touch
// 32 rows at once; instead the lanes of each group of NCH = D / 16 exchange
// 16-byte chunks (an NCH x NCH transpose by xor butterflies), so that store
// i of lane l writes chunk l % NCH of the group's row i and every store
// instruction covers 32 / NCH whole half-rows.  `row_ptr` is this lane's
// half-row, `row_step` the elements from one row to the next (the rows of a
// tile are consecutive); a row whose lane has `row_ok` false is not written.
template <int D>
__device__ __forceinline__ void store_half_rows_bf16(uint16_t *row_ptr, size_t row_step,
                                                     bool row_ok, const uint32_t (&v)[D / 64][32],
                                                     float mul) {
  constexpr int NCH = D / 16;
  const int lane = threadIdx.x & 31;
  uint32_t x[NCH][4];  // chunk c: columns [8c, 8c + 8) of the half
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int k = 8 * c + 2 * w;
      x[c][w] = pack_bf16x2(__uint_as_float(v[k / 32][k % 32]) * mul,
                            __uint_as_float(v[k / 32][k % 32 + 1]) * mul);
    }
  // after the stages lane (base + t) holds chunk t of row (base + c) in x[c]
#pragma unroll
  for (int sft = NCH / 2; sft > 0; sft >>= 1) {
    const bool hi = (lane & sft) != 0;
#pragma unroll
    for (int c0 = 0; c0 < NCH; ++c0) {
      if (c0 & sft) continue;
      const int c1 = c0 | sft;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, hi ? x[c0][w] : x[c1][w], sft);
        if (hi)
          x[c0][w] = recv;
        else
          x[c1][w] = recv;
      }
    }
  }
  const unsigned ok_rows = __ballot_sync(0xffffffffu, row_ok);
  const int sub = lane % NCH, base = lane - sub;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if ((ok_rows >> (base + i)) & 1u) {
      uint16_t *dst = row_ptr + static_cast<ptrdiff_t>(base + i - lane) * static_cast<ptrdiff_t>(row_step) +
                      sub * 8;
      *reinterpret_cast<uint4 *>(dst) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
    }
  }
}

}  // namespace fa
