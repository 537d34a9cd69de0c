// rope_common.cuh - angles of rotary positions.
//
// p * inv_freq is wanted to about 2^-24 of a radian at any position, and the
// product in fp32 is off by 2^-24 of itself (at position 10^6 by 0.06 rad);
// fp64 is slow on this GPU.  So turns a position, inv_freq / 2 pi, are made a
// 64-bit fraction of a turn once for a thread, and the product with a position
// is one integer multiplication: it wraps at whole turns by itself and is
// exact.  Its upper half, 2^-32 of a turn, goes to sincospi.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// Turns a position as a fraction of 2^64 (whole turns left out).
__device__ __forceinline__ uint64_t rope_turns(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of p positions' turns.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turns, int p) {
  const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(p));
  float s, c;
  // (as a signed fraction: half a turn either way, in units of half a turn)
  sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f, &s, &c);
  return make_float2(c, s);
}

}  // namespace fa
