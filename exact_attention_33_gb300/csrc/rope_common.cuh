// rope_common.cuh - angles of rotary positions, and rows turned by them.
//
// p * inv_freq is wanted to about 2^-24 of a radian at any position, and the
// product in fp32 is off by 2^-24 of itself (at position 10^6 by 0.06 rad).
// So turns a position, inv_freq / 2 pi, are made a 64-bit fraction of a turn,
// and the product with a position is one integer multiplication: it wraps at
// whole turns by itself and is exact.  Its upper 56 bits go into sin and cos.  The
// fraction is formed in integers too: with the few fp64 instructions that it takes
// otherwise, this GPU's fp64 rate bound every kernel here (73 k packed tokens of 16 / 4
// heads of d = 128, both directions, 261 us against 232; 34.8 k tokens into the 8-bit
// cache 343 us against 148).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fa {

// Turns a position, inv_freq / (2 pi), as a fraction of 2^64, whole turns left
// out.  inv_freq = m 2^(e - 1075) with a 53-bit m, 1 / (2 pi) = K 2^-66.
__device__ __forceinline__ uint64_t rope_turns(double inv_freq) {
  constexpr uint64_t K = 0xa2f9836e4e44152aull;  // 2^65 / pi
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int e = static_cast<int>(bits >> 52) & 0x7FF;
  uint64_t m = bits & 0xFFFFFFFFFFFFFull;
  if (e != 0) m |= 1ull << 52;
  const uint64_t hi = __umul64hi(m, K), lo = m * K;
  const int s = 1077 - max(e, 1);  // turns 2^64 = (hi 2^64 + lo) 2^-s
  uint64_t t = 0;
  if (s >= 64)
    t = s < 128 ? hi >> (s - 64) : 0;
  else if (s > 0)
    t = (hi << (64 - s)) | (lo >> s);
  else if (s > -64)
    t = lo << -s;
  return bits >> 63 ? 0 - t : t;
}

// sin and cos of v + below 2^-32 (2^-32 turns), at most an eighth of a turn either
// way: the angle in two floats t + tl, the Taylor series' terms behind the first one
// (of cos: behind 1 - t^2 / 2, also in two floats) with their rounding errors and tl
// added to it last.  t is of the nearest multiple of 128, so that small angles of
// either sign lie in tl alone and nothing cancels.  So there is little but the last
// rounding: 0.29 units in the last place root mean square; sin is within 3.1 x 2^-24
// of itself from 2^-32 of a turn up (1.2 units above 64 x 2^-32) and within 2^-54 of a
// turn below, cos within 2^-24.  Keys on their way to e4m3 whose code is not that of
// the exact product are so 1.09 in a million, with sincospif 1.33 (50 million counted);
// the calls take the same time.
__device__ __forceinline__ void sin_cos_eighth(int32_t v, uint32_t below, float &s, float &c) {
  constexpr float K = 0x1.921fb6p-30f, Kl = -0x1.777a5cp-55f;  // 2 pi 2^-32
  const int32_t near = (v + 64) & ~127;
  const float vh = static_cast<float>(near);
  // what is left, in 2^-24ths of v's units
  const float vl = static_cast<float>(static_cast<int32_t>(
      __funnelshift_l(below, static_cast<uint32_t>(v - near), 24)));
  const float t = vh * K;
  const float tl = fmaf(vh, K, -t) + fmaf(vh, Kl, vl * (K * 0x1p-24f));
  const float w = t * t, wl = fmaf(t, t, -w);
  const float h = fmaf(-0.5f, w, 1.f);  // 1 - w / 2
  float q = fmaf(w, 1.f / 362880.f, -1.f / 5040.f);
  q = fmaf(w, q, 1.f / 120.f);
  q = fmaf(w, q, -1.f / 6.f);
  s = t + fmaf(tl, h, t * w * q);
  q = fmaf(w, -1.f / 3628800.f, 1.f / 40320.f);
  q = fmaf(w, q, -1.f / 720.f);
  q = fmaf(w, q, 1.f / 24.f);
  const float hl = fmaf(-0.5f, w, 1.f - h);
  c = h + fmaf(w * w, q, fmaf(-t, tl, fmaf(-0.5f, wl, hl)));
}

// cos and sin of p positions' turns: the nearest quarter of a turn by signs and
// places, the rest as above.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turns, int p) {
  const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(p));
  const uint32_t hi = static_cast<uint32_t>(a >> 32);  // 2^32 of a turn
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  float s, c;
  sin_cos_eighth(static_cast<int32_t>(hi - (quarter << 30)), static_cast<uint32_t>(a), s, c);
  const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
  return make_float2((quarter + 1u) & 2u ? -x : x, quarter & 2u ? -y : y);
}

// A head row of D values is D / 16 units of two 16-byte pieces: 8 pairs (half
// layout: a piece of each half; interleaved: neighbours), or 16 values that pass
// through.
struct RopeUnit {
  bool turns;  // the unit's values are rotated
  int o0, o1;  // where its pieces start in the row
  __device__ __forceinline__ RopeUnit(int u, int pairs, bool interleaved) {
    turns = u < pairs / 8;
    o0 = turns && !interleaved ? 8 * u : 16 * u;
    o1 = turns && !interleaved ? pairs + 8 * u : 16 * u + 8;
  }
};

// cos and sin of a unit's 8 pairs, by two's.
struct UnitAngles {
  float2 c[4], s[4];

  // of_pair(i): (cos, sin) of pair i
  template <typename OfPair>
  __device__ __forceinline__ void set(OfPair of_pair) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = of_pair(2 * i), y = of_pair(2 * i + 1);
      c[i] = make_float2(x.x, y.x);
      s[i] = make_float2(x.y, y.y);
    }
  }
};

// A unit's pieces x and y, rotated in fp32: v[0..3] are piece x's values by
// two's, v[4..7] piece y's.
template <bool INTER>
__device__ __forceinline__ void rotate_unit(const UnitAngles &t, const uint4 &x, const uint4 &y,
                                            float2 (&v)[8]) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (INTER) {
      // word w of x is pair w, of y pair 4 + w
      const float2 p = bf16x2_to_float2(a[w]), q = bf16x2_to_float2(b[w]);
      const float pc = w & 1 ? t.c[w / 2].y : t.c[w / 2].x, ps = w & 1 ? t.s[w / 2].y : t.s[w / 2].x;
      const float qc = w & 1 ? t.c[2 + w / 2].y : t.c[2 + w / 2].x;
      const float qs = w & 1 ? t.s[2 + w / 2].y : t.s[2 + w / 2].x;
      v[w] = make_float2(fmaf(p.x, pc, -(p.y * ps)), fmaf(p.x, ps, p.y * pc));
      v[4 + w] = make_float2(fmaf(q.x, qc, -(q.y * qs)), fmaf(q.x, qs, q.y * qc));
    } else {
      // word w of x holds the a's of pairs 2w and 2w + 1, that of y their b's
      const float2 p = bf16x2_to_float2(a[w]), q = bf16x2_to_float2(b[w]);
      const float2 ns = make_float2(-t.s[w].x, -t.s[w].y);
      v[w] = ffma2(p, t.c[w], fmul2(q, ns));
      v[4 + w] = ffma2(p, t.s[w], fmul2(q, t.c[w]));
    }
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float2 *v) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                    pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
}

}  // namespace fa
