// Per-token int8 codes: the quantiser's arithmetic, shared by the kernels
// that make codes.
#pragma once

#include <stdint.h>

namespace tern {

// Per-token code of v: rint(v / scale) clamped to [-127, 127], the quotient
// rounded as one IEEE single-precision division (nearest-even, as rint).
// Without a division per element: with inv = 1 / scale rounded, q0 = v * inv
// differs from v / scale by less than 128 * (2^-23 + 2^-48) < 1.53e-5 (|v| <=
// absmax, so |v / scale| < 128; two roundings of relative error 2^-24 each),
// and the rounded quotient from v / scale by at most half an ulp below 128,
// 2^-18; so the two are less than kQMargin = 2^-15 apart.  When q0 lies
// farther than kQMargin from every half-integer, both fall strictly inside
// the same rounding interval and rint(q0) is the code; otherwise the element
// takes the division.  fast: scale and 1 / scale normal (absmax >= 127 *
// 2^-126), where those relative bounds hold; else every element divides.
constexpr float kQMargin = 3.0517578125e-05f;  // 2^-15
__device__ __forceinline__ float quant_code(float v, float scale, float inv, bool fast) {
  float r;
  if (fast) {
    const float q0 = v * inv;
    r = rintf(q0);
    if (!(fabsf(q0 - r) < 0.5f - kQMargin)) r = rintf(v / scale);
  } else {
    r = rintf(v / scale);
  }
  return fminf(fmaxf(r, -127.f), 127.f);
}
__device__ __forceinline__ bool quant_fast(float scale) {
  return scale >= 1.1754943508222875e-38f && scale < 8.507059173023462e+37f;  // [2^-126, 2^126)
}

}  // namespace tern
