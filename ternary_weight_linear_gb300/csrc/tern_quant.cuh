// Per-token int8 codes: the quantiser's arithmetic, shared by the kernels
// that make codes.
#pragma once

#include <stdint.h>

namespace tern {

// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

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

// The codes of four values, |v| <= 127 scale, as bytes.  r = v * inv rounded
// to an integer (by adding 1.5 * 2^23, whose last place is 1) leaves the code
// in the sum's low byte; where every v * inv lies farther than kQMargin from
// the half-integers the four are the codes, as above; else each takes
// quant_code.
__device__ __forceinline__ uint32_t quant_codes4(float v0, float v1, float v2, float v3,
                                                 float scale, float inv, bool fast) {
  constexpr float kMagic = 12582912.f;
  const float m0 = fmaf(v0, inv, kMagic), m1 = fmaf(v1, inv, kMagic);
  const float m2 = fmaf(v2, inv, kMagic), m3 = fmaf(v3, inv, kMagic);
  const float far = fmaxf(fmaxf(fabsf(fmaf(v0, inv, kMagic - m0)), fabsf(fmaf(v1, inv, kMagic - m1))),
                          fmaxf(fabsf(fmaf(v2, inv, kMagic - m2)), fabsf(fmaf(v3, inv, kMagic - m3))));
  uint32_t c0 = __float_as_uint(m0), c1 = __float_as_uint(m1);
  uint32_t c2 = __float_as_uint(m2), c3 = __float_as_uint(m3);
  if (!(fast && far < 0.5f - kQMargin)) {
    c0 = static_cast<uint32_t>(static_cast<int>(quant_code(v0, scale, inv, fast)));
    c1 = static_cast<uint32_t>(static_cast<int>(quant_code(v1, scale, inv, fast)));
    c2 = static_cast<uint32_t>(static_cast<int>(quant_code(v2, scale, inv, fast)));
    c3 = static_cast<uint32_t>(static_cast<int>(quant_code(v3, scale, inv, fast)));
  }
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
}
__device__ __forceinline__ uint2 quant_codes8(const float (&v)[8], float scale, float inv,
                                              bool fast) {
  const uint32_t lo = quant_codes4(v[0], v[1], v[2], v[3], scale, inv, fast);
  return make_uint2(lo, quant_codes4(v[4], v[5], v[6], v[7], scale, inv, fast));
}

}  // namespace tern
