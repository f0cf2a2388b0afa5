// Rotary positions: the turn of a pair at a position, eight elements of a row
// in registers, and the arguments that the kernels which rotate share.
//
// Pair i of a head's first `rotary` elements is turned by position * freq[i],
// freq in turns a token.  It is held in units of 2^-64 of a turn, so that
// position * freq modulo one turn is the low 64 bits of an integer product:
// exact at every position (an angle in fp32 is off by 2^-24 of itself, 0.06
// radians at a million).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tern.h"
#include "tern_internal.h"

namespace tern {

// Eight consecutive elements i .. i + 7 of p, 16-byte loads.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, long long i, float (&v)[8]) {
  if constexpr (TYPE == TERN_F32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == TERN_BF16) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        v[2 * j] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[j])));
        v[2 * j + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[j] >> 16)));
      }
    }
  }
}

// And back, rounded once to nearest even.
template <int TYPE>
__device__ __forceinline__ void store8(void* p, long long i, const float (&v)[8]) {
  if constexpr (TYPE == TERN_F32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == TERN_BF16)
        w[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j]))) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j + 1]))) << 16);
      else
        w[j] = static_cast<uint32_t>(__half_as_ushort(__float2half_rn(v[2 * j]))) |
               (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(v[2 * j + 1]))) << 16);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A thread's unit of a head's row: two groups of eight elements, from a and
// from b on.  In the half layout they are the two sides of eight pairs; else
// they follow each other and hold eight pairs side by side, or elements that do
// not turn.  Unit u of dim / 16.
struct RopeUnit {
  int a, b;
  int pair;  // the first of its eight pairs; -1: none, the elements stay
  __device__ __forceinline__ RopeUnit(const RopeArgs& r, int u) {
    const bool turns = 16 * u < r.rotary;
    const bool half = turns && !r.interleaved;
    a = half ? 8 * u : 16 * u;
    b = half ? (r.rotary >> 1) + 8 * u : 16 * u + 8;
    pair = turns ? 8 * u : -1;
  }
};

// (cos, sin) of a turn in units of 2^-32: the quarter turn from its upper bits,
// the rest within an eighth of a turn to either side by Taylor's series, whose
// first terms left out are below 2^-29.  (Off by some 2^-23: the rest's
// rounding to fp32 and the sums'.)
__device__ __forceinline__ float2 turn_cos_sin(uint32_t turn) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) *
                  1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(z, s, 1.f / 120.f);
  s = fmaf(z, s, -1.f / 6.f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(z, c, -1.f / 720.f);
  c = fmaf(z, c, 1.f / 24.f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float cs = quarter & 1 ? -s : c, sn = quarter & 1 ? c : s;
  return quarter & 2 ? make_float2(-cs, -sn) : make_float2(cs, sn);
}

// The eight pairs' (cos, sin) at a position, times the magnitude.  Negative
// positions turn backwards.
__device__ __forceinline__ void rope_turns(const RopeArgs& r, int pair, int pos, float2 (&t)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t f = r.freq[pair + i];
    const uint32_t lo = static_cast<uint32_t>(f), p = static_cast<uint32_t>(pos);
    // bits 32 to 63 of f * pos
    uint32_t turn = __umulhi(lo, p) + static_cast<uint32_t>(f >> 32) * p;
    if (pos < 0) turn -= lo;
    t[i] = turn_cos_sin(turn);
    t[i].x *= r.magnitude;
    t[i].y *= r.magnitude;
  }
}

__device__ __forceinline__ void rope_pair(const float2 t, float& u, float& v) {
  const float x = u;
  u = fmaf(x, t.x, -(v * t.y));
  v = fmaf(x, t.y, v * t.x);
}

// Turns a unit's elements.
__device__ __forceinline__ void rope_apply(const RopeArgs& r, const float2 (&t)[8], float (&a)[8],
                                           float (&b)[8]) {
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rope_pair(t[i], a[2 * i], a[2 * i + 1]);
      rope_pair(t[4 + i], b[2 * i], b[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_pair(t[i], a[i], b[i]);
  }
}

}  // namespace tern
