// Rotary positions: the turn of a pair at a position, a few elements of a row
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

// Four consecutive elements as they are stored, in one load.
template <int TYPE>
struct Raw4 {
  uint2 w;
};
template <>
struct Raw4<TERN_F32> {
  float4 w;
};
template <int TYPE>
__device__ __forceinline__ Raw4<TYPE> raw4(const void* p, long long i) {
  if constexpr (TYPE == TERN_F32)
    return {*reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)};
  else
    return {*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i)};
}
template <int TYPE>
__device__ __forceinline__ void unpack4(const Raw4<TYPE>& r, float (&v)[4]) {
  if constexpr (TYPE == TERN_F32) {
    v[0] = r.w.x, v[1] = r.w.y, v[2] = r.w.z, v[3] = r.w.w;
  } else {
    const uint32_t w[2] = {r.w.x, r.w.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
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
__device__ __forceinline__ void store4(void* p, long long i, const float (&v)[4]) {
  if constexpr (TYPE == TERN_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (TYPE == TERN_BF16)
        w[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j]))) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v[2 * j + 1]))) << 16);
      else
        w[j] = static_cast<uint32_t>(__half_as_ushort(__float2half_rn(v[2 * j]))) |
               (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(v[2 * j + 1]))) << 16);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(w[0], w[1]);
  }
}

// A thread's unit of a head's row: two groups of four elements, from a and from b
// on.  In the half layout they are the two sides of four pairs; else they follow
// each other and hold four pairs side by side, or elements that do not turn.
// Unit u of dim / 8.
struct RopeUnit {
  int a, b;
  int pair;  // the first of its four pairs; -1: none, the elements stay
  __device__ __forceinline__ RopeUnit(const RopeArgs& r, int u) {
    const bool turns = 8 * u < r.rotary;
    const bool half = turns && !r.interleaved;
    a = half ? 4 * u : 8 * u;
    b = half ? (r.rotary >> 1) + 4 * u : 8 * u + 4;
    pair = turns ? 4 * u : -1;
  }
};

// Heads whose elements a thread has in flight at a time.
constexpr int kRopeBatch = 4;

// A unit of kRopeBatch heads, from head h0 on and `step` apart: loaded, then turned
// (with turns made while the loads are on their way) and stored.  (A load may not
// pass the stores before it, which it may alias: head by head, each would wait for
// the one before.)
template <int TYPE>
struct RopeHeads {
  Raw4<TYPE> u[kRopeBatch], v[kRopeBatch];
  __device__ __forceinline__ void load(const RopeUnit& unit, const void* x, long long row,
                                       long long hd, int h0, int step, int heads) {
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      if (h0 + k * step >= heads) continue;
      const long long from = row + (h0 + k * step) * hd;
      u[k] = raw4<TYPE>(x, from + unit.a);
      v[k] = raw4<TYPE>(x, from + unit.b);
    }
  }
  template <int OUT>
  __device__ __forceinline__ void store(const RopeArgs& rope, const RopeUnit& unit,
                                        const float2 (&turn)[4], void* out, long long row,
                                        long long hd, int h0, int step, int heads) const;
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

// The four pairs' (cos, sin) at a position, times the magnitude.  Negative
// positions turn backwards.
__device__ __forceinline__ void rope_turns(const RopeArgs& r, int pair, int pos, float2 (&t)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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
__device__ __forceinline__ void rope_apply(const RopeArgs& r, const float2 (&t)[4], float (&a)[4],
                                           float (&b)[4]) {
  if (r.interleaved) {
    rope_pair(t[0], a[0], a[1]);
    rope_pair(t[1], a[2], a[3]);
    rope_pair(t[2], b[0], b[1]);
    rope_pair(t[3], b[2], b[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) rope_pair(t[i], a[i], b[i]);
  }
}

template <int TYPE>
template <int OUT>
__device__ __forceinline__ void RopeHeads<TYPE>::store(const RopeArgs& rope, const RopeUnit& unit,
                                                       const float2 (&turn)[4], void* out,
                                                       long long row, long long hd, int h0, int step,
                                                       int heads) const {
#pragma unroll
  for (int k = 0; k < kRopeBatch; ++k) {
    if (h0 + k * step >= heads) continue;
    float a[4], b[4];
    unpack4<TYPE>(u[k], a);
    unpack4<TYPE>(v[k], b);
    if (unit.pair >= 0) rope_apply(rope, turn, a, b);
    const long long to = row + (h0 + k * step) * hd;
    store4<OUT>(out, to + unit.a, a);
    store4<OUT>(out, to + unit.b, b);
  }
}

}  // namespace tern
