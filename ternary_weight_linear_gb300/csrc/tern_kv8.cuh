// The int8 cache of keys and values as its kernels see it: arguments, checks
// of the index arrays, and which pages a sequence's query rows see.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tern.h"
#include "tern_device.cuh"
#include "tern_internal.h"

namespace tern {

constexpr int kBlk = TERN_KV8_BLOCK;

// A sequence of the batch.  ok: its entries are consistent.
struct KvSeq {
  int len, m, row0;  // tokens, new tokens, first row of q / k / v
  bool ok;
};

__device__ __forceinline__ KvSeq kv_seq(const Kv8Args& a, int b) {
  KvSeq s;
  s.len = a.lens[b];
  s.row0 = a.starts[b];
  const int end = a.starts[b + 1];
  s.ok = s.row0 >= 0 && end >= s.row0 && end <= a.rows;
  s.m = s.ok ? end - s.row0 : 0;
  s.ok = s.ok && s.len >= 0 && (static_cast<long long>(s.len) + kBlk - 1) / kBlk <= a.width &&
         s.m <= s.len && s.m <= a.max_new;
  return s;
}

// New token of row n (row = new token * group + head): n / group, by a
// multiplication (n < 2^31; see kv8_set_group).
__device__ __forceinline__ int kv_token(const Kv8Args& a, int n) {
  return static_cast<int>((__umulhi(static_cast<unsigned>(n), a.group_mul) +
                           static_cast<unsigned>(n)) >> a.group_shift);
}

// The pages that query positions [p0, p1] see: [0, sinks) then [first, last].
// Entry i of that list is page i or first + i - sinks.
struct KvPages {
  int sinks, first, count;
  __device__ __forceinline__ int page(int i) const { return i < sinks ? i : first + i - sinks; }
};

__device__ __forceinline__ KvPages kv_pages(const Kv8Args& a, int p0, int p1) {
  KvPages v;
  v.first = 0;
  v.sinks = 0;
  if (a.window > 0 && p0 >= a.window) {
    v.first = (p0 - a.window + 1) / kBlk;
    const int s = a.sinks / kBlk + (a.sinks % kBlk != 0);
    v.sinks = s < v.first ? s : v.first;
  }
  v.count = v.sinks + p1 / kBlk - v.first + 1;
  return v;
}

// Whether any row at positions [p0, p1] sees one of the tokens [j0, j1].
__device__ __forceinline__ bool kv_any(const Kv8Args& a, int p0, int p1, int j0, int j1) {
  return j0 <= p1 && (a.window == 0 || j1 > p0 - a.window || j0 < a.sinks);
}

// Whether every row at positions [p0, p1] sees all tokens [j0, j1].
__device__ __forceinline__ bool kv_all(const Kv8Args& a, int p0, int p1, int j0, int j1) {
  return j1 <= p0 && (a.window == 0 || j0 > p1 - a.window || j1 < a.sinks);
}

// A value scale as 2^e * f, f in [1, 2), for scales > 0 (subnormal ones too).
// Zero is kZeroExp: below every other exponent, so that 2^(e - E) is 0, whatever
// the block's codes are.
constexpr int kZeroExp = -100000, kNoExp = -150;  // kNoExp: below every scale's exponent
struct VScale {
  int e;
  float f;
};
__device__ __forceinline__ VScale split_vscale(float s) {
  if (s == 0.f) return {kZeroExp, 1.f};
  const bool sub = s < 1.17549435e-38f;  // 2^-126
  const uint32_t u = __float_as_uint(sub ? s * 16777216.f : s);
  return {static_cast<int>(u >> 23) - 127 - (sub ? 24 : 0),
          __uint_as_float((u & 0x007FFFFFu) | 0x3F800000u)};
}

// Whether a block's scales can be used: finite and not negative.  (A block
// whose scales cannot makes the rows that see it NaN, and only them.)
__device__ __forceinline__ bool good_scales(float ks, float vs) {
  return ks >= 0.f && ks < INFINITY && vs >= 0.f && vs < INFINITY;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// mbar_wait for loops that pass many barriers per microsecond: the time limit
// is kept with the SM's clock, which is read in some 20 cycles (%globaltimer
// takes about a microsecond, which every wait that did not succeed at once
// would pay).  Gives up after kWaitCycles, 2 s at the highest clock and
// longer below it.
constexpr long long kWaitCycles = 4140000000ll;
__device__ __forceinline__ bool mbar_wait_clk(uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    // (asleep for up to 20 us: attempts would take issue slots of the warps at
    // work)
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if (clock64() - t0 > kWaitCycles) {
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}

// Requests the 128-byte line of src into L2.
__device__ __forceinline__ void prefetch_l2(const void* src) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
}

// The lowest n bits of 64 (none for n <= 0, all for n >= 64).
__device__ __forceinline__ uint64_t bits_below(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
// A bit for each of the 64 tokens from j0 that the row at position p sees.
__device__ __forceinline__ uint64_t kv_mask(const Kv8Args& a, int p, int j0) {
  uint64_t see = bits_below(p - j0 + 1);
  if (a.window) see &= ~bits_below(p - a.window + 1 - j0) | bits_below(a.sinks - j0);
  return see;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two values as 16-bit words of the type.
__device__ __forceinline__ uint32_t pack_out(int type, float lo, float hi) {
  if (type != TERN_BF16) return half2_bits(lo, hi);
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}
// The two 16-bit elements of a word.
__device__ __forceinline__ void unpack16(uint32_t w, int type, float& lo, float& hi) {
  if (type == TERN_BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    lo = __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
    hi = __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16)));
  }
}

// Queries are held in fp16, each row scaled by a power of two that takes its
// largest element to [2^14, 2^15): exact for every element within 2^-31 of
// it.  big: the row's largest magnitude, as the bits of the type (which order
// as the magnitudes do).  The power's exponent is at most 126, so that it and
// its inverse are normal floats: rows below 2^-112 are scaled by less.
__device__ __forceinline__ int q_exponent(uint32_t big, int type) {
  if (big == 0) return 0;
  const uint32_t f = type == TERN_BF16
                         ? big << 16
                         : __float_as_uint(__half2float(
                               __ushort_as_half(static_cast<uint16_t>(big))));
  const int ex = static_cast<int>(f >> 23) - 127;
  return 14 - (ex < -112 ? -112 : ex);
}
__device__ __forceinline__ float pow2f(int x) {
  return __uint_as_float(static_cast<uint32_t>(x + 127) << 23);
}

// log sum_j exp(s_j) from the weights' reference (base 2; they are 2^off times
// larger) and sum.
__device__ __forceinline__ float kv_log_sum(float ref, float sum, float off) {
  return sum == 0.f ? -INFINITY : (ref - off + log2f(sum)) * 0.6931471805599453f;
}

// fp32 pairs in one 64-bit register (each half as its scalar instruction).
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 2^k as an fp16 bit pattern for k <= 0 (0 below the smallest subnormal).
__device__ __forceinline__ uint32_t half_pow2(int k) {
  return k >= -14 ? static_cast<uint32_t>(k + 15) << 10 : (k >= -24 ? 1u << (k + 24) : 0u);
}

}  // namespace tern
