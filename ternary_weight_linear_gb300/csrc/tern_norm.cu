// tern_add_rmsnorm_s8: the residual's addition, the root-mean-square norm and
// the s8 rung's int8 codes of a token row, in one pass:
//   r = round(x + res);  y = (r w) (mean(r^2) + eps)^-1/2;
//   xs = max|y| / 127;   q = clamp(rint(y / xs), -127, 127).
//
// One CTA per token, the whole row in registers: every input byte is read
// once and every output byte written once, so a prompt's call is bound by
// HBM (9 bytes per element with fp32 x and bf16 residuals).  The row's mean
// square and its largest |y| come out of the same reduction: rounding is
// monotonic, so max|(r w) inv| = max|r w| inv exactly, and one barrier
// separates the loads from the stores.  A single token is bound by that
// latency chain (launch, one load round trip, one barrier, the stores).
// A thread holds as few of the row's vectors as a CTA of 1024 allows: with two
// each and half the threads the 2048 rows below take 20.5 us (each thread's
// chain of loads, sums and stores is longer, and no more of them are resident).
// 32 registers a thread keep three CTAs of 640 threads on an SM; with 41 the
// same rows take 21.8 us.
//
// Measured (width 5120, fp32 x, bf16 residual and weight): one token 2.6 us;
// 2048 tokens 19.0 us, 4.96 TB/s (0.73 of the copy rate); 4096 tokens with y
// 37.8 us, 6.1 TB/s (0.90): some 4 us of each call start and drain the SMs.
#include <cuda_bf16.h>

#include "tern.h"
#include "tern_device.cuh"
#include "tern_internal.h"
#include "tern_quant.cuh"

namespace tern {
namespace {

// Eight elements of a row.
struct F8 {
  float v[8];
};

// Elements i .. i + 7 of p, fp32 or bf16, in 16-byte loads.
template <int TYPE>
__device__ __forceinline__ F8 load8(const void* p, long long i) {
  F8 r;
  if constexpr (TYPE == TERN_F32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
    r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[2 * j] = __uint_as_float(w[j] << 16);
      r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}

// Rounds r to the residual's type (in place) and stores it.
template <int TYPE>
__device__ __forceinline__ void round_store8(F8& r, void* p, long long i) {
  if constexpr (TYPE == TERN_F32) {
    if (p) {
      float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      f[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
      f[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
    }
  } else {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = pack_bf16(r.v[2 * j], r.v[2 * j + 1]);
      r.v[2 * j] = __uint_as_float(u[j] << 16);
      r.v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
    if (p)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

constexpr int kNoResidual = -1;

// XT, RT: types of x and of the residual (kNoResidual: none; the norm then
// runs on x itself).  NV: vectors of eight elements per thread.
template <int XT, int RT, int NV>
__global__ void __launch_bounds__(1024, NV == 1 ? 2 : 1)
    add_rmsnorm_kernel(const NormArgs a) {
  grid_dependents_launch();
  __shared__ float red_s[32], red_m[32];
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = a.K >> 3;
  const long long row = static_cast<long long>(t) * a.K;
  const long long xrow = static_cast<long long>(t) * a.x_ld;
  grid_dependency_wait();  // the inputs and the output buffers come from earlier work
  F8 r[NV];
  float sum = 0.f, big = 0.f;
  // one or two vectors' loads in flight per thread before their arithmetic
  // (more would not fit the registers of a 1024-thread CTA)
  constexpr int kBatch = NV == 2 ? 2 : 1;
#pragma unroll
  for (int j0 = 0; j0 < NV; j0 += kBatch) {
    F8 res[kBatch], w[kBatch];
    if (j0 > 0) asm volatile("" ::: "memory");  // keeps the next loads here
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = threadIdx.x + (j0 + k) * blockDim.x;
      if (i < vecs) {
        r[j0 + k] = load8<XT>(a.x, xrow + 8ll * i);
        if constexpr (RT != kNoResidual) res[k] = load8<RT>(a.residual, row + 8ll * i);
        w[k] = a.weight_type == TERN_F32 ? load8<TERN_F32>(a.weight, 8ll * i)
                                         : load8<TERN_BF16>(a.weight, 8ll * i);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      F8& rj = r[j0 + k];
      const int i = threadIdx.x + (j0 + k) * blockDim.x;
      if (i < vecs) {
        if constexpr (RT != kNoResidual) {
#pragma unroll
          for (int e = 0; e < 8; ++e) rj.v[e] += res[k].v[e];
          round_store8<RT>(rj, a.residual_out, row + 8ll * i);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum = fmaf(rj.v[e], rj.v[e], sum);
          rj.v[e] *= w[k].v[e];
          big = max_nan(big, fabsf(rj.v[e]));  // (the weight's NaN is not in the sum)
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
  }
  if (lane == 0) {
    red_s[warp] = sum;
    red_m[warp] = big;
  }
  __syncthreads();
  {
    // every warp adds the warps' sums in the same order
    const int warps = blockDim.x >> 5;
    sum = lane < warps ? red_s[lane] : 0.f;
    big = lane < warps ? red_m[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      big = max_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
    }
  }
  const float inv = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  const float amax = big * inv;
  const float scale = amax / 127.0f;  // IEEE single-precision division
  if (a.q && threadIdx.x == 0) a.x_scale[t] = scale;
  const float sinv = 1.0f / scale;
  const bool fast = quant_fast(scale);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < vecs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j].v[e] *= inv;
      if (a.y)
        *reinterpret_cast<uint4*>(a.y + row + 8ll * i) =
            make_uint4(pack_bf16(r[j].v[0], r[j].v[1]), pack_bf16(r[j].v[2], r[j].v[3]),
                       pack_bf16(r[j].v[4], r[j].v[5]), pack_bf16(r[j].v[6], r[j].v[7]));
      if (a.q) {
        uint2 out = make_uint2(0u, 0u);
        if (amax > 0.f) out = quant_codes8(r[j].v, scale, sinv, fast);
        *reinterpret_cast<uint2*>(a.q + row + 8ll * i) = out;
      }
    }
  }
}

template <int XT, int RT, int NV>
cudaError_t launch_one(const NormArgs& a, int threads, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_launch_config(attr, dim3(static_cast<unsigned>(a.T)), dim3(threads), 0, stream);
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<XT, RT, NV>, a);
}

template <int XT, int RT>
cudaError_t launch_types(const NormArgs& a, cudaStream_t stream) {
  const int vecs = a.K / 8;
  auto threads = [&](int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; };
  if (vecs <= 1024) return launch_one<XT, RT, 1>(a, threads(1), stream);
  if (vecs <= 2048) return launch_one<XT, RT, 2>(a, threads(2), stream);
  return launch_one<XT, RT, 4>(a, threads(4), stream);
}

// tern_norm_add_norm_s8: the norm after a block, its gate, the residual's
// addition and the norm before the next block:
//   n = (x w1) (mean(x^2) + eps)^-1/2;    r = round(a res + b g n);
//   y = (r w2) (mean(r^2) + eps)^-1/2;    codes and scale of y as above.
// The same plan with a second reduction: one CTA per token, the row in
// registers from the first load to the last store, so every input is read and
// every output written once.  Rows of one and two vectors a thread load the residual
// before the first barrier, those of four, whose registers are the row's, behind it, as
// all do with the weights and the gate, which other tokens' CTAs have left in L1.
// Bound by instructions: 2048 rows of 5120, fp32 x, a gate a channel, bf16 weights
// take 22.5 us (their bytes 13.9 at the copy rate; the issue slots were 67 % busy at
// 25.5), 41.8 with all loads before the barrier, whose 56 registers left one CTA of
// 640 threads an SM.  kBf16: weights and gate are all bf16, which saves the choice
// at each load, 2 us of it.
template <int XT, int RT, int NV, bool kBf16>
__global__ void __launch_bounds__(1024, NV == 1 ? 2 : 1)
    norm_pair_kernel(const NormPairArgs a) {
  grid_dependents_launch();
  __shared__ float red_x[32], red_s[32], red_m[32];
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = a.K >> 3, warps = blockDim.x >> 5;
  const long long row = static_cast<long long>(t) * a.K;
  const long long xrow = static_cast<long long>(t) * a.x_ld;
  const long long grow = static_cast<long long>(t) * a.gate_ld;
  auto weight8 = [](const void* p, int type, long long i) {
    return !kBf16 && type == TERN_F32 ? load8<TERN_F32>(p, i) : load8<TERN_BF16>(p, i);
  };
  constexpr bool kEarly = NV <= 2;
  grid_dependency_wait();  // the inputs and the output buffers come from earlier work
  F8 r[NV], res[kEarly ? NV : 1];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < vecs) {
      r[j] = load8<XT>(a.x, xrow + 8ll * i);
      if (kEarly) res[j] = load8<RT>(a.residual, row + 8ll * i);
      uint64_t s2 = 0;  // pairs of sums from +0
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint64_t x = pair_f32(r[j].v[e], r[j].v[e + 1]);
        s2 = fma_pair(x, x, s2);
      }
      float s0, s1;
      unpair_f32(s2, s0, s1);
      sum += s0 + s1;
    }
  }
  float inv = 1.f;  // of the block's output, with the branch's scale below
  if (a.post) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red_x[warp] = sum;
    __syncthreads();
    sum = lane < warps ? red_x[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = rsqrtf(sum * a.inv_k + a.eps);
  }
  inv *= a.branch_scale;
  sum = 0.f;
  float big = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < vecs) {
      // (the barriers to the compiler keep the loads out of each other's registers,
      // which there are not enough of)
      if (NV != 2) asm volatile("" ::: "memory");
      F8& rs = res[kEarly ? j : 0];
      if (!kEarly) rs = load8<RT>(a.residual, row + 8ll * i);
      auto times = [&](const F8& f) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          unpair_f32(mul_pair(pair_f32(r[j].v[e], r[j].v[e + 1]), pair_f32(f.v[e], f.v[e + 1])),
                     r[j].v[e], r[j].v[e + 1]);
      };
      if (a.post) times(weight8(a.post, a.post_type, 8ll * i));
      if (a.gate) times(weight8(a.gate, a.gate_type, grow + 8ll * i));
      const uint64_t inv2 = pair_f32(inv, inv);
      const uint64_t rs2 = pair_f32(a.residual_scale, a.residual_scale);
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        unpair_f32(fma_pair(pair_f32(r[j].v[e], r[j].v[e + 1]), inv2,
                            mul_pair(pair_f32(rs.v[e], rs.v[e + 1]), rs2)),
                   r[j].v[e], r[j].v[e + 1]);
      if (NV != 2) asm volatile("" ::: "memory");
      const F8 w = weight8(a.weight, a.weight_type, 8ll * i);
      round_store8<RT>(r[j], a.residual_out, row + 8ll * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(r[j].v[e], r[j].v[e], sum);
      times(w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        big = max_nan(big, fabsf(r[j].v[e]));  // (the weight's NaN is not in the sum)
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  big = warp_max_nan(big);
  if (lane == 0) {
    red_s[warp] = sum;
    red_m[warp] = big;
  }
  __syncthreads();
  sum = lane < warps ? red_s[lane] : 0.f;
  big = warp_max_nan(lane < warps ? red_m[lane] : 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  inv = 1.0f / sqrtf(sum / static_cast<float>(a.K) + a.eps);
  const float amax = big * inv;
  const float scale = amax / 127.0f;  // IEEE single-precision division
  if (a.q && threadIdx.x == 0) a.x_scale[t] = scale;
  const float sinv = 1.0f / scale;
  const bool fast = quant_fast(scale);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < vecs) {
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        unpair_f32(mul_pair(pair_f32(r[j].v[e], r[j].v[e + 1]), pair_f32(inv, inv)), r[j].v[e],
                   r[j].v[e + 1]);
      if (a.y)
        *reinterpret_cast<uint4*>(a.y + row + 8ll * i) =
            make_uint4(pack_bf16(r[j].v[0], r[j].v[1]), pack_bf16(r[j].v[2], r[j].v[3]),
                       pack_bf16(r[j].v[4], r[j].v[5]), pack_bf16(r[j].v[6], r[j].v[7]));
      if (a.q) {
        uint2 out = make_uint2(0u, 0u);
        if (amax > 0.f) {
          const float lo[4] = {r[j].v[0], r[j].v[1], r[j].v[2], r[j].v[3]};
          const float hi[4] = {r[j].v[4], r[j].v[5], r[j].v[6], r[j].v[7]};
          out.x = quant_codes4_short(lo, scale, sinv, fast);
          out.y = quant_codes4_short(hi, scale, sinv, fast);
        }
        *reinterpret_cast<uint2*>(a.q + row + 8ll * i) = out;
      }
    }
  }
}

template <int XT, int RT, int NV>
cudaError_t launch_pair_one(const NormPairArgs& a, int threads, cudaStream_t stream) {
  const bool bf16 = a.weight_type == TERN_BF16 && (!a.post || a.post_type == TERN_BF16) &&
                    (!a.gate || a.gate_type == TERN_BF16);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_launch_config(attr, dim3(static_cast<unsigned>(a.T)), dim3(threads), 0, stream);
  return cudaLaunchKernelEx(
      &cfg, bf16 ? norm_pair_kernel<XT, RT, NV, true> : norm_pair_kernel<XT, RT, NV, false>, a);
}

template <int XT, int RT>
cudaError_t launch_pair_types(const NormPairArgs& a, cudaStream_t stream) {
  const int vecs = a.K / 8;
  auto threads = [&](int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; };
  if (vecs <= 1024) return launch_pair_one<XT, RT, 1>(a, threads(1), stream);
  if (vecs <= 2048) return launch_pair_one<XT, RT, 2>(a, threads(2), stream);
  return launch_pair_one<XT, RT, 4>(a, threads(4), stream);
}

}  // namespace

cudaError_t launch_add_rmsnorm_s8(const NormArgs& a, cudaStream_t stream) {
  const int rt = a.residual ? a.residual_type : kNoResidual;
#define TERN_NORM_CASE(XT, RT) \
  if (a.x_type == XT && rt == RT) return launch_types<XT, RT>(a, stream);
  TERN_NORM_CASE(TERN_F32, TERN_BF16)
  TERN_NORM_CASE(TERN_F32, TERN_F32)
  TERN_NORM_CASE(TERN_F32, kNoResidual)
  TERN_NORM_CASE(TERN_BF16, TERN_BF16)
  TERN_NORM_CASE(TERN_BF16, TERN_F32)
  TERN_NORM_CASE(TERN_BF16, kNoResidual)
#undef TERN_NORM_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_add_norm_s8(const NormPairArgs& a, cudaStream_t stream) {
#define TERN_NORM_CASE(XT, RT) \
  if (a.x_type == XT && a.residual_type == RT) return launch_pair_types<XT, RT>(a, stream);
  TERN_NORM_CASE(TERN_F32, TERN_BF16)
  TERN_NORM_CASE(TERN_F32, TERN_F32)
  TERN_NORM_CASE(TERN_BF16, TERN_BF16)
  TERN_NORM_CASE(TERN_BF16, TERN_F32)
#undef TERN_NORM_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tern
