// tern_kv8_append: new keys and values into the paged int8 cache.
//
// One CTA per (page that receives new tokens, keys | values, head): the page's
// new rows sit in registers, one reduction gives their absmax, the block's
// scale becomes max(old, absmax / 127) and the codes follow.  Where the scale
// grew, the codes of the older tokens are read and rounded to the new scale
// (a token's code is rounded once more per growth, each time by at most half
// a step of the scale then reached).  Every input is read once; a prompt is
// bound by HBM, a decode step by the latency of one load, one reduction and
// one store.  The rows are loaded beside the page table, which only the
// stores need.
//
// Measured (8 heads of 128): 16 sequences' decode step (bf16) 2.6 us; three
// ragged prompt chunks, 3554 tokens in fp32, 9.8 us, 3.7 TB/s (0.55 of the
// copy rate; 5 waves of CTAs, each a load, a reduction and a store).  Four
// CTAs an SM at 64 registers take as long as two at 90.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tern_kv8.cuh"
#include "tern_quant.cuh"

namespace tern {
namespace {

constexpr int kAppThreads = 256;

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

template <int TYPE, int D>
__global__ void __launch_bounds__(kAppThreads) kv8_append_kernel(const Kv8Args a) {
  grid_dependents_launch();
  grid_dependency_wait();  // every input and the cache come from earlier work
  constexpr int kChunks = D / 8;                       // vectors of a token
  constexpr int kTok = kAppThreads / kChunks;          // tokens per step
  constexpr int kSteps = kBlk / kTok;
  __shared__ float red[kAppThreads / 32];
  const int b = blockIdx.z;
  const int which = blockIdx.y & 1, h = blockIdx.y >> 1;
  const KvSeq s = kv_seq(a, b);
  if (!s.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  if (s.m == 0) return;
  const int begin = s.len - s.m;  // first new token
  const int pg = begin / kBlk + static_cast<int>(blockIdx.x);
  if (pg > (s.len - 1) / kBlk) return;
  const int page = a.table[static_cast<size_t>(b) * a.width + pg];
  const int first = begin > pg * kBlk ? begin - pg * kBlk : 0;       // new slots [first, last)
  const int last = s.len - pg * kBlk < kBlk ? s.len - pg * kBlk : kBlk;
  const int chunk = threadIdx.x % kChunks, slot0 = threadIdx.x / kChunks;
  const void* src = which ? a.v : a.k;

  float x[kSteps][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kTok;
    if (slot >= first && slot < last) {
      const long long row = s.row0 + static_cast<long long>(pg * kBlk + slot - begin);
      load8<TYPE>(src, row * a.ld + h * a.hd + 8 * chunk, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    }
  }
  // only now: the rows' loads need not wait for the table's
  if (page < 0 || page >= a.pages) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  const size_t blk = (static_cast<size_t>(page) * 2 + which) * a.hkv + h;
  int8_t* codes = a.codes + blk * (kBlk * D);
  const float old = first > 0 ? a.scales[blk] : 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(x[i][e]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppThreads / 32; ++i) amax = max_nan(amax, red[i]);
  float fresh = amax / 127.0f;                                     // IEEE division
  if (!(fresh < __uint_as_float(0x7F800000u))) fresh = __uint_as_float(0x7FC00000u);
  // a NaN on either side stays
  const bool grew = !(fresh <= old) && !(old != old);
  const float scale = grew ? fresh : old;
  if (threadIdx.x == 0 && (grew || first == 0)) a.scales[blk] = scale;
  const float inv = 1.0f / scale;
  const bool fast = quant_fast(scale);
  if (grew && first > 0) {
    const float ratio = old / scale;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int slot = slot0 + i * kTok;
      if (slot < first) {
        uint2* p = reinterpret_cast<uint2*>(codes + slot * D + 8 * chunk);
        const uint2 u = *p;
        uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t o = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float c = static_cast<float>(static_cast<int8_t>((w[j] >> (8 * e)) & 0xFFu));
            o |= (static_cast<uint32_t>(static_cast<int>(rintf(c * ratio))) & 0xFFu) << (8 * e);
          }
          w[j] = o;
        }
        *p = make_uint2(w[0], w[1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kTok;
    if (slot >= first && slot < last) {
      uint2 w = make_uint2(0u, 0u);
      if (scale > 0.f) w = quant_codes8(x[i], scale, inv, fast);
      *reinterpret_cast<uint2*>(codes + slot * D + 8 * chunk) = w;
    }
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, cudaStream_t stream, int* launches) {
  // m new tokens touch at most (m + 62) / 64 + 1 pages
  const unsigned pages = static_cast<unsigned>((a.max_new + kBlk - 2) / kBlk + 1);
  cudaLaunchAttribute attr[1];
  // the grid's last index has 16 bits
  for (int b0 = 0; b0 < a.seqs; b0 += 32768) {
    Kv8Args p = a;
    p.seqs = a.seqs - b0 < 32768 ? a.seqs - b0 : 32768;
    p.table += static_cast<size_t>(b0) * a.width;
    p.lens += b0;
    p.starts += b0;
    const cudaLaunchConfig_t cfg =
        pdl_launch_config(attr, dim3(pages, 2u * a.hkv, p.seqs), dim3(kAppThreads), 0, stream);
    cudaError_t e = cudaErrorInvalidValue;
#define TERN_APP_CASE(TYPE, D) \
  if (a.type == TYPE && a.dim == D) e = cudaLaunchKernelEx(&cfg, kv8_append_kernel<TYPE, D>, p);
    TERN_APP_CASE(TERN_F32, 64)
    TERN_APP_CASE(TERN_F32, 128)
    TERN_APP_CASE(TERN_BF16, 64)
    TERN_APP_CASE(TERN_BF16, 128)
    TERN_APP_CASE(TERN_F16, 64)
    TERN_APP_CASE(TERN_F16, 128)
#undef TERN_APP_CASE
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace tern
