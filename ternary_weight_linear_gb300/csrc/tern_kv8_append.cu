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
#include "tern_kv8.cuh"
#include "tern_quant.cuh"
#include "tern_rope.cuh"

namespace tern {
namespace {

constexpr int kAppThreads = 256;

// The codes of eight elements of an older token to a larger scale.
__device__ __forceinline__ void shrink8(int8_t* codes, float ratio) {
  uint2* p = reinterpret_cast<uint2*>(codes);
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

// The block's scale from its threads' largest new magnitudes and the older
// tokens' scale (0 without any).  Whole CTA; red: a float a warp.
__device__ __forceinline__ float block_scale(float amax, float old, float* red, bool& grew) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppThreads / 32; ++i) amax = max_nan(amax, red[i]);
  float fresh = amax / 127.0f;                                     // IEEE division
  if (!(fresh < __uint_as_float(0x7F800000u))) fresh = __uint_as_float(0x7FC00000u);
  // a NaN on either side stays
  grew = !(fresh <= old) && !(old != old);
  return grew ? fresh : old;
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
  bool grew;
  const float scale = block_scale(amax, old, red, grew);
  if (threadIdx.x == 0 && (grew || first == 0)) a.scales[blk] = scale;
  const float inv = 1.0f / scale;
  const bool fast = quant_fast(scale);
  if (grew && first > 0) {
    const float ratio = old / scale;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int slot = slot0 + i * kTok;
      if (slot < first) shrink8(codes + slot * D + 8 * chunk, ratio);
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

// The append with the keys and the rows' queries turned on the way: CTAs of a
// page's keys or values of a head as above, whose threads hold whole pairs
// (sixteen elements of a token), and behind them CTAs of the page's new tokens
// and t.q_heads query heads, whose threads use a token's turns for several
// heads.  One launch takes a projection's output to the cache and to the
// attention's queries; a prompt is bound by HBM, a decode step by latency.
template <int TYPE, int D>
__global__ void __launch_bounds__(kAppThreads)
    kv8_append_rope_kernel(const Kv8Args a, const Kv8Turn t) {
  grid_dependents_launch();
  constexpr int kUnits = D / 16;
  constexpr int kTok = kAppThreads / kUnits;  // tokens per step
  constexpr int kSteps = kBlk / kTok;
  __shared__ float red[kAppThreads / 32];
  const int b = blockIdx.z;
  const int slot0 = threadIdx.x / kUnits;
  const int hq = static_cast<int>(blockIdx.y) - 2 * a.hkv;  // of the queries' CTAs
  const int which = blockIdx.y & 1, h = blockIdx.y >> 1;
  RopeUnit unit(t.rope, threadIdx.x % kUnits);
  if (hq < 0 && which) unit = RopeUnit(RopeArgs{nullptr, 0, 0, 1.f}, threadIdx.x % kUnits);
  grid_dependency_wait();  // every input and the cache come from earlier work
  const KvSeq s = kv_seq(a, b);
  if (!s.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  if (s.m == 0) return;
  const int begin = s.len - s.m;  // first new token
  const int pg = begin / kBlk + static_cast<int>(blockIdx.x);
  if (pg > (s.len - 1) / kBlk) return;
  const int first = begin > pg * kBlk ? begin - pg * kBlk : 0;       // new slots [first, last)
  const int last = s.len - pg * kBlk < kBlk ? s.len - pg * kBlk : kBlk;
  auto row_of = [&](int slot) { return s.row0 + static_cast<long long>(pg * kBlk + slot - begin); };
  auto position = [&](int slot) {
    return t.positions ? t.positions[row_of(slot)] : pg * kBlk + slot;
  };
  if (hq >= 0) {
    // few tokens: their heads side by side, the more the fewer they are
    int side = kTok;
    while (side > 1 && side * (last - first) > kTok) side >>= 1;
    const int h0 = hq * t.q_heads;
    const int h1 = a.heads < h0 + t.q_heads ? a.heads : h0 + t.q_heads;
    for (int slot = first + slot0 / side; slot < last; slot += kTok / side) {
      const long long row = row_of(slot);
      float2 turn[8];
      if (unit.pair >= 0) rope_turns(t.rope, unit.pair, position(slot), turn);
#pragma unroll 2
      for (int i = h0 + slot0 % side; i < h1; i += side) {
        float u[8], v[8];
        const long long from = row * t.q_ld + i * t.q_hd;
        load8<TYPE>(a.q, from + unit.a, u);
        load8<TYPE>(a.q, from + unit.b, v);
        if (unit.pair >= 0) rope_apply(t.rope, turn, u, v);
        const long long to = (row * a.heads + i) * D;
        if (t.out_type == TERN_BF16) {
          store8<TERN_BF16>(t.out, to + unit.a, u);
          store8<TERN_BF16>(t.out, to + unit.b, v);
        } else {
          store8<TERN_F16>(t.out, to + unit.a, u);
          store8<TERN_F16>(t.out, to + unit.b, v);
        }
      }
    }
    return;
  }
  const int page = a.table[static_cast<size_t>(b) * a.width + pg];
  const void* src = which ? a.v : a.k;
  float x[kSteps][2][8];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kTok;
    if (slot >= first && slot < last) {
      const long long from = row_of(slot) * a.ld + h * a.hd;
      load8<TYPE>(src, from + unit.a, x[i][0]);
      load8<TYPE>(src, from + unit.b, x[i][1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][0][e] = x[i][1][e] = 0.f;
    }
  }
  if (page < 0 || page >= a.pages) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  const size_t blk = (static_cast<size_t>(page) * 2 + which) * a.hkv + h;
  int8_t* codes = a.codes + blk * (kBlk * D);
  const float old = first > 0 ? a.scales[blk] : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kTok;
    if (unit.pair >= 0 && slot >= first && slot < last) {
      float2 turn[8];
      rope_turns(t.rope, unit.pair, position(slot), turn);
      rope_apply(t.rope, turn, x[i][0], x[i][1]);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = max_nan(amax, fabsf(x[i][e >> 3][e & 7]));
  }
  bool grew;
  const float scale = block_scale(amax, old, red, grew);
  if (threadIdx.x == 0 && (grew || first == 0)) a.scales[blk] = scale;
  const float inv = 1.0f / scale;
  const bool fast = quant_fast(scale);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int slot = slot0 + i * kTok;
    int8_t* at = codes + slot * D;
    if (slot < first) {
      if (grew) {
        shrink8(at + unit.a, old / scale);
        shrink8(at + unit.b, old / scale);
      }
    } else if (slot < last) {
      uint2 w[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
      if (scale > 0.f) {
        w[0] = quant_codes8(x[i][0], scale, inv, fast);
        w[1] = quant_codes8(x[i][1], scale, inv, fast);
      }
      *reinterpret_cast<uint2*>(at + unit.a) = w[0];
      *reinterpret_cast<uint2*>(at + unit.b) = w[1];
    }
  }
}

// Launches `kernel` over the pages that a.max_new new tokens of a sequence
// touch, `rows` CTAs each; more.. : its arguments behind a.
template <typename Kernel, typename... More>
cudaError_t launch_pages(const Kv8Args& a, unsigned rows, Kernel kernel, cudaStream_t stream,
                         int* launches, const More&... more) {
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
        pdl_launch_config(attr, dim3(pages, rows, p.seqs), dim3(kAppThreads), 0, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, more...);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, cudaStream_t stream, int* launches) {
#define TERN_APP_CASE(TYPE, D)          \
  if (a.type == TYPE && a.dim == D)     \
    return launch_pages(a, 2u * a.hkv, kv8_append_kernel<TYPE, D>, stream, launches);
  TERN_APP_CASE(TERN_F32, 64)
  TERN_APP_CASE(TERN_F32, 128)
  TERN_APP_CASE(TERN_BF16, 64)
  TERN_APP_CASE(TERN_BF16, 128)
  TERN_APP_CASE(TERN_F16, 64)
  TERN_APP_CASE(TERN_F16, 128)
#undef TERN_APP_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv8_append_rope(const Kv8Args& a, const Kv8Turn& turn, cudaStream_t stream,
                                   int* launches) {
  Kv8Turn t = turn;
  unsigned chunks = 0;
  if (a.q) {
    // heads of a query CTA: few tokens fill its threads with heads, many use
    // their turns for eight; the grid's second index has 16 bits
    const int lanes = kAppThreads / (a.dim / 16);
    t.q_heads = a.max_new * 8 < lanes ? lanes : 8;
    const int room = 65535 - 2 * a.hkv;
    if ((a.heads - 1) / t.q_heads >= room) t.q_heads = (a.heads - 1) / room + 1;
    chunks = (a.heads + t.q_heads - 1) / t.q_heads;
  }
#define TERN_APP_CASE(TYPE, D)          \
  if (a.type == TYPE && a.dim == D)     \
    return launch_pages(a, 2u * a.hkv + chunks, kv8_append_rope_kernel<TYPE, D>, stream, launches, t);
  TERN_APP_CASE(TERN_F32, 64)
  TERN_APP_CASE(TERN_F32, 128)
  TERN_APP_CASE(TERN_BF16, 64)
  TERN_APP_CASE(TERN_BF16, 128)
  TERN_APP_CASE(TERN_F16, 64)
  TERN_APP_CASE(TERN_F16, 128)
#undef TERN_APP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tern
