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

// Four codes of an older token to a larger scale.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = static_cast<float>(static_cast<int8_t>((w >> (8 * e)) & 0xFFu));
    o |= (static_cast<uint32_t>(static_cast<int>(rintf(c * ratio))) & 0xFFu) << (8 * e);
  }
  return o;
}

// A block's scale from the largest new magnitude and the older tokens' scale (0
// without any).
__device__ __forceinline__ float block_scale(float amax, float old, bool& grew) {
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
  const KvSeq s = kv_whole_seq(a, b);
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
  bool grew;
  const float scale = block_scale(amax, old, grew);
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
        *p = make_uint2(shrink4(u.x, ratio), shrink4(u.y, ratio));
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

// The append with the keys and the rows' queries turned on the way, in one launch
// that takes a projection's output to the cache and to the attention's queries.
// CTAs of a page's keys or values of some heads (two of 128 elements or four of 64,
// half as many for few tokens), kPer threads each, and behind them CTAs of some of its
// new tokens and t.q_heads query heads.  A thread holds units of eight elements (whole
// pairs) as they are stored, and turns them twice, for the block's largest and for its
// codes.  A CTA makes its tokens' turns, some 30 instructions each, once for its heads,
// while the rows are on their way; what a block's threads share (its scale and that
// inverted) one warp makes for all.  (256 threads that each made their own, in 16
// unrolled copies for several heads, waited for instructions: 39 us for three ragged
// chunks of 3554 tokens, 48 query and 8 other heads of 128 in fp32; 34 here, 4.9 TB/s,
// 0.72 of the copy rate.)
template <int TYPE, int D, int kTurnThreads>
__global__ void __launch_bounds__(kTurnThreads, 1024 / kTurnThreads)
    kv8_append_rope_kernel(const Kv8Args a, const Kv8Turn t) {
  constexpr int kPer = 2 * D;  // threads of a head: four steps of sixteen tokens
  constexpr int kTurnHeads = kTurnThreads / kPer;
  grid_dependents_launch();
  constexpr int kUnits = D / 8;
  constexpr int kTok = kPer / kUnits;  // tokens per step
  constexpr int kSteps = kBlk / kTok;
  __shared__ float red[kTurnHeads][kPer / 32];
  __shared__ float4 block[kTurnHeads];  // scale, 1 / scale, old / scale, grew
  __shared__ float4 turns[2][kBlk * kUnits];
  const int b = blockIdx.z;
  const int kv_groups = (a.hkv + kTurnHeads - 1) / kTurnHeads;
  const int at_q = static_cast<int>(blockIdx.y) - 2 * kv_groups;  // of the queries' CTAs
  const int which = blockIdx.y & 1;
  RopeUnit unit(t.rope, threadIdx.x % kUnits);
  if (at_q < 0 && which) unit = RopeUnit(RopeArgs{nullptr, 0, 0, 1.f}, threadIdx.x % kUnits);
  grid_dependency_wait();  // every input and the cache come from earlier work
  const KvSeq s = kv_whole_seq(a, b);
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
  if (at_q >= 0) {
    // few tokens: their heads side by side, the more the fewer they are
    constexpr int kLanes = kTurnThreads / kUnits;
    const int lane = threadIdx.x / kUnits;
    int side = kLanes;
    while (side > 1 && side * (last - first) > kLanes) side >>= 1;
    const int h0 = at_q / t.q_cuts * t.q_heads, cut = at_q % t.q_cuts;
    const int h1 = a.heads < h0 + t.q_heads ? a.heads : h0 + t.q_heads;
    const int step = kLanes / side;
    for (int slot = first + lane / side + cut * step; slot < last; slot += t.q_cuts * step) {
      const long long row = row_of(slot);
      float2 turn[4];
      bool made = false;
      for (int h = h0 + lane % side; h < h1; h += kRopeBatch * side) {
        RopeHeads<TYPE> x;
        x.load(unit, a.q, row * t.q_ld, t.q_hd, h, side, h1);
        if (!made && unit.pair >= 0) rope_turns(t.rope, unit.pair, position(slot), turn);
        made = true;
        const long long to = row * a.heads * D;
        if (t.out_type == TERN_BF16)
          x.template store<TERN_BF16>(t.rope, unit, turn, t.out, to, D, h, side, h1);
        else
          x.template store<TERN_F16>(t.rope, unit, turn, t.out, to, D, h, side, h1);
      }
    }
    return;
  }
  const int at = threadIdx.x / kPer, tid = threadIdx.x % kPer;
  const int head = (blockIdx.y >> 1) * kTurnHeads + at;
  const bool live = head < a.hkv;
  const int slot0 = tid / kUnits;
  const int page = a.table[static_cast<size_t>(b) * a.width + pg];
  Raw4<TYPE> raw[kSteps][2];
  {
    // the thread's elements of the page's slot 0, which may lie before the rows
    const void* src = which ? a.v : a.k;
    const long long from = (row_of(0) + slot0) * a.ld + head * a.hd;
    const long long step = kTok * a.ld;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int slot = slot0 + k * kTok;
      if (live && slot >= first && slot < last) {
        raw[k][0] = raw4<TYPE>(src, from + k * step + unit.a);
        raw[k][1] = raw4<TYPE>(src, from + k * step + unit.b);
      }
    }
  }
  const bool turned = unit.pair >= 0;
  if (turned) {
#pragma unroll 1
    for (int i = threadIdx.x; i < kBlk * kUnits; i += kTurnThreads) {
      const int slot = i / kUnits;
      if (slot < first || slot >= last) continue;
      float2 turn[4];
      rope_turns(t.rope, unit.pair, position(slot), turn);
      turns[0][i] = make_float4(turn[0].x, turn[0].y, turn[1].x, turn[1].y);
      turns[1][i] = make_float4(turn[2].x, turn[2].y, turn[3].x, turn[3].y);
    }
  }
  if (page < 0 || page >= a.pages) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  const size_t blk = (static_cast<size_t>(page) * 2 + which) * a.hkv + head;
  const float old = live && first > 0 ? a.scales[blk] : 0.f;
  __syncthreads();
  // a unit's eight values
  auto values = [&](int k, float (&u)[4], float (&v)[4]) {
    unpack4<TYPE>(raw[k][0], u);
    unpack4<TYPE>(raw[k][1], v);
    if (turned) {
      const float4 x = turns[0][k * kPer + tid], y = turns[1][k * kPer + tid];
      const float2 turn[4] = {make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y),
                              make_float2(y.z, y.w)};
      rope_apply(t.rope, turn, u, v);
    }
  };
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int slot = slot0 + k * kTok;
    if (!live || slot < first || slot >= last) continue;
    float u[4], v[4];
    values(k, u, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = max_nan(amax, max_nan(fabsf(u[e]), fabsf(v[e])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[at][tid >> 5] = amax;
  __syncthreads();
  if (tid < 32) {
    amax = red[at][tid % (kPer / 32)];
#pragma unroll
    for (int o = kPer / 64; o > 0; o >>= 1)
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    bool grew;
    const float scale = block_scale(amax, old, grew);
    if (tid == 0) {
      block[at] = make_float4(scale, 1.0f / scale, old / scale, grew ? 1.f : 0.f);
      if (live && (grew || first == 0)) a.scales[blk] = scale;
    }
  }
  __syncthreads();
  if (!live) return;
  const float4 bl = block[at];
  const float scale = bl.x, inv = bl.y, ratio = bl.z;
  const bool grew = bl.w != 0.f, fast = quant_fast(scale);
  int8_t* codes = a.codes + blk * (kBlk * D) + slot0 * D;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int slot = slot0 + k * kTok;
    uint32_t* to_a = reinterpret_cast<uint32_t*>(codes + k * kTok * D + unit.a);
    uint32_t* to_b = reinterpret_cast<uint32_t*>(codes + k * kTok * D + unit.b);
    if (slot < first) {
      if (grew) {
        *to_a = shrink4(*to_a, ratio);
        *to_b = shrink4(*to_b, ratio);
      }
    } else if (slot < last) {
      float u[4], v[4];
      values(k, u, v);
      *to_a = scale > 0.f ? quant_codes4_short(u, scale, inv, fast) : 0u;
      *to_b = scale > 0.f ? quant_codes4_short(v, scale, inv, fast) : 0u;
    }
  }
}

// Launches `kernel` over the pages that a.max_new new tokens of a sequence
// touch, `rows` CTAs each; more.. : its arguments behind a.
template <typename Kernel, typename... More>
cudaError_t launch_pages(const Kv8Args& a, unsigned rows, int threads, Kernel kernel,
                         cudaStream_t stream, int* launches, const More&... more) {
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
        pdl_launch_config(attr, dim3(pages, rows, p.seqs), dim3(threads), 0, stream);
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
    return launch_pages(a, 2u * a.hkv, kAppThreads, kv8_append_kernel<TYPE, D>, stream, launches);
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
  // Few tokens have few turns to share: smaller CTAs of more heads.  So and otherwise:
  // 16 sequences of a token 3.2 and 3.9 us; three
  // chunks of 3554 tokens together 46 and 34.
  const bool few = a.max_new * kRopeBatch < kAppThreads / (a.dim / 8);
  const int threads = few ? 256 : 512;
  const int kv = 2 * ((a.hkv - 1) / (threads / (2 * a.dim)) + 1);
  unsigned chunks = 0;
  if (a.q) {
    // Heads of a query CTA, and CTAs that take its page's tokens in turn: few tokens
    // fill its threads with heads, many are batches of heads for each thread and
    // one step of tokens a CTA.  The grid's second index has 16 bits.
    const int lanes = threads / (a.dim / 8);  // tokens of a step
    t.q_heads = few ? lanes : 2 * kRopeBatch;
    t.q_cuts = few || lanes >= kBlk ? 1 : kBlk / lanes;
    const int room = (65535 - kv) / t.q_cuts;
    if ((a.heads - 1) / t.q_heads >= room) t.q_heads = (a.heads - 1) / room + 1;
    chunks = (a.heads - 1) / t.q_heads * t.q_cuts + t.q_cuts;
  }
#define TERN_APP_CASE(TYPE, D, N)                                                            \
  if (a.type == TYPE && a.dim == D && threads == N)                                          \
    return launch_pages(a, kv + chunks, N, kv8_append_rope_kernel<TYPE, D, N>, stream, launches, t);
#define TERN_APP_CASES(TYPE)    \
  TERN_APP_CASE(TYPE, 64, 256)  \
  TERN_APP_CASE(TYPE, 64, 512)  \
  TERN_APP_CASE(TYPE, 128, 256) \
  TERN_APP_CASE(TYPE, 128, 512)
  TERN_APP_CASES(TERN_F32)
  TERN_APP_CASES(TERN_BF16)
  TERN_APP_CASES(TERN_F16)
#undef TERN_APP_CASES
#undef TERN_APP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace tern
