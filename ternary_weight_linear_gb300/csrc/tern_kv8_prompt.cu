// tern_kv8_attention for sequences with many query rows per key-value head
// (prompt chunks): bound by the tensor cores and what feeds them.
//
// The rows of a sequence that share a key-value head (row r = new token
// r / group, head r % group) are cut into blocks of 256, two tiles of 128 that
// share every page of keys and values.  Per tile and page of 64 tokens, with
// tcgen05 kind::f16 (fp16 operands, fp32 accumulators in TMEM):
//   S = Q Kc^T,  s = S * (softmax_scale * log2(e) * k_scale * 2^-a(row))
//   P = 2^(s + log2 f - ref + 10),  O += P (2^(e - E) Vc),  l += P / f
// with Q scaled by 2^a per row into fp16, Kc and Vc the int8 codes (exact in
// fp16), v_scale = 2^e f and E the largest e so far.  (Where the blocks' e lie
// more than 8 apart P takes the whole v_scale and each row has a reference of its
// own for it: wide_pages.)  P is rounded to fp16
// (relative 2^-11, the tensor instruction's operand; the row's sum takes it
// unrounded).  ref is the row's running maximum, raised (and O rescaled) only
// when a score passes it by 2^4: P stays below 2^15 (fp16 ends at 65504) and
// its range below is 2^-34 of that reference, so a weight is lost only where
// it is that much smaller.
//
// There is no int8 tcgen05 on sm_103a, so four warps turn each page of codes
// into fp16 in shared memory, once for the two query tiles: the keys as
// (code + 128) 2^-24, whose bias each row takes off its scores.
//
// Warps: 0-3 and 4-7 the two query tiles' softmax, one row per thread (a
// page's 64 scores read from TMEM once; P written over them); 8-11 the
// conversion; 12-15 the MMAs, for each query tile one thread that issues the
// scores and one that issues the products with the values: a barrier wait
// costs an issuing thread about 200 cycles even on a completed phase, which
// the other three cover.  Each tile has two score buffers, so the scores run
// up to two pages ahead of the values and the softmax finds them ready.
// Work: one CTA per (block of rows, sequence, head), the longest rows first;
// the blocks of the last wave are cut along the keys into parts, whose (ref,
// sum, O) go to the workspace, and the last CTA of a block adds them in order.
//
// Measured: 2048 tokens of 6 query heads per key-value head over 8190 cached,
// head of 128: 292 us, 1233 TFLOP/s (0.65 of the bf16 GEMM rate; 484 us by
// wide_pages); 4096 over 16384: 1017 us, 1420 TFLOP/s (0.75); 2048 over 8192 of 32
// query and 8 key-value heads of 64: 172 us, 699 TFLOP/s (0.37: a page's
// exponentials are as many for half the products).  Both score buffers in one product pair
// that reads the queries from shared memory once lost a quarter: the softmax
// then waits for each pair.
#include "tern_kv8.cuh"

namespace tern {
namespace {

constexpr int kPRows = 128;  // rows of a query tile
constexpr int kSoftW = 8, kConvW = 4;
constexpr int kMmaW = kSoftW + kConvW;
constexpr int kPThreads = (kMmaW + 4) * 32;
constexpr int kPRecs = 512;  // page records held at a time
constexpr int kAhead = 4;    // pages requested into L2 ahead of their conversion (kSplit)
constexpr float kPOff = 10.f, kPLazy = 4.f;
// Value scales whose exponents lie up to this far apart share one.  (A code times
// 2^-8 is exact in fp16; a weight below 2^-35 of the row's largest is lost, and
// with it at most 2^-27 of the largest weight times value scale.)
constexpr int kSpan = 8;
// Pages of time in sequence on an SM when `items` blocks of `pages` pages are cut
// into parts, each of which costs some pages for its start, its result and the
// join.  Parts have kPartPages pages at least.
constexpr int kPartPages = 8, kPartCost = 14;
__host__ __device__ constexpr unsigned part_cost(unsigned pages, unsigned parts, unsigned items,
                                                 unsigned sms) {
  return (items * parts + sms - 1) / sms * ((pages + parts - 1) / parts + kPartCost);
}
constexpr float kUp = 16777216.f;  // 2^24, 1 over the keys' unit

template <int D>
struct PL {
  static constexpr int kBlocks = D / 64;               // 128-byte wide blocks of a row
  static constexpr int kQBlockB = kPRows * 128;
  static constexpr int kQTileB = kBlocks * kQBlockB;   // a query tile in fp16
  static constexpr int kBlockB = kBlk * 128;
  static constexpr int kTileB = kBlocks * kBlockB;     // a page's keys or values in fp16
  static constexpr int kRawB = kBlk * D;               // and as codes
  static constexpr int kConv = D == 128 ? 4 : 6;       // converted pages (keys and values)
  static constexpr int kQOff = 0;
  static constexpr int kConvOff = kQOff + 2 * kQTileB;
  static constexpr int kRecOff = kConvOff + 2 * kConv * kTileB;  // PageRec, then pages and e
  static constexpr int kBarOff = kRecOff + kPRecs * 24;
  static constexpr int kNumBars = 3 * kConv + 4 + 4 + 4 + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // TMEM address, last, emax, emin
  static constexpr int kBytes = kMiscOff + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kSCol = 0, kOCol = 256;
  static_assert(kBarOff % 8 == 0 && kRecOff % 16 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// What the softmax needs of a page, in one 16-byte load.
struct __align__(16) PageRec {
  float ks, lf, rf;  // key scale; log2 f and 1 / f of the value scale 2^e f
  int meta;          // page index in the sequence * 4, bit q: every row of query
                     // tile q sees the whole page; -1: no page
};

constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// The whole warp calls these, and one lane issues: with uniform control flow
// the descriptors stay in uniform registers (under a branch of one lane each
// product moved six of them, and eight products took 1050 cycles to issue).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void mma_commit_warp(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar))
      : "memory");
}

// 128-byte swizzled operand: rows of 128 bytes, 8-row atoms 1024 bytes apart.
// K-major (rows are M or N) and MN-major (rows are K, 64 elements of N wide,
// the next 64 a block further) share the bytes; lbo is the block stride of the
// latter.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// All threads of the CTA, from any role.
__device__ __forceinline__ void cta_barrier() {
  asm volatile("bar.sync 0;" ::: "memory");
}
// A block's rows of the output, staged in shared memory where the queries were
// (a warp's own rows, whose products are done): chunks of 16 bytes swizzled by
// the row, written D / 8 lanes a row.
template <int D>
struct OutRows {
  const Kv8Args& a;
  uint8_t* stage;
  int r0, row0, hk;
  __device__ __forceinline__ uint8_t* staged(int row, int c) const {
    return stage + row * (2 * D) + ((c ^ (row & 7)) << 4);
  }
  __device__ __forceinline__ long long row(int r) const {  // of out and lse
    const int tok = kv_token(a, r0 + r);
    return static_cast<long long>(row0 + tok) * a.heads + hk * a.group +
           (r0 + r - tok * a.group);
  }
  // (whole warp) rows [begin, end), none if end <= begin
  __device__ __forceinline__ void write_out(int lane, int begin, int end) const {
    constexpr int kLanes = D / 8;
#pragma unroll 4
    for (int r = begin + lane / kLanes; r < end; r += 32 / kLanes)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row(r) * D +
                                8 * (lane % kLanes)) = lds_v4(staged(r, lane % kLanes));
  }
};

// Named barriers (0 is the whole CTA's, 1 the softmax warps').
enum : int { kUsed = 2, kReady, kWritten, kQueries };
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The last part to arrive adds them all in order (every thread of the CTA) and
// stages the rows.
template <int D>
__device__ __forceinline__ void join_parts(const Kv8Args& a, uint8_t* smem, const float* first,
                                           int parts, int rows, int r0, int row0, int hk) {
  using L = PL<D>;
  constexpr size_t kPart = 2 * kPRows * (D + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const OutRows<D> put{a, smem + L::kQOff, r0, row0, hk};
  const int rows32 = (rows + 31) & ~31;
  float* weight = reinterpret_cast<float*>(smem + L::kConvOff);  // [part][rows32]
  // a row per thread: the parts' weights over the row's sum
  if (threadIdx.x < rows) {
    const int row = threadIdx.x;
    float top = -INFINITY;
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
      const float2 ms =
          __ldcg(reinterpret_cast<const float2*>(first + p * kPart + 2 * kPRows * D) + row);
      const float w = ms.y == 0.f ? -INFINITY : ms.x + log2f(ms.y);
      weight[p * rows32 + row] = w;
      top = fmaxf(top, w);
    }
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float w = exp2f(weight[p * rows32 + row] - base);
      weight[p * rows32 + row] = w;
      l += w;
    }
    const float one = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) weight[p * rows32 + row] *= one;
    if (a.lse) a.lse[put.row(row)] = kv_log_sum(base, l, kPOff);
  }
  cta_barrier();
  // sixteen elements of 32 rows per warp, four parts' loads in flight
  for (int i = warp; i < rows32 / 32 * (D / 16); i += kPThreads / 32) {
    constexpr int kAtOnce = 4, kC = 4;
    const int c = i % (D / 16) * kC, row = i / (D / 16) * 32 + lane;
    if (row >= rows) continue;
    const float4* from = reinterpret_cast<const float4*>(first) + c * (2 * kPRows) + row;
    float4 acc[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += kAtOnce) {
      float4 v[kAtOnce][kC];
#pragma unroll
      for (int p = 0; p < kAtOnce; ++p)
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          v[p][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p0 + p < parts) v[p][k] = __ldcg(from + (p0 + p) * (kPart / 4) + k * (2 * kPRows));
        }
#pragma unroll
      for (int p = 0; p < kAtOnce; ++p) {
        const float w = p0 + p < parts ? weight[(p0 + p) * rows32 + row] : 0.f;
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          acc[k].x = fmaf(w, v[p][k].x, acc[k].x);
          acc[k].y = fmaf(w, v[p][k].y, acc[k].y);
          acc[k].z = fmaf(w, v[p][k].z, acc[k].z);
          acc[k].w = fmaf(w, v[p][k].w, acc[k].w);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kC; k += 2)
      *reinterpret_cast<uint4*>(put.staged(row, (c + k) >> 1)) =
          make_uint4(pack_out(a.type, acc[k].x, acc[k].y), pack_out(a.type, acc[k].z, acc[k].w),
                     pack_out(a.type, acc[k + 1].x, acc[k + 1].y),
                     pack_out(a.type, acc[k + 1].z, acc[k + 1].w));
  }
}

// The row of O at o_col times alpha.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t o_col, float alpha) {
#pragma unroll 1
  for (int q = 0; q < D / 16; ++q) {
    uint32_t x[16];
    tmem_ld16(o_col + 16 * q, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * alpha);
    tmem_st16(o_col + 16 * q, x);
  }
}

// A row's softmax: its reference and sum, and the unit of its O, 2^(ref + lead).
struct SoftState {
  float ref, sum, lead;
  bool ok;
};

// The softmax warps' part where value scales are too far apart for one
// exponent: a row's O has a unit of its own, which follows its largest weight
// times value scale, beside the sum's 2^ref.  A set of `count` pages from page
// jt on, every kStep-th of them of query tile qt; row: the row's place in TMEM.
// (Rare, and a function of its own: inlined, it cost the usual loop 1.5 % by its
// registers; 2048 tokens over 8190 296 and 292 us.)
template <int D, int kStep>
__device__ __noinline__ SoftState wide_pages(uint8_t* smem, const Kv8Args& a, SoftState st, int qt,
                                             int jt, int count, uint32_t row, int pos, float cs,
                                             float bias) {
  using L = PL<D>;
  uint64_t* s_full = reinterpret_cast<uint64_t*>(smem + L::kBarOff) + 3 * L::kConv;
  uint64_t* p_full = s_full + 4;
  uint64_t* o_done = p_full + 4;
  const PageRec* recs = reinterpret_cast<const PageRec*>(smem + L::kRecOff);
  const int* rec_e = reinterpret_cast<const int*>(recs + kPRecs) + kPRecs;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int j = jt + (kStep == 2 ? qt : 0); j < jt + count; j += kStep) {
    const int n = j / kStep, buf = 2 * qt + (n & 1);
    st.ok = st.ok && mbar_wait_clk(&s_full[buf], (n >> 1) & 1, a.err);
    st.ok = __all_sync(0xffffffffu, st.ok);
    if (!st.ok) break;
    tc_fence_after();
    const uint32_t sc = row + L::kSCol + qt * 128 + (n & 1) * kBlk;
    const PageRec rec = recs[j - jt];
    const float c = fmaxf(cs * rec.ks * kUp, 1e-37f);
    const uint64_t see = rec.meta >= 0 ? kv_mask(a, pos, (rec.meta >> 2) * kBlk) : 0;
    auto scores = [&](int q, uint32_t (&x)[16]) {
      tmem_ld16(sc + 16 * q, x);
      tmem_wait_ld();
      const uint32_t bits = static_cast<uint32_t>(see >> (16 * q));
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (!(bits & (1u << k))) x[k] = __float_as_uint(-INFINITY);
    };
    float big = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t x[16];
      scores(q, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) big = fmaxf(big, __uint_as_float(x[k]));
    }
    const float top = (big - bias) * c;  // -inf: no visible token
    const float lv = rec.lf + static_cast<float>(rec_e[j - jt]);
    float unit = st.ref + st.lead, alpha = 1.f;  // (-inf at the row's first)
    const bool raise = top + lv > unit + kPLazy;
    if (raise) {
      alpha = exp2_approx(unit - (top + lv));
      unit = top + lv;
    }
    if (top > st.ref + kPLazy) {
      st.sum *= exp2_approx(st.ref - top);
      st.ref = top;
    }
    if (st.ref != -INFINITY) st.lead = unit - st.ref;
    if (__any_sync(0xffffffffu, raise) && n > 0) {
      // O has to hold everything up to the page before
      st.ok = st.ok && mbar_wait_clk(&o_done[buf ^ 1], ((n - 1) >> 1) & 1, a.err);
      tc_fence_after();
      rescale_row<D>(row + L::kOCol + qt * 128, alpha);
    }
    // weights for the sum and, times the value scale, for the products
    const float add = fmaf(-bias, c, kPOff - (st.ref == -INFINITY ? 0.f : st.ref));
    const float add_o = add + (lv - st.lead);
    float part = 0.f;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t x[16], w[8];
      scores(q, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x0 = __uint_as_float(x[2 * k]), x1 = __uint_as_float(x[2 * k + 1]);
        part += exp2_approx(fmaf(x0, c, add)) + exp2_approx(fmaf(x1, c, add));
        w[k] = half2_bits(exp2_approx(fmaf(x0, c, add_o)), exp2_approx(fmaf(x1, c, add_o)));
      }
      tmem_st8(sc + 8 * q, w);  // (over scores that have been read)
    }
    // (a NaN for the rows that see a block whose scales cannot be used)
    if (big != -INFINITY) st.sum = rec.rf == rec.rf ? st.sum + part : rec.rf;
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&p_full[buf]);
  }
  return st;
}

// kSplit: no sequence of the batch has more than kSplitRows = 64 rows for a
// key-value head.  Both query tiles are then the same rows and take alternate
// pages (page j of the CTA is tile i's page j / 2, for j % 2 == i), joined at
// the end, and the four softmax warps without rows are a second group for the
// conversion.  Measured when it came, with it and without: 36.5 and 42.9 us (8
// sequences, 20 rows, window 4096), 92 and 123 us (4 sequences of 32000 tokens, 24 rows); at
// 96 rows, where no warps are idle, it loses (46.5 and 43.2 us, 16 tokens over
// 16000).
constexpr int kSplitRows = 64;
template <int D, bool kSplit>
__global__ void __launch_bounds__(kPThreads, 1)
    kv8_prompt_kernel(const __grid_constant__ Kv8Args a, int min_rows, int row_blocks, int whole,
                      int tail_parts, int tail_items, int sms, float* __restrict__ partials,
                      int* __restrict__ tickets) {
  using L = PL<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);  // converted keys
  uint64_t* v_full = k_full + L::kConv;                               // converted values
  uint64_t* conv_empty = v_full + L::kConv;
  uint64_t* s_full = conv_empty + L::kConv;  // [tile][buffer] scores
  uint64_t* p_full = s_full + 4;           // [tile][buffer] weights, O rescaled
  uint64_t* o_done = p_full + 4;           // [tile][page parity] O holds the page
  uint64_t* mma_end = o_done + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  int* is_last = reinterpret_cast<int*>(tmem_slot + 1);
  int* emax = is_last + 1;  // largest and smallest exponent of the value scales so far
  int* emin = emax + 1;
  PageRec* recs = reinterpret_cast<PageRec*>(smem + L::kRecOff);
  int* rec_page = reinterpret_cast<int*>(recs + kPRecs);  // -1: none
  int* rec_e = rec_page + kPRecs;

  grid_dependency_wait();  // every input, the output and the workspace belong to earlier work

  // ---- this CTA's block of rows, sequence, head and part; late rows first
  const int tail = static_cast<int>(blockIdx.x) - whole;  // of the items in parts
  const int part = tail < 0 ? 0 : tail % tail_parts;
  const int item = tail < 0 ? static_cast<int>(blockIdx.x) : whole + tail / tail_parts;
  const int hk = item % a.hkv;
  const int b = (item / a.hkv) % a.seqs;
  const int rb = row_blocks - 1 - item / a.hkv / a.seqs;
  const KvSeq sq = kv_seq(a, b);
  const int R = sq.m * a.group;
  const int r0 = rb * (2 * kPRows);
  if (!sq.ok && threadIdx.x == 0) atomicOr(a.err, kErrIndex);
  if (!sq.ok || R < min_rows || r0 >= R) return;
  const int rows = R - r0 < 2 * kPRows ? R - r0 : 2 * kPRows;
  const int tiles_q = rows > kPRows ? 2 : 1;  // that see a page
  constexpr int kStep = kSplit ? 2 : 1;
  const int p_base = sq.len - sq.m;
  const int p_first = p_base + kv_token(a, r0);
  const int p_last = p_base + kv_token(a, r0 + rows - 1);
  const KvPages pages = kv_pages(a, p_first, p_last);
  // (The launch chose the parts by the table's width, the most pages that a
  // block can have: by its own it may need fewer, or none.)
  int parts = 1;
  if (tail >= 0 && tail_parts > 1) {
    const int fit = pages.count / kPartPages;
    const int p = tail_parts < fit ? tail_parts : fit;
    if (p > 1 && part_cost(pages.count, p, tail_items, sms) <
                     static_cast<unsigned>(pages.count + kPartCost))
      parts = p;
  }
  if (part >= parts) return;
  const int t_begin = static_cast<int>(static_cast<long long>(pages.count) * part / parts);
  const int t_end = static_cast<int>(static_cast<long long>(pages.count) * (part + 1) / parts);

  // warps of query tile i that have rows
  auto soft_warps = [&](int i) {
    const int w = (rows - (kSplit ? 0 : i * kPRows) + 31) / 32;
    return w < 0 ? 0 : w > 4 ? 4 : w;
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kConv; ++s) {
      mbar_init(&k_full[s], kConvW);
      mbar_init(&v_full[s], kConvW);
      mbar_init(&conv_empty[s], 2 * tiles_q);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], soft_warps(i >> 1) > 0 ? soft_warps(i >> 1) : 1);
      mbar_init(&o_done[i], 1);
    }
    *emax = kNoExp;
    *emin = -kNoExp;
    mbar_init(mma_end, 4);
    fence_mbar_init();
  }
  if (warp == kMmaW) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  cta_barrier();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // only now: a dependent kernel's CTA that took this SM's TMEM first would
  // hold it until this grid ends
  grid_dependents_launch();

  // ---- softmax warps: a row per thread
  const int qt = warp >> 2;  // query tile (softmax warps)
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int tr = (warp & 3) * 32 + lane;  // row of the tile
  const int r = (kSplit ? 0 : qt * kPRows) + tr;  // row of the block
  const bool live = warp < kSoftW && r < rows;
  int pos = -1;           // its position
  float cs = 0.f;         // softmax scale * log2(e) * 2^-a
  float bias = 0.f;       // what 128 in every key's place adds to the row's scores
  const bool soft = warp < kSoftW && (warp & 3) < soft_warps(qt);
  if (soft) {
    const int rr = r0 + (live ? r : rows - 1);  // (past the last: a copy of it)
    const int tok = kv_token(a, rr);
    const int head = hk * a.group + rr - tok * a.group;
    const long long qrow = sq.row0 + tok;
    if (live) pos = p_base + tok;
    // The warp's rows are copied to their places as they are, D / 8 lanes a
    // row, then each thread scales its own.
    const unsigned long long mine = reinterpret_cast<unsigned long long>(
        static_cast<const uint16_t*>(a.q) + qrow * a.ld + static_cast<long long>(head) * a.hd);
    constexpr int kLanes = D / 8;
    auto place = [&](int row, int c) {
      return smem + L::kQOff + qt * L::kQTileB + (c >> 3) * L::kQBlockB + row * 128 +
             (((c & 7) ^ (row & 7)) << 4);
    };
#pragma unroll 4
    for (int i = lane / kLanes; i < 32; i += 32 / kLanes)
      cp_async_16(place((warp & 3) * 32 + i, lane % kLanes),
                  reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, i)) +
                      16 * (lane % kLanes),
                  16);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    uint32_t m2 = 0;  // the largest magnitudes of the even and the odd elements
#pragma unroll
    for (int c = 0; c < kLanes; ++c) {
      const uint4 w = lds_v4(place(tr, c));
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                 __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
    }
    const uint32_t big = (m2 & 0xFFFFu) > (m2 >> 16) ? m2 & 0xFFFFu : m2 >> 16;
    const int up = q_exponent(big, a.type);
    const float f = pow2f(up);
    cs = a.scale_log2 * pow2f(-up);
#pragma unroll 1
    for (int c0 = 0; c0 < kLanes; c0 += 4) {
      uint4 raw[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) raw[c] = lds_v4(place(tr, c0 + c));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          unpack16(w[e], a.type, lo, hi);
          w[e] = half2_bits(lo * f, hi * f);
          unpack16(w[e], TERN_F16, lo, hi);
          bias += lo + hi;
        }
        *reinterpret_cast<uint4*>(place(tr, c0 + c)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    bias *= 128.f / kUp;
    fence_proxy_async_smem();
  }
  // positions of the block's last rows of tile 0 and first rows of tile 1
  const int p_end0 = p_base + kv_token(a, r0 + (rows < kPRows ? rows : kPRows) - 1);
  const int p_beg1 = kSplit ? p_first : p_base + kv_token(a, r0 + kPRows);

  // columns of tile i's scores (and weights) of its page n
  auto s_col = [](int i, int n) -> uint32_t { return L::kSCol + i * 128 + (n & 1) * kBlk; };

  int jt = 0;  // pages so far
  // Waits until tile i's O holds its page n.  Two pages may be under way and a
  // parity tells only neighbouring phases apart, so odd and even pages have
  // barriers of their own: page n - 2 is done before page n's scores exist,
  // which is before anyone waits for page n.
  auto wait_values = [&](int i, int n) {
    return mbar_wait_clk(&o_done[2 * i + (n & 1)], (n >> 1) & 1, a.err);
  };

  float lead = kNoExp;  // (softmax) the row's O is in units of 2^(ref + lead): E's once a page
                        // has rescaled it, which in kSplit may not be this set of records'
  float ref = -INFINITY, sum = 0.f;
  bool ok = true;

  for (int t0 = t_begin, chunk = 0; t0 < t_end; t0 += kPRecs, ++chunk) {
    const int t1 = t_end < t0 + kPRecs ? t_end : t0 + kPRecs;
    // ---- records of pages [t0, t1) of the list
    // (written by the warps that do not stage queries, so that the conversion
    // starts under that)
    if (warp >= kSoftW) {
      if (chunk > 0) named_sync(kUsed, kPThreads);  // those of the chunk before
    } else if (chunk > 0) {
      named_arrive(kUsed, kPThreads);
    }
    for (int i = static_cast<int>(threadIdx.x) - kSoftW * 32; i >= 0 && i < t1 - t0;
         i += kPThreads - kSoftW * 32) {
      int e = kZeroExp;
      PageRec rec = {0.f, 0.f, 0.f, -1};
      {
        const int lp = pages.page(t0 + i);
        int page = a.table[static_cast<size_t>(b) * a.width + lp];
        if (page < 0 || page >= a.pages) {
          atomicOr(a.err, kErrIndex);
          page = -1;
        } else {
          const float* sc = a.scales + static_cast<size_t>(page) * 2 * a.hkv + hk;
          const float ks = sc[0];
          const float vs = sc[a.hkv];
          // scales that cannot be used keep out of the arithmetic and make 1 / f
          // NaN
          const bool good = good_scales(ks, vs);
          const VScale v = split_vscale(good ? vs : 0.f);
          rec.ks = good ? ks : 0.f;
          rec.lf = good ? log2f(v.f) : 0.f;
          rec.rf = good ? 1.0f / v.f : __uint_as_float(0x7FC00000u);
          const int j0 = lp * kBlk, j1 = j0 + kBlk - 1;
          rec.meta = lp * 4 | (kv_all(a, p_first, p_end0, j0, j1) ? 1 : 0) |
                     (kv_all(a, p_beg1, p_last, j0, j1) ? 2 : 0);
          e = v.e;
          if (e != kZeroExp) {
            atomicMax(emax, e);
            atomicMin(emin, e);
          }
        }
        rec_page[i] = page;
      }
      recs[i] = rec;
      rec_e[i] = e;
    }
    __syncwarp();
    if (warp >= kSoftW) {
      named_arrive(kReady, kPThreads);
      named_sync(kWritten, kPThreads - kSoftW * 32);
      if (chunk == 0 && warp >= kMmaW) named_sync(kQueries, kPThreads - kConvW * 32);
    } else {
      if (chunk == 0) named_arrive(kQueries, kPThreads - kConvW * 32);
      named_sync(kReady, kPThreads);
    }
    // The exponent that the converted values share, unless (and then to the end)
    // they lie too far apart.  (The next pages' records wait until every thread
    // has been here.)
    const int E = *emax;
    const bool wide = E - *emin > kSpan;

    if (warp >= kMmaW) {
      // ---------------------------------------------------------- MMAs
      const int role = __shfl_sync(0xffffffffu, warp, 0) - kMmaW;
      const int i = role >> 1;  // query tile
      const int j0 = __shfl_sync(0xffffffffu, jt, 0) + (kSplit ? i : 0);
      const int j_end = __shfl_sync(0xffffffffu, jt + t1 - t0, 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tbase, 0);
      const int see = __shfl_sync(0xffffffffu, kSplit ? 2 : tiles_q, 0);
      auto wait_conv = [&](uint64_t* full, int j) {
        return mbar_wait_clk(&full[j % L::kConv], (j / L::kConv) & 1, a.err);
      };
      const uint64_t dc = desc_sw128(smem_addr(smem + L::kConvOff), L::kBlockB);
      if (i < see) {
        if ((role & 1) == 0) {
          // S of page n, into the columns of page n - 2's scores and weights
          constexpr uint32_t idesc = idesc_f16_f32(kPRows, kBlk, false);
          const uint64_t q = desc_sw128(smem_addr(smem + L::kQOff + i * L::kQTileB), 16);
          for (int j = j0; j < j_end; j += kStep) {
            const int n = j / kStep;
            ok = ok && wait_conv(k_full, j) && (n < 2 || wait_values(i, n - 2));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = dc + static_cast<uint64_t>(((j % L::kConv) * 2 * L::kTileB) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tm + s_col(i, n),
                     q + static_cast<uint64_t>(((kk >> 2) * L::kQBlockB + (kk & 3) * 32) >> 4),
                     k + static_cast<uint64_t>(((kk >> 2) * L::kBlockB + (kk & 3) * 32) >> 4),
                     idesc, kk != 0);
            mma_commit_warp(&s_full[2 * i + (n & 1)]);
            mma_commit_warp(&conv_empty[j % L::kConv]);
          }
        } else {
          // O += P V of page j
          constexpr uint32_t idesc = idesc_f16_f32(kPRows, D, true);
          for (int j = j0; j < j_end; j += kStep) {
            const int n = j / kStep;
            ok = ok && wait_conv(v_full, j) &&
                 mbar_wait_clk(&p_full[2 * i + (n & 1)], (n >> 1) & 1, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v =
                dc + static_cast<uint64_t>((((j % L::kConv) * 2 + 1) * L::kTileB) >> 4);
#pragma unroll
            for (int kk = 0; kk < kBlk / 16; ++kk)
              mma_ts(tm + L::kOCol + i * 128, tm + s_col(i, n) + kk * 8,
                     v + static_cast<uint64_t>((kk * 2048) >> 4), idesc, n != 0 || kk != 0);
            mma_commit_warp(&o_done[2 * i + (n & 1)]);
            mma_commit_warp(&conv_empty[j % L::kConv]);
          }
        }
      }
    } else if (warp >= kSoftW || (kSplit && (warp & 2))) {
      // ---------------------------------------------------------- conversion
      constexpr int groups = kSplit ? 2 : 1;
      const int group = warp >= kSoftW ? 0 : 1;
      const int tid =
          (group ? (warp & 1) + ((warp >> 1) & 2) : warp - kSoftW) * 32 + lane;
      constexpr int kC = D / 16;            // 16-byte chunks of a row of codes
      constexpr int kRowStep = 128 / kC;    // rows per step
      // lanes of a row's second half take the row beside it: the stores of
      // eight lanes then cover all banks
      const int c = tid % kC, row0 = (tid / kC) ^ ((c >> 2) & 1);
      // a page's 64 rows to out: the values as code * mul (add = -1152 mul), the
      // keys as subnormals (code + 128) 2^-24, a byte beside a zero byte
      auto convert = [&](const uint4 (&v)[kBlk / kRowStep], uint8_t* out, bool keys, uint32_t mul,
                         uint32_t add) {
#pragma unroll
        for (int k = 0; k < kBlk / kRowStep; ++k) {
          const int row = row0 + k * kRowStep;
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = w[e] ^ 0x80808080u;
            const uint32_t high = keys ? 0u : 0x64646464u;
            o[2 * e] = __byte_perm(x, high, 0x4140);
            o[2 * e + 1] = __byte_perm(x, high, 0x4342);
            if (!keys) {
              asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[2 * e]) : "r"(mul), "r"(add));
              asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(o[2 * e + 1]) : "r"(mul), "r"(add));
            }
          }
          // 16-byte chunks 2c and 2c + 1 of the row's 128-byte blocks
          uint8_t* dst = out + row * 128;
          *reinterpret_cast<uint4*>(dst + ((((2 * c) & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + ((((2 * c + 1) & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      // A page's codes are in registers a page (of the group) ahead: their way from L2 (or
      // HBM) comes under the conversion of the page before, and they cross
      // shared memory once, as fp16.
      const int j_end = jt + t1 - t0;
      uint4 kv[kBlk / kRowStep], vv[kBlk / kRowStep];
      auto load_page = [&](int j) {
        const int page = rec_page[j - jt];
        const int8_t* src = a.codes + (static_cast<size_t>(page < 0 ? 0 : page) * 2 * a.hkv + hk) *
                                          L::kRawB + row0 * D + c * 16;
#pragma unroll
        for (int k = 0; k < kBlk / kRowStep; ++k) {
          kv[k] = vv[k] = make_uint4(0u, 0u, 0u, 0u);
          if (page >= 0) {
            kv[k] = ldg_v4(src + k * kRowStep * D);
            vv[k] = ldg_v4(src + static_cast<size_t>(a.hkv) * L::kRawB + k * kRowStep * D);
          }
        }
      };
      // (few rows: a page is read once, from HBM; a line per thread is
      // requested into L2 kAhead pages before)
      constexpr int kLines = L::kRawB / 128;  // of a page's keys or values
      auto request_page = [&](int j) {
        const int page = rec_page[j - jt];
        if (page >= 0 && tid < 2 * kLines)
          prefetch_l2(a.codes + ((static_cast<size_t>(page) * 2 + tid / kLines) * a.hkv + hk) *
                                    L::kRawB + tid % kLines * 128);
      };
      if (kSplit)
        for (int j = jt + group; j < jt + kAhead && j < j_end; j += groups) request_page(j);
      if (!kSplit) load_page(jt);
      for (int j = jt + group; j < j_end; j += groups) {
        const int d = j % L::kConv;
        if (kSplit) {
          if (j + kAhead < j_end) request_page(j + kAhead);
          load_page(j);
        }
        ok = ok && (j < L::kConv ||
                    mbar_wait_clk(&conv_empty[d], ((j / L::kConv) & 1) ^ 1, a.err));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* out = smem + L::kConvOff + d * (2 * L::kTileB) + (c >> 2) * L::kBlockB;
        const uint32_t hp = half_pow2((rec_e[j - jt] - E) & (wide ? 0 : -1));
        const uint32_t mul = hp | (hp << 16);
        uint32_t add;  // -1152 * 2^(e - E), exact
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(add) : "r"(mul), "r"(0xE480E480u));
        auto both = [&](const uint4 (&kc)[kBlk / kRowStep], const uint4 (&vc)[kBlk / kRowStep]) {
          convert(kc, out, true, 0u, 0u);
          if (lane == 0) mbar_arrive(&k_full[d]);
          convert(vc, out + L::kTileB, false, mul, add);
        };
        if constexpr (kSplit) {
          both(kv, vv);
        } else {
          uint4 kc[kBlk / kRowStep], vc[kBlk / kRowStep];
#pragma unroll
          for (int k = 0; k < kBlk / kRowStep; ++k) {
            kc[k] = kv[k];
            vc[k] = vv[k];
          }
          if (j + 1 < j_end) load_page(j + 1);
          both(kc, vc);
        }
        if (lane == 0) mbar_arrive(&v_full[d]);
      }
    } else if (soft) {
      // ---------------------------------------------------------- softmax
      const uint32_t o_col = tbase + lane_off + L::kOCol + qt * 128;
      const int j_end = jt + t1 - t0;
      float escale = lead == static_cast<float>(E) ? 1.f : exp2f(lead - static_cast<float>(E));
      if (wide) {
        const SoftState now = wide_pages<D, kStep>(
            smem, a, {ref, sum, lead, ok}, qt, jt, t1 - t0, tbase + lane_off, pos, cs, bias);
        ref = now.ref, sum = now.sum, lead = now.lead, ok = now.ok;
      }
      for (int j = jt + (kSplit ? qt : 0); !wide && j < j_end; j += kStep) {
        const int n = j / kStep;
        ok = ok && mbar_wait_clk(&s_full[2 * qt + (n & 1)], (n >> 1) & 1, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // the page's 64 scores in registers, read once
        const uint32_t sc = tbase + lane_off + s_col(qt, n);
        float v[64];
        tmem_ld32(sc, reinterpret_cast<uint32_t*>(v));
        tmem_ld32(sc + 32, reinterpret_cast<uint32_t*>(v) + 32);
        const PageRec rec = recs[j - jt];
        // (a scale of 0 must not turn a masked -inf into a NaN)
        const float c = fmaxf(cs * rec.ks * kUp, 1e-37f);
        tmem_wait_ld();
        if (!(rec.meta >= 0 && ((rec.meta >> qt) & 1))) {
          const uint64_t see = rec.meta >= 0 ? kv_mask(a, pos, (rec.meta >> 2) * kBlk) : 0;
          const uint32_t see0 = static_cast<uint32_t>(see);
          const uint32_t see1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!(see0 & (1u << k))) v[k] = -INFINITY;
            if (!(see1 & (1u << k))) v[k + 32] = -INFINITY;
          }
        }
        float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int k = 4; k < 64; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m4[e] = fmaxf(fmaxf(m4[e], v[k + e]), k + e + 4 < 64 ? v[k + e + 4] : v[k + e]);
        const float big = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float top = (big - bias) * c;  // -inf: no visible token
        const bool raise = top > ref + kPLazy;
        if (__any_sync(0xffffffffu, raise || escale != 1.f)) {
          float alpha = escale;
          escale = 1.f;
          lead = static_cast<float>(E);
          if (raise) {
            const float f = exp2_approx(ref - top);  // 0 for the row's first
            alpha *= f;
            sum *= f;
            ref = top;
          }
          if (n > 0) {
            // O has to hold everything up to the page before
            ok = ok && wait_values(qt, n - 1);
            tc_fence_after();
            rescale_row<D>(o_col, alpha);
          }
        }
        const float add = fmaf(-bias, c, kPOff + rec.lf - (ref == -INFINITY ? 0.f : ref));
        const uint64_t c2 = pair_f32(c, c), add2 = pair_f32(add, add);
        uint64_t s2[2] = {0, 0};  // pairs of sums from +0
        uint32_t pw[32];
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          float p0, p1;
          unpair_f32(fma_pair(pair_f32(v[k], v[k + 1]), c2, add2), p0, p1);
          p0 = exp2_approx(p0);
          p1 = exp2_approx(p1);
          s2[(k >> 1) & 1] = add_pair(s2[(k >> 1) & 1], pair_f32(p0, p1));
          pw[k / 2] = half2_bits(p0, p1);
        }
        tmem_st32(sc, pw);
        float s0, s1;
        unpair_f32(add_pair(s2[0], s2[1]), s0, s1);
        // (scales that cannot be used have 1 / f = NaN: the rows that see the
        // page, and only they, become NaN)
        if (big != -INFINITY) sum = fmaf(s0 + s1, rec.rf, sum);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * qt + (n & 1)]);
      }
    }
    __syncwarp();  // one-thread roles
    jt += t1 - t0;
  }

  // ---- results
  if (warp >= kMmaW) {
    __syncwarp();
    mma_commit_warp(mma_end);  // every MMA of the CTA has run before TMEM is freed
    mbar_wait_clk(mma_end, 0, a.err);
  }
  __syncwarp();
  if (kSplit) cta_barrier();  // no converted page is read any more
  // A part: O in chunks of four elements, [D / 4][rows], then (ref, sum).
  constexpr size_t kPart = 2 * kPRows * (D + 2);
  const OutRows<D> put{a, smem + L::kQOff, r0, sq.row0, hk};
  int out0 = 0, out1 = 0;  // the staged rows that this warp writes
  if (soft) {
    const bool mine_out = !(kSplit && qt);  // (tile 0 writes for both)
    // both tiles' softmax warps
    auto softmax_barrier = [&] {
      asm volatile("bar.sync 1, %0;" ::"r"(64 * soft_warps(0)) : "memory");
    };
    const uint32_t o_col = tbase + lane_off + L::kOCol + qt * 128;
    float* mine = partials + static_cast<size_t>(tail < 0 ? 0 : tail) * kPart;
    const int n = kSplit ? (jt + 1 - qt) >> 1 : jt;  // pages of the tile
    const bool have = n > 0 && __all_sync(0xffffffffu, ok && wait_values(qt, n - 1));
    tc_fence_after();
    float inv = sum == 0.f ? 0.f : exp2f(lead) / sum;
    float inv1 = 0.f;  // tile 1's share of the sum
    // tile 1's sixteen columns q of the row, in the converted pages' place
    float4* other = reinterpret_cast<float4*>(smem + L::kConvOff) + tr;
    if (kSplit && qt == 0) {
      softmax_barrier();  // (tile 1 has written)
      const float2 ms = *reinterpret_cast<const float2*>(other + (D / 4) * kPRows);
      const float top = fmaxf(ref, ms.x), base = top == -INFINITY ? 0.f : top;
      const float w0 = sum * exp2f(ref - base), w1 = ms.y * exp2f(ms.x - base);
      const float all = w0 + w1;
      inv = all == 0.f ? 0.f : inv * (w0 / all);
      inv1 = all == 0.f ? 0.f : w1 / all;
      ref = top;
      sum = all;
    }
#pragma unroll 2
    for (int q = 0; q < D / 16; ++q) {
      uint32_t x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = 0u;
      if (have) {
        tmem_ld16(o_col + 16 * q, x);
        tmem_wait_ld();
      }
      float f[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) f[k] = __uint_as_float(x[k]) * inv;
      if (kSplit) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4* o = other + (4 * q + k) * kPRows;
          if (qt) {
            *o = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
          } else {
            const float4 y = *o;
            f[4 * k] = fmaf(y.x, inv1, f[4 * k]);
            f[4 * k + 1] = fmaf(y.y, inv1, f[4 * k + 1]);
            f[4 * k + 2] = fmaf(y.z, inv1, f[4 * k + 2]);
            f[4 * k + 3] = fmaf(y.w, inv1, f[4 * k + 3]);
          }
        }
      }
      if (!mine_out) {
      } else if (live && parts == 1) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_out(a.type, f[2 * k], f[2 * k + 1]);
        if (kSplit) {  // (few rows: straight to their places)
          uint4* o =
              reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + put.row(r) * D + 16 * q);
          o[0] = make_uint4(w[0], w[1], w[2], w[3]);
          o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          *reinterpret_cast<uint4*>(put.staged(r, 2 * q)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(put.staged(r, 2 * q + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      } else if (live) {
        float4* o = reinterpret_cast<float4*>(mine) + 4 * q * (2 * kPRows) + r;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k * (2 * kPRows)] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
      }
    }
    if (!kSplit && parts == 1) {
      out0 = r - lane;
      out1 = rows < out0 + 32 ? rows : out0 + 32;
    }
    if (kSplit && qt) {
      *reinterpret_cast<float2*>(other + (D / 4) * kPRows) = make_float2(ref, sum);
      softmax_barrier();
    }
    if (mine_out && live && parts > 1)
      reinterpret_cast<float2*>(mine + 2 * kPRows * D)[r] = make_float2(ref, sum);
    if (mine_out && live && parts == 1 && a.lse) a.lse[put.row(r)] = kv_log_sum(ref, sum, kPOff);
  }
  __syncwarp();
  if (parts > 1) {
    // The last part to arrive adds them all in order.
    __threadfence();
    cta_barrier();
    if (threadIdx.x == 0)
      *is_last = atomic_add_acq_rel_gpu(&tickets[item - whole], 1) == parts - 1;
    cta_barrier();
    if (*is_last) {
      if (threadIdx.x == 0) tickets[item - whole] = 0;
      join_parts<D>(a, smem, partials + static_cast<size_t>(item - whole) * tail_parts * kPart, parts,
                    rows, r0, sq.row0, hk);
      cta_barrier();
      static_assert(kPThreads / 32 * 16 == 2 * kPRows, "rows of a warp");
      out0 = 16 * warp;
      out1 = rows < out0 + 16 ? rows : out0 + 16;
    }
  }
  __syncwarp();
  put.write_out(lane, out0, out1);
  __syncwarp();
  tc_fence_before();
  cta_barrier();
  tc_fence_after();
  if (warp == kMmaW) tmem_dealloc(tbase, 512);
}

}  // namespace

size_t kv8_prompt_partial_bytes(int dim) {
  return static_cast<size_t>(2 * kSmallTMaxCtas) * 2 * kPRows * (dim + 2) * sizeof(float);
}

// Blocks of rows of a sequence, a CTA each (and more where the last wave is cut).
static long long row_blocks_of(long long max_new, int group) {
  return (max_new * group + 2 * kPRows - 1) / (2 * kPRows);
}

bool kv8_prompt_fits(int max_new, int group, int kv_heads, int seqs) {
  return row_blocks_of(max_new, group) * kv_heads <=
         (0x7FFFFFFFll - 2 * kSmallTMaxCtas) / seqs;
}

cudaError_t kv8_prompt_set_attributes() {
  const auto allow = [](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = allow(kv8_prompt_kernel<64, false>, PL<64>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_prompt_kernel<64, true>, PL<64>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_prompt_kernel<128, false>, PL<128>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_prompt_kernel<128, true>, PL<128>::kAlloc);
  return e;
}

cudaError_t launch_kv8_prompt(const Kv8Args& a, int min_rows, float* partials, int* tickets,
                              int num_sms, cudaStream_t stream, int* launches) {
  const long long most = static_cast<long long>(a.max_new) * a.group;
  const long long row_blocks = row_blocks_of(a.max_new, a.group);
  // Whole waves of items run as they are.  The keys of the items left (the
  // earliest rows, the last to start) are cut into parts so that they end
  // together: as many as cost the least pages of time in sequence on an SM (at
  // the table's width; the kernel leaves blocks of few pages whole).
  // Measured when it came, with the cut and without (2048 tokens of 6 heads over
  // 8190, 384 items on 152 SMs): 316 and 328 us; 4096 tokens over 16384: 1106 and
  // 1227 us.
  const long long items = row_blocks * a.hkv * a.seqs;
  const long long sms = num_sms < kSmallTMaxCtas ? num_sms : kSmallTMaxCtas;
  const long long tail = items % sms, whole = items - tail;
  unsigned parts = 1, best = a.width;
  // (the join holds a weight per part and row in the converted pages' place)
  const long long rows32 = most < 2 * kPRows ? (most + 31) / 32 * 32 : 2 * kPRows;
  const long long room = 2 * PL<64>::kConv * PL<64>::kTileB / 4 / rows32;
  static_assert(PL<64>::kConv * PL<64>::kTileB <= PL<128>::kConv * PL<128>::kTileB, "room");
  for (unsigned p = 2; p * tail <= 2 * sms && p <= static_cast<unsigned>(a.width) / kPartPages &&
                       p <= room;
       ++p) {
    const unsigned cost = part_cost(a.width, p, static_cast<unsigned>(tail),
                                    static_cast<unsigned>(sms));
    if (cost < best) best = cost, parts = p;
  }
  const long long grid = whole + tail * parts;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_launch_config(attr, dim3(static_cast<unsigned>(grid)), dim3(kPThreads),
                        a.dim == 128 ? PL<128>::kAlloc : PL<64>::kAlloc, stream);
  const auto kernel = most <= kSplitRows
                          ? (a.dim == 128 ? kv8_prompt_kernel<128, true> : kv8_prompt_kernel<64, true>)
                          : (a.dim == 128 ? kv8_prompt_kernel<128, false>
                                          : kv8_prompt_kernel<64, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, min_rows, static_cast<int>(row_blocks),
                                           static_cast<int>(whole), static_cast<int>(parts),
                                           static_cast<int>(tail), static_cast<int>(sms),
                                           partials, tickets);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace tern
