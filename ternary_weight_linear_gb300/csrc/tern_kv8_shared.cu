// tern_kv8_attention_shared: attention of a batch whose sequences begin with the
// same pages.
//
// A row's softmax over the prefix and over its sequence's own tokens are parts
// of one softmax: with O_p the output of part p and W_p = sum 2^s the weight of
// its scores,
//   o = sum_p (W_p / W) O_p,  W = sum_p W_p.
// So the prefix is one "sequence" of all rows of the batch, whose every cache
// byte is read once, cut into parts along its tokens; the own tokens are short
// spans of few rows each.  All parts go to the workspace in fp32 and one launch
// joins them (a CTA that joined all parts of 256 rows, as the last of them,
// read 2 MB through one SM: 50 us of 109 at 32 sequences of 6 query heads a
// key-value head behind 16384 tokens).
//
// The launches:
//   the prefix on the tensor cores (kv8_prompt_kernel), where it is long for
//   the batch's rows (kSpanPrefixUnits); otherwise it is spans too;
//   spans (kv8_span_kernel), of sequences of up to kSpanRows rows, beside the
//   former: it waits for it at its end only;
//   longer sequences' own tokens by kv8_prompt_kernel;
//   the join.
//
// Measured, 32 sequences of 40 to 1500 tokens (6 query heads on each of 8 key-value
// heads of 128) behind 16384: 36.8 us; every page's codes once are 12.7 at the copy
// rate, each sequence for itself takes 150.  Alone, the prefix's launch
// (80 CTAs) takes 33 us, 1700 cycles a page, whose scores' products read the queries
// from shared memory: its tensor pipe is 48 % busy.  The spans beside it take 30, of
// which some 5 go until the first codes arrive, three warps a scheduler; the join 5
// to 8, dependent reads from L2.
#include "tern_kv8_half.cuh"

namespace tern {
namespace {

constexpr int kSW = 3;           // warps of a span's CTA
constexpr int kSThreads = 32 * kSW;
constexpr int kSpanRecs = 32;    // pages whose records are held at a time
// CTAs of spans that an SM holds, by their tiles of rows (registers and rings).
constexpr int span_ctas(int tiles) { return 5 - tiles; }
constexpr int kSpanPages = 2;    // pages of a span at least, where there are more
// Halvings of the range that a quota is looked for in (each costs 0.05 us; 32 sequences
// of up to 2000 tokens behind 128 take 40.9 us with none, 34.2 with two, 32.7 with four).
constexpr int kQuotaSteps = 4;
// A prefix of up to this many pages, times key-value heads and groups of rows (twice
// of 24 rows), is spans as well, where a CTA for each and one for each of the own
// tokens' are resident at once.  Measured, as spans and on the tensor cores, in us: 4
// sequences of 6 rows behind 2048 tokens (768 of the units) 11.3 and 13.6; 6 (1280)
// 12.7 and 14.1; 8 (1536) 13.7 and 13.7; 8 behind 4096 17.4 and 15.0; 2 of 24 rows
// behind 4096 (twice 1024) 17.8 and 16.5; 32 of 20 rows behind 256, 472 CTAs where 304
// are resident, 28.6 and 20.3.
constexpr long long kSpanPrefixUnits = 1500;

// The pages of a span's list: [s0, s1), then from f0 on.
struct SpanPages {
  int s0, s1, f0, count;
  __device__ __forceinline__ int page(int i) const {
    return i < s1 - s0 ? s0 + i : f0 + i - (s1 - s0);
  }
};

// One part of the prefix (for rows of the whole batch) or of a sequence's own
// tokens: up to 8 NT rows of a key-value head over a range of pages.  Bound by
// the cache's bytes where there are many pages, by latency elsewhere: small CTAs
// without barriers in the loop, of which an SM holds several, so that one's
// dependent reads (lengths, table, scales, codes) pass under another's work.
// Each warp takes every third half-page through a ring of TMA boxes of its own,
// kStages ahead.  (Loads straight to the registers of the tensor instructions,
// the values' under the scores and the next keys' under the values, left each
// half-page waiting for its values: 52 us instead of 47 for 32 sequences behind
// 16384 tokens, with 40 to 1500 of their own.)
template <int D, int NT>
struct Span {
  static constexpr int kRows = 8 * NT;
  static constexpr int kW = D / 16;
  static constexpr int kMT = D / 16;
  static constexpr int kQStride = 2 * D + 16;
  static constexpr int kMStride = D + 4;
  static constexpr bool kBiased = biased(NT);

  static constexpr int kFar = 1 << 30;  // (a place has less: 2^31 over a page's rows)
  static constexpr int kStage = 2 * kHalf * D;  // bytes: keys, then values
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRing = kSW * kStages * kStage;
  static_assert(kSW * 8 * kMStride * sizeof(float) <= kRing, "the merge is in the ring's place");

  struct Smem {
    alignas(1024) uint8_t ring[kRing];  // [warp][stage]
    alignas(16) uint8_t q[kRows * kQStride];
    uint64_t full[kSW][kStages];
    alignas(16) PageRec recs[kSpanRecs];
    int blk[kSpanRecs];   // its place among the cache's (page, keys, head), kFar; -1: none
    int meta[kSpanRecs];  // its number in the sequence * 16, kMHalf, kMAll
    float2 ml[kSW][kRows];
    float fac[kRows][kSW];
    float weight[kRows], qscale[kRows];
    int pos[kRows];
    int range[2];
    int far;
  };

  const CUtensorMap& tm;
  const Kv8Args& a;
  Smem& sm;
  int warp, lane, g, t;
  int hk, slot, table_row;  // key-value head, part, row of the page table
  int n0, rows;             // first row (of the head's) and how many
  int p_first, p_last;
  SpanPages pages;

  // (whole warp) half h & 1 of the page at blk into stage n % kStages of the warp's
  // ring
  __device__ __forceinline__ void request(int blk, int h, unsigned n) const {
    if (lane == 0) {
      uint64_t* full = &sm.full[warp][n % kStages];
      uint8_t* to = sm.ring + (warp * kStages + n % kStages) * kStage;
      const int row = blk * kBlk + (h & 1) * kHalf;
      mbar_arrive_expect_tx(full, kStage);
      tma_load_2d(to, &tm, 0, row, full);
      tma_load_2d(to + kHalf * D, &tm, 0, row + a.hkv * kBlk, full);
    }
  }

  // The rows' queries in fp16, each scaled by a power of two; a row per warp.
  // between: what is done while they are on their way.
  template <typename Between>
  __device__ __forceinline__ void stage_queries(const Between& between) {
    constexpr int kX = (kRows + kSW - 1) / kSW;
    uint32_t raw[kX][D / 64];
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      const int r = warp + x * kSW;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) raw[x][e] = 0u;
      if (r < rows) {
        const int tok = kv_token(a, n0 + r);
        const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                              static_cast<long long>(tok) * a.ld +
                              static_cast<long long>(hk * a.group + n0 + r - tok * a.group) * a.hd +
                              lane * (D / 32);
        if constexpr (D == 128) {
          const uint2 w = *reinterpret_cast<const uint2*>(src);
          raw[x][0] = w.x, raw[x][1] = w.y;
        } else {
          raw[x][0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
    }
    between();
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      const int r = warp + x * kSW;
      if (r >= kRows) break;
      uint32_t m2 = 0;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) m2 = __vmaxu2(m2, raw[x][e] & 0x7FFF7FFFu);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, k));
      const int up = q_exponent((m2 & 0xFFFFu) > (m2 >> 16) ? m2 & 0xFFFFu : m2 >> 16, a.type);
      const float f = pow2f(up);
      uint32_t* dst = reinterpret_cast<uint32_t*>(sm.q + r * kQStride);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        float lo, hi;
        unpack16(raw[x][e], a.type, lo, hi);
        const int word = lane * (D / 64) + e;
        const int unit = word >> 1;  // (placed as staged_query reads it)
        dst[((unit ^ (unit / (D / 8))) << 1) | (word & 1)] = half2_bits(lo * f, hi * f);
      }
      if (lane == 0) sm.qscale[r] = pow2f(-up);
    }
  }

  // A thread's page of the table: entry c0 + threadIdx.x of the list, of n.
  __device__ __forceinline__ int table_page(int c0, int n) const {
    static_assert(kSpanRecs <= kSThreads, "a page per thread");
    if (static_cast<int>(threadIdx.x) >= n) return -1;
    return a.table[static_cast<size_t>(table_row) * a.width + pages.page(c0 + threadIdx.x)];
  }
  // Its record.
  __device__ __forceinline__ void make_record(int c0, int n, int page) {
    const int i = threadIdx.x;
    if (i >= n) return;
    const int lp = pages.page(c0 + i);
    PageRec rec = {0.f, 0.f, 1.f, 0.f};
    int blk = -1, meta = lp * 16;
    if (page < 0 || page >= a.pages) {
      atomicOr(a.err, kErrIndex);
    } else {
      blk = page * 2 * a.hkv + hk;
      const float ks = a.scales[blk], vs = a.scales[blk + a.hkv];
      const bool far = far_scales(ks, vs);
      if (far) sm.far = 1;
      rec = page_rec(ks, vs);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int j0 = lp * kBlk + hf * kHalf, j1 = j0 + kHalf - 1;
        if (kv_any(a, p_first, p_last, j0, j1)) meta |= kMHalf << hf;
        if (!far && kv_all(a, p_first, p_last, j0, j1)) meta |= kMAll << hf;
      }
      if (far) blk |= kFar;
    }
    sm.recs[i] = rec;
    sm.blk[i] = blk;
    sm.meta[i] = meta;
  }

  // Pages [begin, end) of the list, into part `slot` of the rows.
  __device__ __forceinline__ void run(int begin, int end) {
    // the first pages' and the queries' dependent reads side by side
    const int n_first = end - begin < kSpanRecs ? end - begin : kSpanRecs;
    const int page = table_page(begin, n_first);
    // each warp's first half-pages are requested as soon as it has read where they
    // are: lane l < kStages, the l-th
    unsigned issued = 0, used = 0;  // stages of the warp's ring
    const int h_lane = warp + lane * kSW;
    int at_lane = -1;
    if (lane < kStages && h_lane < 2 * n_first)
      at_lane = a.table[static_cast<size_t>(table_row) * a.width + pages.page(begin + (h_lane >> 1))];
    stage_queries([&] {
      int blk = -1;
      if (at_lane >= 0 && at_lane < a.pages) {
        const int j0 = pages.page(begin + (h_lane >> 1)) * kBlk + (h_lane & 1) * kHalf;
        if (kv_any(a, p_first, p_last, j0, j0 + kHalf - 1)) blk = at_lane * 2 * a.hkv + hk;
      }
#pragma unroll
      for (int l = 0; l < kStages; ++l) {
        const int at = __shfl_sync(0xffffffffu, blk, l);
        if (at >= 0) request(at, warp + l * kSW, issued++);
      }
      make_record(begin, n_first, page);
    });
    __syncthreads();

    uint2 qf[NT == 1 ? kW : 1];  // one tile's query fragments
#pragma unroll
    for (int j = 0; NT == 1 && j < kW; ++j) qf[j] = staged_query<D>(sm.q, 0, j, g, t);
    auto query = [&](int n, int j) {
      if (NT == 1) return qf[j];
      return staged_query<D>(sm.q, n, j, g, t);
    };
    float o[NT][kMT][4];
    float ref[NT][2], sum[NT][2], cs[NT][2], s0[NT][4];
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * n + 2 * t + x;
        ref[n][x] = -INFINITY;
        sum[n][x] = 0.f;
        cs[n][x] = sm.qscale[r] * a.scale_log2;
        pos[n][x] = sm.pos[r];
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][i][x] = 0.f;
      query_bias<D, kBiased>([&](int j) { return query(n, j); }, s0[n]);
    }

    constexpr float kUp = kBiased ? kCodeUp : 1.f;  // 1 over the codes' unit
    for (int c0 = begin; c0 < end; c0 += kSpanRecs) {
      const int n_here = end - c0 < kSpanRecs ? end - c0 : kSpanRecs;
      if (c0 > begin) {
        __syncthreads();  // the records before have been read
        make_record(c0, n_here, table_page(c0, n_here));
        __syncthreads();
      }
      const int h_end = 2 * n_here;
      auto next = [&](int h) {  // the warp's half-page from h on that some row sees
        while (h < h_end && !(sm.meta[h >> 1] & (kMHalf << (h & 1)))) h += kSW;
        return h;
      };
      int h = next(warp), ahead = next(c0 == begin ? warp + kStages * kSW : warp);
      for (; ahead < h_end && issued - used < kStages; ahead = next(ahead + kSW))
        request(sm.blk[ahead >> 1] & ~kFar, ahead, issued++);
      for (; h < h_end; h = next(h + kSW)) {
        const PageRec rec = sm.recs[h >> 1];
        const int meta = sm.meta[h >> 1];
        const uint8_t* kb = sm.ring + (warp * kStages + used % kStages) * kStage;
        const bool ok = __all_sync(
            0xffffffffu, mbar_wait_clk(&sm.full[warp][used % kStages], (used / kStages) & 1, a.err));
        if (!ok) break;
        float sc[NT][2][4];
        {
          uint32_t kw[4][kW];
          half_keys<D>(kb, g, t, kw);
          half_scores<D, NT>(kw, s0, sc, query);
        }
        if (!(meta & (kMAll << (h & 1)))) {
          if (sm.blk[h >> 1] & kFar) {  // left to far_row: none of it here
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < 8; ++x) sc[n][x >> 2][x & 3] = -INFINITY;
          } else {
            half_mask<NT>(a, pos, (meta >> 4) * kBlk + (h & 1) * kHalf, g, sc);
          }
        }
        // the values' codes, on their way under the softmax
        uint32_t vw[2][4][D / 32];
        half_values<D>(kb + kHalf * D, g, t, vw);
        half_softmax<D, NT>(rec, cs, sc, ref, sum, o);
        half_products<D, NT>(sc, half2_bits(rec.any, rec.any), vw, o);
        __syncwarp();  // the stage has been read
        ++used;
        if (ahead < h_end) {
          request(sm.blk[ahead >> 1] & ~kFar, ahead, issued++);
          ahead = next(ahead + kSW);
        }
      }
    }
    // (after a wait that ran out: no copy outlives the CTA)
    for (; used < issued; ++used)
      if (!mbar_wait_clk(&sm.full[warp][used % kStages], (used / kStages) & 1, a.err)) break;

    // ---- the warps' results to one
    float* merge = reinterpret_cast<float*>(sm.ring);  // (behind the barrier below)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) sum[n][x] += __shfl_xor_sync(0xffffffffu, sum[n][x], k);
        if (g == 0) sm.ml[warp][8 * n + 2 * t + x] = make_float2(ref[n][x], sum[n][x]);
      }
    __syncthreads();
    if (threadIdx.x < kRows) {  // (the ring has been read, by every warp)
      const int r = threadIdx.x;
      float big = -INFINITY, l = 0.f, f[kSW];
#pragma unroll
      for (int w = 0; w < kSW; ++w) {
        const float2 v = sm.ml[w][r];
        if (v.y != 0.f) big = fmaxf(big, v.x);
      }
      const float base = big == -INFINITY ? 0.f : big;
#pragma unroll
      for (int w = 0; w < kSW; ++w) {
        const float2 v = sm.ml[w][r];
        f[w] = v.y == 0.f ? 0.f : exp2f(v.x - base);
        if (v.y != 0.f) l = fmaf(v.y, f[w], l);
      }
#pragma unroll
      for (int w = 0; w < kSW; ++w) sm.fac[r][w] = l == 0.f ? 0.f : f[w] / l;
      sm.weight[r] = part_weight(base, l);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int q = 0; q < D / 32; ++q)
          *reinterpret_cast<float4*>(merge + (warp * 8 + 2 * t + x) * kMStride + (D / 8) * g +
                                     4 * q) =
              make_float4(kUp * o[n][2 * q][x], kUp * o[n][2 * q][x + 2], kUp * o[n][2 * q + 1][x],
                          kUp * o[n][2 * q + 1][x + 2]);
      __syncthreads();
      for (int i = threadIdx.x; i < 8 * (D / 4); i += kSThreads) {
        const int row = i / (D / 4), c = i % (D / 4);
        if (8 * n + row >= rows) break;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSW; ++w) {
          const float f = sm.fac[8 * n + row][w];
          const float4 v =
              *reinterpret_cast<const float4*>(merge + (w * 8 + row) * kMStride + 4 * c);
          if (f != 0.f) {
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
        }
        *kv_part_o(a, hk, slot, c, n0 + 8 * n + row) = acc;
      }
      if (n + 1 < NT) __syncthreads();
    }
    if (sm.far) {
      // the pages left out join what has been written beside them
      __syncthreads();
      for (int r = warp; r < rows; r += kSW) {
        const FarRow<D> f =
            far_row<D>(a, sm.q + r * kQStride, sm.qscale[r] * a.scale_log2, sm.pos[r], table_row, hk,
                       pages, begin, end);
        constexpr int kV = D / 32;
        float* to = reinterpret_cast<float*>(kv_part_o(a, hk, slot, lane * kV / 4, n0 + r)) +
                    lane * kV % 4;
        const float was = sm.weight[r], now = part_weight(f.ref, f.sum);
        const float top = fmaxf(was, now), base = top == -INFINITY ? 0.f : top;
        const float w0 = exp2f(was - base), w1 = exp2f(now - base), l = w0 + w1;
        const float f0 = l == 0.f ? 0.f : w0 / l, f1 = l == 0.f ? 0.f : w1 / l;
#pragma unroll
        for (int y = 0; y < kV; ++y) to[y] = to[y] * f0 + f.o[y] * f1;
        __syncwarp();
        if (lane == 0) sm.weight[r] = part_weight(base, l);
      }
      __syncthreads();
    }
    write_weights(false);
  }

  // (every thread) none: the part has no pages
  __device__ __forceinline__ void write_weights(bool none) {
    const int r = threadIdx.x;
    if (r < rows) *kv_part_w(a, hk, slot, n0 + r) = none ? -INFINITY : sm.weight[r];
  }
};

// The pages that rows at positions p_first to p_last see, before the prefix's end
// or behind it.
__device__ __forceinline__ SpanPages span_pages(const Kv8Args& a, bool prefix, int p_first,
                                                int p_last) {
  const int common = a.shared / kBlk;
  int first = 0, sinks = 0;
  if (a.window > 0 && p_first >= a.window) {
    first = (p_first - a.window + 1) / kBlk;
    const int n = a.sinks / kBlk + (a.sinks % kBlk != 0);
    sinks = n < first ? n : first;
  }
  SpanPages v;
  int stop;
  if (prefix) {
    v.f0 = first < common ? first : common;
    v.s0 = 0;
    v.s1 = sinks < v.f0 ? sinks : v.f0;
    stop = common;
  } else {
    v.f0 = first > common ? first : common;
    v.s0 = common;
    v.s1 = sinks > common ? sinks : common;
    stop = p_last / kBlk + 1;
  }
  v.count = v.s1 - v.s0 + stop - v.f0;
  return v;
}

// CTAs of spans that are resident at once: beside the prefix's launch, and after it;
// the launch is for the former if that takes no spans of more than `longest` pages.
struct SpanSlots {
  int free, all, longest;
};

// The spans of the sequences' own tokens: those of a sequence with pages and rows
// for the kernel are cut into parts of `quota` pages and fewer, the same for all,
// so that a launch has about as many spans as CTAs are resident at once, of about the
// same length, however long the sequences are; but into no more parts than the
// workspace holds of every row (kSpanPartRows): of 256 rows of 48 heads 3, from 427 on 1.
// There a sequence that is far longer than the others has the launch's longest spans:
// 256 sequences of up to 300 tokens behind 4096 94 us, with one of 32000 among them 208;
// behind 64 70 and 195 (each for itself 106 and 137).
struct OwnJob {
  int seq, part, parts, group, hk;
  KvSeq s;
  SpanPages pages;
};
template <int kRows>
struct OwnJobs {
  const Kv8Args& a;
  SpanSlots slots;
  int max_parts, max_rows;
  // sequence i's pages and row groups (none: 0)
  __device__ __forceinline__ void sequence(int i, KvSeq& s, SpanPages& pages, int& groups) const {
    groups = 0;
    pages = {0, 0, 0, 0};
    s = {0, 0, 0, true};
    if (i >= a.seqs) return;
    s = kv_seq(a, i);
    const int rows = s.m * a.group;
    if (s.ok && s.m > 0 && rows <= max_rows) {
      groups = static_cast<unsigned>(rows + kRows - 1) / kRows;
      pages = span_pages(a, false, a.shared + s.len - s.m, a.shared + s.len - 1);
    }
  }
  // Job x, false if there are not as many.  Every warp finds it for itself, 32
  // sequences at a time: no barrier, and few reads one after the other.
  __device__ __forceinline__ bool find(unsigned x, OwnJob& job) const {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    SpanPages pages;
    KvSeq s;
    int groups;
    // all pages (times heads and groups), and the spans if no sequence were cut;
    // the same order of the same sums in every warp
    float all = 0.f, least = 0.f;
    int top = 0;  // pages of the longest sequence
    for (int i0 = 0; i0 < a.seqs; i0 += 32) {
      sequence(i0 + lane, s, pages, groups);
      if (!s.ok && x == 0) atomicOr(a.err, kErrIndex);
      all += static_cast<float>(pages.count) * static_cast<float>(groups);
      least += static_cast<float>(groups);
      if (groups > 0 && pages.count > top) top = pages.count;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      all += __shfl_xor_sync(kAll, all, k);
      least += __shfl_xor_sync(kAll, least, k);
    }
    top = __reduce_max_sync(kAll, top);
    all *= static_cast<float>(a.hkv);
    least *= static_cast<float>(a.hkv);
    // The quota that makes `most` spans: with most - least of them for the cuts it
    // makes no more, whatever the lengths are; up to 32 sequences are counted for less.
    int quota;
#pragma unroll 1
    for (int slot = slots.free;; slot = slots.all) {
      const float most = static_cast<float>(slot);
      const float room = fmaxf(most - least, 0.25f * most);
      quota = max(kSpanPages, static_cast<int>(fminf(ceilf(all / room), 1e9f)));
      if (a.seqs <= 32) {
        if (quota > top) quota = max(kSpanPages, top);
        int low = max(kSpanPages, static_cast<int>(fminf(ceilf(all / most), 1e9f)));
#pragma unroll 1
        for (int step = 0; step < kQuotaSteps && low < quota; ++step) {
          const int q = (low + quota) >> 1;
          const unsigned cut =
              static_cast<unsigned>(pages.count + q - 1) / static_cast<unsigned>(q);
          const unsigned spans = __reduce_add_sync(kAll, cut * groups);
          if (static_cast<float>(spans) * a.hkv <= most)
            quota = q;
          else
            low = q + 1;
        }
      }
      if (min(quota, top) <= slots.longest || slot == slots.all) break;
    }
    unsigned before = 0;
    for (int i0 = 0; i0 < a.seqs; i0 += 32) {
      if (a.seqs > 32) sequence(i0 + lane, s, pages, groups);
      const unsigned cut =
          (static_cast<unsigned>(pages.count) + quota - 1) / static_cast<unsigned>(quota);
      const unsigned parts = cut < static_cast<unsigned>(max_parts) ? cut : max_parts;
      const unsigned mine = groups > 0 ? parts * groups * a.hkv : 0u;
      unsigned end = mine;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const unsigned up = __shfl_up_sync(kAll, end, k);
        if (lane >= k) end += up;
      }
      const unsigned here = __ballot_sync(kAll, x - before - (end - mine) < mine);
      if (here) {
        const int from = __ffs(here) - 1;
        unsigned at = x - before - __shfl_sync(kAll, end - mine, from);
        job.seq = i0 + from;
        job.parts = __shfl_sync(kAll, static_cast<int>(parts), from);
        groups = __shfl_sync(kAll, groups, from);
        const unsigned rest = at / static_cast<unsigned>(job.parts);
        job.part = at - rest * job.parts;
        job.hk = rest / static_cast<unsigned>(groups);
        job.group = rest - job.hk * groups;
        job.s.len = __shfl_sync(kAll, s.len, from);
        job.s.m = __shfl_sync(kAll, s.m, from);
        job.s.row0 = __shfl_sync(kAll, s.row0, from);
        job.pages.s0 = __shfl_sync(kAll, pages.s0, from);
        job.pages.s1 = __shfl_sync(kAll, pages.s1, from);
        job.pages.f0 = __shfl_sync(kAll, pages.f0, from);
        job.pages.count = __shfl_sync(kAll, pages.count, from);
        return true;
      }
      before += __shfl_sync(kAll, end, 31);
    }
    return false;
  }
};

template <int D, int NT>
__device__ __forceinline__ void span_part(const CUtensorMap& tm, const Kv8Args& a,
                                          int prefix_groups, const SpanSlots& slots,
                                          int max_rows) {
  using S = Span<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(
      smem_raw + (-smem_addr(smem_raw) & 1023u));
  const int lane = threadIdx.x & 31;
  S s{tm, a, sm, static_cast<int>(threadIdx.x >> 5), lane, lane >> 2, lane & 3};
  if (threadIdx.x == 0) sm.far = 0;  // (a barrier follows before it is set)
  if (lane == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(&sm.full[s.warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int pre = a.prefix_parts * prefix_groups * a.hkv;  // CTAs of the prefix
  int part, parts;
  if (static_cast<int>(blockIdx.x) < pre) {
    int x = static_cast<int>(blockIdx.x);
    parts = a.prefix_parts;
    part = x % parts;
    x /= parts;
    const int r0 = x % prefix_groups * S::kRows;
    s.hk = x / prefix_groups;
    s.table_row = 0;
    s.slot = part;
    // the rows' positions: those of the sequences that have them, -1 elsewhere
    const int R = a.rows * a.group;
    s.n0 = r0;
    s.rows = R - r0 < S::kRows ? R - r0 : S::kRows;
    if (threadIdx.x < S::kRows) sm.pos[threadIdx.x] = -1;
    if (threadIdx.x == 0) sm.range[0] = 0x7FFFFFFF, sm.range[1] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.seqs; i += kSThreads) {
      const KvSeq q = kv_seq(a, i);
      if (!q.ok || q.m == 0) continue;
      const long long first = static_cast<long long>(q.row0) * a.group;
      const long long last = first + static_cast<long long>(q.m) * a.group;
      for (int r = 0; r < s.rows; ++r) {
        if (r0 + r < first || r0 + r >= last) continue;
        const int p = a.shared + q.len - q.m + kv_token(a, r0 + r) - q.row0;
        sm.pos[r] = p;
        atomicMin(&sm.range[0], p);
        atomicMax(&sm.range[1], p);
      }
    }
    __syncthreads();
    s.p_first = sm.range[0];
    s.p_last = sm.range[1];
    if (s.p_last < 0) {
      s.write_weights(true);
      return;
    }
    s.pages = span_pages(a, true, s.p_first, s.p_last);
  } else {
    OwnJob job;
    const OwnJobs<S::kRows> jobs{a, slots, a.parts - a.prefix_parts, max_rows};
    if (!jobs.find(blockIdx.x - pre, job)) return;
    part = job.part;
    parts = job.parts;
    s.hk = job.hk;
    s.table_row = job.seq;
    s.slot = a.prefix_parts + part;
    s.pages = job.pages;
    const int r0 = job.group * S::kRows, R = job.s.m * a.group;
    s.n0 = job.s.row0 * a.group + r0;
    s.rows = R - r0 < S::kRows ? R - r0 : S::kRows;
    s.p_first = a.shared + job.s.len - job.s.m;
    s.p_last = a.shared + job.s.len - 1;
    if (threadIdx.x < S::kRows)
      sm.pos[threadIdx.x] = static_cast<int>(threadIdx.x) < s.rows
                                ? s.p_first + kv_token(a, r0 + threadIdx.x)
                                : -1;
    // the parts that the sequence does not have
    if (part == 0 && threadIdx.x < s.rows)
      for (int p = a.prefix_parts + parts; p < a.parts; ++p)
        *kv_part_w(a, s.hk, p, s.n0 + threadIdx.x) = -INFINITY;
    __syncthreads();
  }
  const int begin = static_cast<int>(static_cast<long long>(s.pages.count) * part / parts);
  const int end = static_cast<int>(static_cast<long long>(s.pages.count) * (part + 1) / parts);
  if (begin == end)
    s.write_weights(true);
  else
    s.run(begin, end);
}

// beside: the launch before this one is the prefix's on the tensor cores, which
// neither writes what this one reads nor reads what it writes, and whose
// dependents begin when all that came before it is done.  So what came before is seen
// through a.ready, and one CTA of this launch waits for the prefix's, at its end (and
// the launch is complete only when both are).  (With all of them waiting, those that
// find no job begin when the prefix has left its SMs, and the join 2 us later.)
template <int D, int NT>
__global__ void __launch_bounds__(kSThreads, span_ctas(NT))
    kv8_span_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ Kv8Args a,
                    int prefix_groups, SpanSlots slots, int max_rows, int beside) {
  if (beside) {
    grid_ready_or_wait(a.ready);
  } else {
    grid_dependency_wait();
    if (blockIdx.x == 0 && threadIdx.x == kSThreads - 1) grid_ready(a.ready);
  }
  grid_dependents_launch();
  span_part<D, NT>(tm, a, prefix_groups, slots, max_rows);
  if (beside && blockIdx.x == 0) grid_dependency_wait();
}

// The join.  A CTA takes kJoinRows (4, or 8 of many) rows of a key-value head: a warp makes the
// weights of a row, then each thread adds four elements of one over every kG-th
// part, the first of them loaded under the weights, and the kG sums are added in
// their order.  It is a chain of a few dependent reads from L2: with all parts of
// eight rows' elements in a thread's hands, batch after batch, it took 5 us more (32
// sequences behind 16384 tokens, with 12 parts of their own).
constexpr int kJoinThreads = 256;
template <int D, int kJoinRows>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const __grid_constant__ Kv8Args a) {
  constexpr int kR = kJoinRows, kC = D / 4, kG = kJoinThreads / (kR * kC);
  extern __shared__ float weight[];  // [kR][parts]
  __shared__ bool s_row[kR];  // the row is one of a sequence that is not skipped
  __shared__ float4 sums[kG > 1 ? kG - 1 : 1][kR * kC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  const int n0 = blockIdx.x * kR;  // first row of the head
  const int R = a.rows * a.group;
  auto row_of = [&](int n) {
    const int tok = kv_token(a, n);
    return static_cast<long long>(tok) * a.heads + hk * a.group + (n - tok * a.group);
  };
  // (the call's inputs, before the parts)
  grid_ready_or_wait(a.ready);
  if (threadIdx.x < kR) s_row[threadIdx.x] = false;
  __syncthreads();
  const int last = n0 + kR < R ? n0 + kR : R;
  const int tok0 = kv_token(a, n0), tok1 = kv_token(a, last - 1);
  for (int b = threadIdx.x; b < a.seqs; b += kJoinThreads) {
    const KvSeq s = kv_seq(a, b);
    if (!s.ok || s.row0 > tok1 || s.row0 + s.m <= tok0) continue;
    for (int n = n0; n < last; ++n) {
      const int tok = kv_token(a, n);
      if (tok >= s.row0 && tok < s.row0 + s.m) s_row[n - n0] = true;
    }
  }
  __syncthreads();
  grid_dependency_wait();
  // (who finds it lowered waits instead)
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) st_release_gpu(a.ready, 0);
  grid_dependents_launch();
  const int c = threadIdx.x % kC, i = threadIdx.x / kC % kR, g = threadIdx.x / (kR * kC);
  const bool mine = n0 + i < R && s_row[i];
  const float4* from = kv_part_o(a, hk, 0, c, n0 + i);
  const size_t step = static_cast<size_t>(R) * kC;
  constexpr int kAtOnce = 8;
  float4 v[kAtOnce];
  // a row's weights, a warp each: loaded ahead of the parts, which would hold them
  // up
  const float* ws = kv_part_w(a, hk, 0, n0 + warp);
  const bool weigh = warp < kR && s_row[warp < kR ? warp : 0];
  float first = -INFINITY;
  if (weigh && lane < a.parts) first = __ldcg(ws + static_cast<size_t>(lane) * R);
  // (a part of no weight may never have been written: what it holds is not used)
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k)
    if (mine && g + k * kG < a.parts) v[k] = __ldcg(from + (g + k * kG) * step);
  static_assert(kR <= kJoinThreads / 32, "a warp a row");
  if (weigh) {
    float* w = weight + warp * a.parts;
    float top = first;
    if (lane < a.parts) w[lane] = first;
    for (int p = lane + 32; p < a.parts; p += 32) {
      const float x = __ldcg(ws + static_cast<size_t>(p) * R);
      w[p] = x;
      top = fmaxf(top, x);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    for (int p = lane; p < a.parts; p += 32) {
      w[p] = exp2f(w[p] - base);
      l += w[p];
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    const float one = l == 0.f ? 0.f : 1.0f / l;
    for (int p = lane; p < a.parts; p += 32) w[p] *= one;
    if (a.lse && lane == 0) a.lse[row_of(n0 + warp)] = kv_log_sum(base, l, kROff);
  }
  __syncthreads();
  const float* w = weight + i * a.parts;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine) {
#pragma unroll 1
    for (int p0 = g;;) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float f = p0 + k * kG < a.parts ? w[p0 + k * kG] : 0.f;
        if (f == 0.f) continue;
        acc.x = fmaf(f, v[k].x, acc.x);
        acc.y = fmaf(f, v[k].y, acc.y);
        acc.z = fmaf(f, v[k].z, acc.z);
        acc.w = fmaf(f, v[k].w, acc.w);
      }
      p0 += kAtOnce * kG;
      if (p0 >= a.parts) break;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (p0 + k * kG < a.parts && w[p0 + k * kG] != 0.f)
          v[k] = __ldcg(from + (p0 + k * kG) * step);
    }
  }
  if (g > 0) sums[g - 1][threadIdx.x % (kR * kC)] = acc;
  __syncthreads();
  if (g > 0 || !mine) return;
#pragma unroll
  for (int k = 0; k < kG - 1; ++k) {
    const float4 x = sums[k][threadIdx.x];
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row_of(n0 + i) * D + 4 * c) =
      make_uint2(pack_out(a.type, acc.x, acc.y), pack_out(a.type, acc.z, acc.w));
}

// Rows (of all key-value heads) times parts that the workspace holds beside one
// part of each: a prefix's blocks of 256 rows on the tensor cores are cut while there
// are fewer than two for each SM.
constexpr long long kPrefixPartRows = 2ll * kSmallTMaxCtas * 256;
constexpr long long kSpanPartRows = 40960;
// Parts of a row that spans cut the prefix, or its own tokens, into at most.
// (The join's weights are in shared memory.)
constexpr long long kSpanParts = 128;
long long clamp_parts(long long parts, long long most, long long rows) {
  if (parts > most) parts = most;
  if (parts > kSpanParts) parts = kSpanParts;
  if (parts * rows > kSpanPartRows) parts = kSpanPartRows / rows;
  return parts < 1 ? 1 : parts;
}

// How the SMs are shared between the prefix's blocks on the tensor cores and the
// spans of the own tokens.  Both are chains of dependent reads before anything else,
// so a prefix's CTAs on some of the SMs, with the spans beside them on the others,
// often end before the two one after the other on all.  Times in us, measured: a
// part of the prefix 7 and 0.95 a page of two tiles of rows (0.62 of one in its split
// form; heads of 64 two thirds), a span 6.5 and 0.77 a page of one tile of eight rows,
// a quarter more for each further tile, 5 between two launches that follow each other.
// The launch knows the table's width, not the sequences' lengths: they are taken to be
// half of it and at most 24 pages.  The best split and all SMs for both: 32 sequences
// of 40 to 1500 tokens behind 16384 36.5 (88 SMs and 64) and 43.6; 16 of up to 300
// behind 4096 15.6 and 20.9; 40 of 20 rows, up to 900 tokens, behind 32768 133 (128
// SMs, and 24 that take all spans in turn) and 145.
struct Plan {
  int parts;  // of the prefix
  SpanSlots slots;
};
Plan plan_prefix(const Kv8Args& a, int pages, int own_pages, int tiles, long long ctas, int sms) {
  const int R = a.rows * a.group, on = span_ctas(tiles);
  const long long items = (R + 255ll) / 256 * a.hkv;
  const double narrow = a.dim == 64 ? 0.65 : 1.0;
  const double page = (R <= 64 ? 0.62 : 0.95) * narrow, own_page = 0.77 * narrow * (tiles + 3) / 4;
  const int average = own_pages < 48 ? (own_pages + 1) / 2 : 24;
  const int longest = own_pages < 48 ? own_pages : 48;
  auto prefix = [&](long long parts) {
    return static_cast<double>((items * parts + sms - 1) / sms) * (7 + page * ((pages + parts - 1) / parts));
  };
  auto own = [&](int slots) {
    if (ctas > slots) {
      const double waves = ctas > 2ll * slots ? static_cast<double>(ctas) / slots : 2;
      return waves * (6.5 + own_page * average) + own_page * (longest - average);
    }
    const double room = slots - ctas > slots / 4 ? slots - ctas : slots / 4;
    const double quota = ctas * average / room;
    return 6.5 + own_page * (quota < longest ? quota : longest);
  };
  const int all = sms * on;
  Plan best = {kv8_prefix_parts(a, pages, sms), {all, all, 1 << 30}};
  double least = prefix(best.parts) + 5 + own(all);
  for (long long p = 1; p * 2 <= pages && items * p <= sms - sms / 8; ++p) {
    const int free = static_cast<int>(sms - items * p) * on;
    const double t1 = prefix(p), t2 = own(free), t = t1 > t2 ? t1 : t2;
    if (t < least) {
      least = t;
      const int fit = static_cast<int>(1.5 * (t - 6.5) / own_page);
      best = {static_cast<int>(p), {free, all, fit < longest ? longest : fit}};
    }
  }
  return best;
}

// Pages that a sequence's rows see at most, of the prefix and of their own.
struct SeenPages {
  int prefix, own;
};
SeenPages seen_pages(const Kv8Args& a, int shared) {
  SeenPages s = {shared / kBlk, a.width - shared / kBlk};
  if (a.window > 0) {
    const long long seen = static_cast<long long>(a.window) / kBlk + 2;
    const long long sinks = a.sinks / kBlk + 1;
    if (seen + sinks < s.prefix) s.prefix = static_cast<int>(seen + sinks);
    if (seen + a.max_new / kBlk + sinks < s.own)
      s.own = static_cast<int>(seen + a.max_new / kBlk + sinks);
  }
  return s;
}

// Tiles of eight rows of a span: those of a sequence, where three hold them, or two
// at a time.  24 rows in one span of three tiles, or in two of two, whose registers
// and rings let an SM hold three CTAs instead of two: 8 sequences of up to 2000
// tokens behind 8192 29.9 and 37.1 us, 32 of up to 4000 behind 2048 100 and 110, 16
// of up to 1500 behind 4096 42.0 and 40.9.  36 rows in two of three tiles 29.8, in
// three of two 26.7 (8 sequences of up to 300 behind 4096).
int span_tiles(long long most) { return most <= 8 ? 1 : most > 16 && most <= 24 ? 3 : 2; }

// Shared memory of a span's CTA (whose layout starts on 1024 bytes).
int span_bytes(int dim, int tiles) {
  const size_t n =
      tiles == 1   ? (dim == 128 ? sizeof(Span<128, 1>::Smem) : sizeof(Span<64, 1>::Smem))
      : tiles == 2 ? (dim == 128 ? sizeof(Span<128, 2>::Smem) : sizeof(Span<64, 2>::Smem))
                   : (dim == 128 ? sizeof(Span<128, 3>::Smem) : sizeof(Span<64, 3>::Smem));
  return static_cast<int>(n) + 1024;
}

}  // namespace

cudaError_t kv8_shared_set_attributes() {
  const auto allow = [](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = allow(kv8_span_kernel<64, 1>, span_bytes(64, 1));
  if (e == cudaSuccess) e = allow(kv8_span_kernel<64, 2>, span_bytes(64, 2));
  if (e == cudaSuccess) e = allow(kv8_span_kernel<128, 1>, span_bytes(128, 1));
  if (e == cudaSuccess) e = allow(kv8_span_kernel<128, 2>, span_bytes(128, 2));
  if (e == cudaSuccess) e = allow(kv8_span_kernel<64, 3>, span_bytes(64, 3));
  if (e == cudaSuccess) e = allow(kv8_span_kernel<128, 3>, span_bytes(128, 3));
  return e;
}

bool kv8_shared_fits(int rows, int group, int kv_heads, int seqs) {
  // (the spans' grid has up to kSpanRows / 8 CTAs a sequence and head)
  return kv8_prompt_fits(rows, group, kv_heads, 1) &&
         static_cast<long long>(seqs) * kv_heads <= (0x7FFFFFFFll - 4 * kSmallTMaxCtas) / (kSpanRows / 8) / 2;
}

// What sharing wins is a pass over the prefix a sequence.  What it loses:
//
// The own tokens' pages in spans take longer than in the ordinary kernels, the more
// so the more rows a span or its groups have.  The launch knows the table's width, not
// the lengths, which may be anything up to it: it shares up to about the width at which
// short sequences would lose by the ordinary kernels what full ones win.  Measured, the
// time of each for itself over that of sharing, for 8 and 32 sequences (8 key-value
// heads of 128) of up to 1000 own tokens, then of up to 17000 (up to 20 rows) or 4000:
//   rows    behind 64               512                      4096 shared tokens
//     6   1.4  1.2   0.96 0.74   1.3  1.4   0.96 0.91   1.3  2.0   0.70 0.95
//    12   1.5  1.1   0.88 0.44   1.3  1.3   0.88 0.78   1.3  1.9   0.86 1.02
//    20   1.3  0.89  0.79 0.59   1.4  1.3   0.81 0.59   1.6  1.7   0.90 0.67
//    30   1.05 0.83  0.85 0.84   1.1  0.90  0.90 0.86   1.4  1.7   1.2  1.25
//    60   0.77 0.56  0.58 0.50   0.86 0.63  0.55 0.53   0.99 1.2   0.67 0.80
// (What the width does not tell: short sequences in a wide table lose by the ordinary
// kernels, 128 of up to 300 tokens with 20 rows behind 512 75 and 101 us; a long one
// among many short ones loses in spans, see OwnJobs.)
//
// Every span's CTA looks through all sequences for its own: 24 rows, up to 300 tokens,
// behind 64 shared ones 1.18 times as fast at 256 sequences, 1.03 at 512, 0.76 at 1024;
// behind 512 1.25, 1.08, 0.81; behind 4096 1.2 at 2048.  6 rows behind 64 1.43 at 512,
// 1.02 at 1024, 0.62 at 2048; behind 512 1.10 and 0.68 at 1024 and 2048.
//
// Chunks of more than kSpanRows rows go through the tensor cores either way, and what
// sharing loses is the parts' way through the workspace and launches that follow each
// other.  Each for itself over shared: 3600 rows 0.38 to 0.9 (2 to 16 sequences behind
// 512 to 16384); 72, 128 and 258 rows, up to 2000 own tokens, behind 512 0.5 to 0.8,
// behind 4096 0.6 to 1.05 at up to 16 sequences.  Longer prefixes of more sequences would
// gain, which the rule leaves: 32 sequences of 72 rows behind 16384 2.3 (454 and 200 us),
// of 258 rows 1.4; 4 of 72 rows 1.04.
//
// In a mixed batch the shorter sequences win a pass over the prefix each (2 bytes an
// element, and there are seqs - R / most of them at least) and all rows lose their parts
// (some 12), with the losses above, sooner, since the spans are of 16 rows.  A chunk of 12
// to 600 tokens among single ones of up to 300 own tokens, behind 64 shared ones 1.0 to
// 1.17 at 128 sequences, 0.88 at 256; behind 512 0.98 to 1.23, then 0.94 to 0.98, 0.71 to
// 0.82 at 512; behind 4096 1.1 at 1024, 0.63 to 0.71 at 2048.  32 sequences of up to 17000,
// with a chunk of 12 or without any (max_new left out), behind 64 0.91 and 0.78, behind 512
// 0.93 and 0.79, of up to 4000 1.02 and 0.97; behind 4096 1.1 and 1.0 (with a chunk of 600
// tokens 0.71, and 1.24 of up to 300).
bool kv8_shared_pays(const Kv8Args& a, int shared) {
  if (a.seqs == 1 || shared == 0) return false;
  const long long R = static_cast<long long>(a.rows) * a.group;
  const long long most = static_cast<long long>(a.max_new) * a.group;
  const SeenPages seen = seen_pages(a, shared);
  const long long prefix = seen.prefix;
  if (most <= kSpanRows) {
    if (a.seqs > (most <= 8 ? 640 : 384) + 64 * prefix) return false;
    const long long groups = (most + 15) / 16;  // beyond 24 rows
    return most <= 8 || seen.own <= (most <= 16   ? 64 * (prefix + 1)
                                     : most <= 24 ? 8 * (prefix + 8)
                                                  : (8 * prefix) >> groups);
  }
  const long long limit = 16 * (prefix + 7);  // of sequences, and of own pages
  const long long shorter = a.seqs - (R + most - 1) / most;
  return a.seqs <= limit && seen.own <= limit && shorter * shared > 6 * R;
}

size_t kv8_shared_part_bytes(int rows, int heads, int dim) {
  const long long all = static_cast<long long>(rows) * heads;  // of all key-value heads
  const long long prefix = all > kPrefixPartRows ? all : kPrefixPartRows;
  const long long own = all > kSpanPartRows ? all : kSpanPartRows;
  return static_cast<size_t>(prefix + own) * (dim + 1) * sizeof(float);
}

cudaError_t launch_kv8_shared(const CUtensorMap* tm, Kv8Args a, float* partials, int* tickets, int num_sms,
                              cudaStream_t stream, int* launches) {
  const int R = a.rows * a.group;
  const long long all = static_cast<long long>(R) * a.hkv;
  const long long most = static_cast<long long>(a.max_new) * a.group;
  const int common = a.shared / kBlk;
  const SeenPages seen = seen_pages(a, a.shared);
  const int pages = seen.prefix, own_pages = seen.own;
  const int tiles = span_tiles(most);
  const int tile_rows = 8 * tiles;
  const int groups =
      static_cast<int>(((most < kSpanRows ? most : kSpanRows) + tile_rows - 1) / tile_rows);
  const long long ctas = static_cast<long long>(a.seqs) * a.hkv * groups;
  const int sms = num_sms < kSmallTMaxCtas ? num_sms : kSmallTMaxCtas;
  const int all_slots = sms * span_ctas(tiles);
  SpanSlots slots = {all_slots, all_slots, 1 << 30};
  // The prefix is spans too while its pages, times heads and groups of rows, are few:
  // each group reads them again.
  const long long all_groups = (R + tile_rows - 1) / tile_rows;
  const long long units = pages * all_groups * a.hkv;
  const bool prefix_spans = units * (tiles == 3 ? 2 : 1) <= kSpanPrefixUnits &&
                            all_groups * a.hkv + ctas <= all_slots;
  const int prefix_groups = prefix_spans ? static_cast<int>(all_groups) : 0;
  if (prefix_spans) {
    // its share of the CTAs that are resident at once, were the sequences half as long
    // as the table has room for
    const long long own_units = ctas * ((own_pages + 1) / 2);
    long long share = all_slots * units / (units + own_units);
    if (share > all_slots * 3 / 4) share = all_slots * 3 / 4;
    a.prefix_parts = static_cast<int>(
        clamp_parts(share / (a.hkv * all_groups), (pages + kSpanPages - 1) / kSpanPages, all));
    slots.free = slots.all =
        all_slots - static_cast<int>(a.prefix_parts * all_groups * a.hkv);
  } else {
    const Plan plan = plan_prefix(a, pages, own_pages, tiles, ctas, sms);
    a.prefix_parts = plan.parts;
    slots = plan.slots;
  }
  const int own_parts = static_cast<int>(
      clamp_parts(slots.all, (own_pages + kSpanPages - 1) / kSpanPages, all));
  a.parts = a.prefix_parts + own_parts;
  a.part_w = a.part_o + static_cast<size_t>(a.parts) * all * a.dim;

  cudaError_t e;
  if (!prefix_spans) {
    e = launch_kv8_prompt(a, kKvPrefix, 1, nullptr, nullptr, num_sms, stream, launches);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  // (own tokens: see OwnJobs; what is left over finds no job)
  // (room for the quota's rounding in fp32: 2^-24 for each 32 sequences)
  long long jobs = ctas + slots.all / 4 > slots.all ? ctas + slots.all / 4 : slots.all;
  jobs += jobs / 16 + 8;
  if (jobs > ctas * own_parts) jobs = ctas * own_parts;
  const long long grid = static_cast<long long>(prefix_groups) * a.hkv * a.prefix_parts + jobs;
  cudaLaunchConfig_t cfg = pdl_launch_config(attr, dim3(static_cast<unsigned>(grid)),
                                             dim3(kSThreads), span_bytes(a.dim, tiles), stream);
  const auto span = tiles == 1   ? (a.dim == 128 ? kv8_span_kernel<128, 1> : kv8_span_kernel<64, 1>)
                    : tiles == 2 ? (a.dim == 128 ? kv8_span_kernel<128, 2> : kv8_span_kernel<64, 2>)
                                 : (a.dim == 128 ? kv8_span_kernel<128, 3> : kv8_span_kernel<64, 3>);
  e = cudaLaunchKernelEx(&cfg, span, *tm, a, prefix_groups, slots, kSpanRows, prefix_spans ? 0 : 1);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (most > kSpanRows) {
    // (positions, pages and lengths from the prefix's end)
    Kv8Args own = a;
    own.table += common;
    own.sinks = a.sinks > a.shared ? a.sinks - a.shared : 0;
    e = launch_kv8_prompt(own, kKvOwn, kSpanRows + 1, partials, tickets, num_sms, stream, launches);
    if (e != cudaSuccess) return e;
  }
  // Four rows a CTA make twice as many threads of as many parts: for few rows.  With
  // 4 and 8: 288 rows (times key-value heads) 12.7 and 13.6 us a call, 1536 18.3 and
  // 19.4, 12288 70.4 and 63.5.
  const int join_rows = all < 16ll * num_sms ? 4 : 8;
  static_assert((2 * kSmallTMaxCtas + 2 * kSpanParts) * 8 * sizeof(float) <= 32 << 10,
                "the join's shared memory");
  cfg = pdl_launch_config(attr, dim3((R - 1) / join_rows + 1, a.hkv), dim3(kJoinThreads),
                          sizeof(float) * join_rows * a.parts, stream);
  e = cudaLaunchKernelEx(
      &cfg,
      join_rows == 4 ? (a.dim == 128 ? kv8_join_kernel<128, 4> : kv8_join_kernel<64, 4>)
                     : (a.dim == 128 ? kv8_join_kernel<128, 8> : kv8_join_kernel<64, 8>),
      a);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace tern
