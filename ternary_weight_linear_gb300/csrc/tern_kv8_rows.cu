// tern_kv8_attention for sequences with few query rows per key-value head
// (decode steps): bound by the bytes of the cache.
//
// The rows of a sequence that share a key-value head (new tokens x heads of
// the group, up to 24) are one to three tiles of eight, so every cache byte is
// read once for all of them.  Per half-page of 32 tokens a warp computes, with
// m16n8k16 fp16 tensor instructions and fp32 sums, transposed so that tokens
// (and then the elements of the output) are the operand of 16 rows and the
// queries the one of eight:
//   S^T = Kc Q^T,  s = S * (softmax_scale * log2(e) * k_scale * 2^-a(row))
//   w = 2^(s + log2(v_scale) - ref + 10),  O^T += Vc^T w,  l += w / v_scale
// with Q scaled by 2^a per row into fp16, Kc and Vc the int8 codes (exact in
// fp16).  w is rounded to fp16 (relative 2^-11, the tensor instruction's operand;
// the row's sum takes it unrounded).  ref is the running maximum of s +
// log2(v_scale) over what the row sees in the warp, raised (and O rescaled) only
// when a score passes it by 2^4: w stays below 2^15 (fp16 ends at 65504), and the
// lanes' maxima are joined only then.  What w loses, below 2^-24, is small beside
// the row's own largest weight times value scale, whatever other rows see.
//
// Why these instructions: the work is 2 MFLOP per 16 KB page and eight rows,
// and operands that come straight from registers never write the codes back:
// three integer instructions per four codes make them fp16.  One tile of rows
// takes them as subnormals, (code + 128) 2^-24, a byte beside a zero byte,
// which saves the subtraction: the bias leaves the scores through the
// accumulators' start and each half-page's output through a product of all
// -128.  (The tcgen05 kernel for more rows writes each page back as fp16 and
// reads its 128 query rows again for every page: four times the shared-memory
// traffic, and a longer chain per page: 630 us where this one takes 181.)
// With tokens as the operand of eight rows (queries padded to 16) the same
// step took 838 instructions instead of 530, and 219 us instead of 196.
//
// Work: all (sequence, head, page) units of the launch in one line, cut into
// ranges, one persistent CTA of eight warps per SM.  Each warp takes every
// eighth half-page of its CTA's range through its own ring of TMA boxes (32
// tokens of keys and of values a stage), so no barrier between warps stands in
// the loop; at a segment's end the warps' (ref, sum, O) are merged through
// shared memory.  Segments cut by a range's end go to the workspace, and the
// last CTA to finish one adds its parts in their order.
//
// Measured: 32 decode sequences of 544000 cached tokens, 8 key-value heads of
// 128, 48 query heads: 181 us, 6.15 TB/s (0.90 of the copy rate; the loads
// alone take 167).  One token over 32000: 21.7 us; over 777: 9.5 us, of which
// the launch, four dependent reads of indexes, pages and scales, the merge and
// the join are all but one.  (A block of the 32 sequences each left to far_row:
// 528 us.)
#include "tern_kv8_half.cuh"

namespace tern {
namespace {

constexpr int kRW = 8;        // warps
constexpr int kMergeRows = 4; // rows merged at a time
constexpr int kRecs = 256;    // pages whose records are held at a time
// From this many pages per CTA an eighth of the units is left for short ranges.
// A static split ends when the SM with the least share of the HBM rate does,
// up to 19 % after the mean; a short range costs its CTA 3 us of records,
// merge and join.  Measured, with them and without: 181 and 197 us (447 pages
// a CTA), 121 and 107 us (237 pages a CTA, 12 rows).
constexpr int kQueueUnits = 384;
constexpr int kQueue = 511;                // the ticket that counts the short ranges taken
// D: elements of a head.  NT: tiles of eight rows.
template <int D, int NT>
struct RL {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStage = 2 * kHalf * D;  // bytes: keys, then values
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRing = kRW * kStages * kStage;  // 1024-aligned stages
  static constexpr int kQStride = 2 * D + 16;           // bytes of a staged query row
  static constexpr int kQOff = kRing;
  static constexpr int kMergeOff = kQOff + kRows * kQStride;  // [kRW][kMergeRows][D] fp32
  static constexpr int kMlOff = kMergeOff + kRW * kMergeRows * D * 4;  // [kRW][kRows] (ref, sum)
  static constexpr int kFacOff = kMlOff + kRW * kRows * 8;    // [kRows][kRW] factors
  static constexpr int kTotOff = kFacOff + kRW * kRows * 4;   // [kRows] (ref, sum)
  static constexpr int kQScaleOff = kTotOff + kRows * 8;      // [kRows] 2^-a
  static constexpr int kRecOff = kQScaleOff + kRows * 4;  // [kRecs] PageRec, then rows
  static constexpr int kSeqOff = kRecOff + kRecs * 20;        // before[n + 1], len, m, row0
  static constexpr int kBarOff = kSeqOff + (kKvSeqsPerLaunch + 1) * 8 + kKvSeqsPerLaunch * 12;
  static constexpr int kBytes = kBarOff + kRW * kStages * 8;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kQOff % 16 == 0 && kMergeOff % 16 == 0 && kRecOff % 16 == 0 && kSeqOff % 8 == 0 &&
                    kBarOff % 8 == 0,
                "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// A warp's ring of half-pages and where they come from.
template <int D>
struct HalfRing {
  uint8_t* ring;
  uint64_t* full;
  const int* where;
  const CUtensorMap* tm;
  int hkv;
  // (whole warp) requests half-pages of the records, pre to end, until the ring
  // is full
  __device__ __forceinline__ void issue(int end, int& pre, unsigned& issued, unsigned used,
                                        int lane) const {
    constexpr int kStages = RL<D, 1>::kStages, kStage = RL<D, 1>::kStage;
    while (pre < end && issued - used < kStages) {
      const int rec = where[pre >> 1];
      const int half = pre & 1;
      if (rec >= 0 && (rec & (kMHalf << half))) {
        if (lane == 0) {
          const int s = issued % kStages;
          const int row = (rec & ~(kBlk - 1)) + half * kHalf;
          mbar_arrive_expect_tx(&full[s], kStage);
          tma_load_2d(ring + s * kStage, tm, 0, row, &full[s]);
          tma_load_2d(ring + s * kStage + kHalf * D, tm, 0, row + hkv * kBlk, &full[s]);
        }
        ++issued;
      }
      pre += kRW;
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kRW * 32, 1)
    kv8_rows_kernel(const __grid_constant__ CUtensorMap tm, const Kv8Args a, int max_rows,
                    int per_head) {
  using L = RL<D, NT>;
  constexpr int kRows = L::kRows;
  constexpr int kW = D / 16;   // words of a lane per key row: 8 or 4 (k steps)
  constexpr int kMT = D / 16;  // tiles of 16 elements of the output
  constexpr int kVW = D / 32;  // words of a lane per value row: 4 or 2
  constexpr bool kBiased = biased(NT);
  // (three tiles read their queries from shared memory at each half-page)
  constexpr bool kQRegs = NT < 3;
  constexpr float kUp = kBiased ? kCodeUp : 1.f;  // 1 over the codes' unit
  grid_dependents_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_addr(smem_raw) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff) + warp * L::kStages;
  uint8_t* ring = smem + warp * (L::kStages * L::kStage);
  float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  float* fac = reinterpret_cast<float*>(smem + L::kFacOff);
  float2* tot = reinterpret_cast<float2*>(smem + L::kTotOff);
  float* qscale = reinterpret_cast<float*>(smem + L::kQScaleOff);
  PageRec* recs = reinterpret_cast<PageRec*>(smem + L::kRecOff);
  int* where = reinterpret_cast<int*>(recs + kRecs);
  long long* before = reinterpret_cast<long long*>(smem + L::kSeqOff);  // units before a sequence
  int* seq_len = reinterpret_cast<int*>(before + kKvSeqsPerLaunch + 1);
  int* seq_m = seq_len + kKvSeqsPerLaunch;
  int* seq_row0 = seq_m + kKvSeqsPerLaunch;
  __shared__ int s_last, s_next;
  __shared__ int s_far;  // the CTA has met pages that are left to far_row

  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    prefetch_tensormap(&tm);
  }
  grid_dependency_wait();  // every input, the output and the workspace belong to earlier work

  // ---- the launch's units: (sequence, head, page), pages fastest
  for (int b = threadIdx.x; b < a.seqs; b += kRW * 32) {
    const KvSeq s = kv_seq(a, b);
    if (!s.ok && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
    long long u = 0;
    if (s.ok && s.m > 0 && s.m * a.group <= max_rows)
      u = static_cast<long long>(kv_pages(a, s.len - s.m, s.len - 1).count) * a.hkv;
    before[b + 1] = u;
    seq_len[b] = s.len;
    seq_m[b] = s.m;
    seq_row0[b] = s.row0;
  }
  if (threadIdx.x == 0) {
    before[0] = 0;
    s_far = 0;
  }
  __syncthreads();
  if (a.seqs > 1) {
    if (warp == 0) {
      // running sums of 32 sequences at a time
      long long carry = 0;
      for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        const int b = b0 + lane;
        long long v = b < a.seqs ? before[b + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += up;
        }
        if (b < a.seqs) before[b + 1] = carry + v;
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
  }
  const long long U = before[a.seqs];
  // Ranges of units: one for each CTA, of [0, fixed), and where there is enough
  // work the rest in short ones that CTAs take as they finish.  A single
  // sequence's heads are cut one by one, into equal numbers of ranges: no CTA
  // then has the end of one head and the start of the next to merge (one token
  // over 32000: 21.7 us instead of 25.8; two over 4000: 12.5 instead of 21.6).
  if (U == 0) return;
  const unsigned ctas = gridDim.x;
  const bool queue = U >= static_cast<long long>(kQueueUnits) * ctas;
  const bool heads = !queue && per_head > 0;  // one sequence, head by head
  // (without short ranges every number here has 32 bits)
  unsigned run = 0, per = 0, cuts = 0;  // units of a head, of a range; ranges of a head
  long long fixed = U, per2 = 1, per1 = 1;
  int extra = 0;  // short ranges
  int range = static_cast<int>(blockIdx.x);
  long long u_begin, u_end;
  if (queue) {
    per1 = U / ctas * 7 / 8;
    fixed = per1 * ctas;
    per2 = (U - fixed + ctas - 1) / ctas;
    extra = static_cast<int>((U - fixed + per2 - 1) / per2);
    u_begin = range * per1;
    u_end = u_begin + per1;
  } else if (heads) {
    run = static_cast<unsigned>(kv_pages(a, seq_len[0] - seq_m[0], seq_len[0] - 1).count);
    per = (run + per_head - 1) / per_head;
    cuts = (run + per - 1) / per;
    const unsigned head = blockIdx.x / cuts, at = (blockIdx.x - head * cuts) * per;
    u_begin = head * run + at;
    u_end = head * run + (run < at + per ? run : at + per);
  } else {
    per = (static_cast<unsigned>(U) + ctas - 1) / ctas;
    u_begin = static_cast<long long>(blockIdx.x) * per;
    u_end = U < u_begin + per ? U : u_begin + per;
  }
  if (u_begin >= U) return;
  auto range_of = [&](long long u) {
    if (queue) return static_cast<int>(u < fixed ? u / per1 : ctas + (u - fixed) / per2);
    const unsigned v = static_cast<unsigned>(u);
    if (!heads) return static_cast<int>(v / per);
    const unsigned head = v / run;
    return static_cast<int>(head * cuts + (v - head * run) / per);
  };

  // the sequence of unit u
  auto seq_of = [&](long long u) {
    int lo = 0, hi = a.seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (before[mid + 1] > u) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  // unit u within its sequence's units: (head, page of the list)
  auto split = [](long long in, int np, int& head, int& page) {
    const unsigned v = static_cast<unsigned>(in);  // (heads * pages of a sequence: 32 bits)
    head = static_cast<int>(v / static_cast<unsigned>(np));
    page = static_cast<int>(v - static_cast<unsigned>(head) * np);
  };

  // ---- state of the current segment (one sequence and head)
  // (lane 4 g + t: rows 8 n + 2 t + x of tile n; sum: of the lane's tokens)
  uint2 qf[NT][kQRegs ? kW : 1];  // the query fragments
  auto query = [&](int n, int j) { return staged_query<D>(smem + L::kQOff, n, j, g, t); };
  float o[NT][kMT][4];
  float ref[NT][2], sum[NT][2], cs[NT][2];
  int pos[NT][2];  // the rows' positions; -1: no row
  float s0[NT][4];  // -128 * 2^-24 times the sums of the rows' queries

  unsigned issued = 0, used = 0;  // stages of this warp so far
  bool ok = true;
  long long c0 = u_begin, c1 = u_begin;  // units whose records are held
  int pre = 0;                           // next half-page of them that this warp requests

  const HalfRing<D> from{ring, full, where, &tm, a.hkv};
  auto issue_ahead = [&]() {
    from.issue(static_cast<int>(2 * (c1 - c0)), pre, issued, used, lane);
  };

  long long u = u_begin;
  while (u < u_end) {  // (the range changes at its end, below)
    // ---- the segment that starts (or continues) at unit u
    const int b = seq_of(u);
    const int len = seq_len[b], m = seq_m[b];
    const int p_first = len - m;
    const KvPages pages = kv_pages(a, p_first, len - 1);
    const int np = pages.count;
    int hk, page0;
    split(u - before[b], np, hk, page0);
    const long long s_begin = u - page0, s_end = s_begin + np;
    const long long e_here = s_end < u_end ? s_end : u_end;
    const int R = m * a.group;
    auto row_of = [&](int r) {  // row r of the tile in q and out (of one head's stride)
      const int tok = kv_token(a, r);
      return make_int2(seq_row0[b] + tok, hk * a.group + r - tok * a.group);
    };

    // queries: each warp scales a row of each tile by a power of two into fp16
    {
      uint32_t raw[NT][D / 64];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int r = warp + x * kRW;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) raw[x][e] = 0u;
        if (r < R) {
          const int2 at = row_of(r);
          const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                                static_cast<long long>(at.x) * a.ld +
                                static_cast<long long>(at.y) * a.hd + lane * (D / 32);
          if constexpr (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2*>(src);
            raw[x][0] = w.x, raw[x][1] = w.y;
          } else {
            raw[x][0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        const int r = warp + x * kRW;
        uint32_t m2 = 0;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) m2 = __vmaxu2(m2, raw[x][e] & 0x7FFF7FFFu);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, k));
        const int up = q_exponent((m2 & 0xFFFFu) > (m2 >> 16) ? m2 & 0xFFFFu : m2 >> 16, a.type);
        const float f = pow2f(up);
        uint32_t* dst = reinterpret_cast<uint32_t*>(smem + L::kQOff + r * L::kQStride);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          float lo, hi;
          unpack16(raw[x][e], a.type, lo, hi);
          // 8-byte unit w of the row sits at w ^ (w / (units / 2)): no two lanes
          // of a fragment load share a bank
          const int word = lane * (D / 64) + e;
          const int unit = word >> 1;
          dst[((unit ^ (unit / (D / 8))) << 1) | (word & 1)] = half2_bits(lo * f, hi * f);
        }
        if (lane == 0) qscale[r] = pow2f(-up);
      }
    }

    // the rest of the segment in this CTA's range, in pieces whose page
    // records fit
    bool first_piece = true;
    while (u < e_here) {
      if (u >= c1) {
        // records of the next units of the range (all segments)
        c0 = u;
        c1 = u_end < c0 + kRecs ? u_end : c0 + kRecs;
        for (int i = threadIdx.x; i < static_cast<int>(c1 - c0); i += kRW * 32) {
          const long long uu = c0 + i;
          const int bb = seq_of(uu);
          const int ll = seq_len[bb], p0 = ll - seq_m[bb];
          const KvPages pp = kv_pages(a, p0, ll - 1);
          int hh, lp;
          split(uu - before[bb], pp.count, hh, lp);
          lp = pp.page(lp);
          const int page = a.table[static_cast<size_t>(bb) * a.width + lp];
          PageRec rec = {0.f, 0.f, 1.f, 0.f};
          int row = -1;
          if (page < 0 || page >= a.pages) {
            atomicOr(a.err, kErrIndex);
          } else {
            const float* sc = a.scales + static_cast<size_t>(page) * 2 * a.hkv + hh;
            const float ks = sc[0];
            const float vs = sc[a.hkv];
            const bool far = far_scales(ks, vs);
            if (far) s_far = 1;
            rec = page_rec(ks, vs);
            row = (page * 2 * a.hkv + hh) * kBlk;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int j0 = lp * kBlk + hf * kHalf, j1 = j0 + kHalf - 1;
              if (!far && kv_any(a, p0, ll - 1, j0, j1)) row |= kMHalf << hf;
              if (kv_all(a, p0, ll - 1, j0, j1)) row |= kMAll << hf;
            }
          }
          recs[i] = rec;
          where[i] = row;
        }
        __syncthreads();
        pre = warp;
        issue_ahead();
      }
      if (first_piece) {
        __syncthreads();  // queries staged
        first_piece = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int j = 0; kQRegs && j < kW; ++j) qf[n][j] = query(n, j);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = 8 * n + 2 * t + x;
            ref[n][x] = -INFINITY;
            sum[n][x] = 0.f;
            cs[n][x] = qscale[r] * a.scale_log2;
            pos[n][x] = r < R ? p_first + kv_token(a, r) : -1;
          }
#pragma unroll
          for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[n][i][x] = 0.f;
          query_bias<D, kBiased>([&](int j) { return qf[n][j]; }, s0[n]);
        }
      }
      const long long piece = e_here < c1 ? e_here : c1;
      // this warp's half-pages of [u, piece): those congruent to its number
      const int h_end = static_cast<int>(2 * (piece - c0));
      int h = static_cast<int>(2 * (u - c0));
      h += (warp + kRW - h % kRW) % kRW;
      for (; h < h_end && ok; h += kRW) {
        const int rec_row = where[h >> 1];
        const int half = h & 1;
        if (rec_row < 0 || !(rec_row & (kMHalf << half))) continue;
        const PageRec rec = recs[h >> 1];
        const int s = used % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait_clk(&full[s], (used / L::kStages) & 1, a.err));
        if (!ok) break;
        const uint8_t* kb = ring + s * L::kStage;
        const uint8_t* vb = kb + kHalf * D;

        float sc[NT][2][4];
        uint32_t kw[4][kW];
        half_keys<D>(kb, g, t, kw);
        half_scores<D, NT>(kw, s0, sc, [&](int n, int j) {
          if (kQRegs) return qf[n][j];
          return query(n, j);
        });
        if (!(rec_row & (kMAll << half))) {
          const int in = static_cast<int>((h >> 1) + c0 - s_begin);
          half_mask<NT>(a, pos, pages.page(in) * kBlk + half * kHalf, g, sc);
        }

        // the values' codes, on their way under the softmax
        uint32_t vw[2][4][D / 32];
        half_values<D>(vb, g, t, vw);
        half_softmax<D, NT>(rec, cs, sc, ref, sum, o);
        half_products<D, NT>(sc, half2_bits(rec.any, rec.any), vw, o);
        __syncwarp();  // the stage has been read
        ++used;
        issue_ahead();
      }
      u = piece;
      // every warp is done with the records before they are replaced
      if (u >= c1 && u < u_end) __syncthreads();
    }

    // ---- the segment's end in this CTA: merge the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) sum[n][x] += __shfl_xor_sync(0xffffffffu, sum[n][x], k);
        if (g == 0) ml[warp * kRows + 8 * n + 2 * t + x] = make_float2(ref[n][x], sum[n][x]);
      }
    if (u >= u_end && extra > 0 && threadIdx.x == 0) {
      // the next range; every CTA fails once, and the last one clears the count
      s_next = atomicAdd(&a.tickets[kQueue], 1);
      if (s_next == extra + static_cast<int>(ctas) - 1) a.tickets[kQueue] = 0;
    }
    const bool whole = s_begin >= u_begin && s_end <= u_end;
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < kRows * 16; i += kRW * 32) {
      // factor of warp w's O in row r: its weight over the sum, in units of 1
      const int r = i / 16, w = i % 16;
      const float2 v = w < kRW ? ml[w * kRows + r] : make_float2(0.f, 0.f);
      float big = v.y == 0.f ? -INFINITY : v.x;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
      const float base = big == -INFINITY ? 0.f : big;
      const float f = v.y == 0.f ? 0.f : exp2f(v.x - base);
      float l = v.y == 0.f ? 0.f : v.y * f;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      if (w < kRW)
        fac[r * kRW + w] = l == 0.f ? 0.f : f / l;
      if (w == 0) tot[r] = make_float2(big, l);
    }
    // the segment's first range (a whole one has its place to itself)
    const int first = whole ? range : range_of(s_begin);
    auto part_of = [&](int i) {  // the partial results of the segment in that range
      return a.partials + static_cast<size_t>(2 * i + (i == first ? 1 : 0)) * (kRows * (D + 2));
    };
    float* mine = part_of(range);
    const bool far = s_far;
    // element d of a merged row, in chunks of four that eight lanes' stores
    // spread over all banks
    auto spread = [](int group, int chunk) {  // group of D / 8 elements, chunk of it
      constexpr int kChunks = D / 32;
      return group * (D / 8) + 4 * ((chunk + group / (8 / kChunks)) % kChunks);
    };
    // (this and the join below run once or twice per launch: what counts is
    // that there is little code to fetch)
    auto merge_rows = [&](int r0, const float (&on)[kMT][4]) {
      // rows r0 to r0 + 3 of every warp
      if ((t >> 1) == ((r0 >> 2) & 1)) {
        float* dst = merge + (warp * kMergeRows + 2 * (t & 1)) * D;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int q = 0; q < kVW; ++q)
            *reinterpret_cast<float4*>(dst + x * D + spread(g, q)) =
                make_float4(kUp * on[2 * q][x], kUp * on[2 * q][x + 2], kUp * on[2 * q + 1][x],
                            kUp * on[2 * q + 1][x + 2]);
      }
      __syncthreads();
      constexpr int kDT = D / 64;  // elements of a thread
      const int rl = threadIdx.x / 64, r = r0 + rl, d = threadIdx.x % 64 * kDT;
      if (r < R) {
        const float* src = merge + rl * D + spread(d / (D / 8), d / 4 % (D / 32)) + d % 4;
        float acc[kDT];
#pragma unroll
        for (int y = 0; y < kDT; ++y) acc[y] = 0.f;
#pragma unroll
        for (int w = 0; w < kRW; ++w) {
          const float f = fac[r * kRW + w];
#pragma unroll
          for (int y = 0; y < kDT; ++y)
            if (f != 0.f) acc[y] = fmaf(f, src[w * kMergeRows * D + y], acc[y]);
        }
        const float2 v = tot[r];
        if (whole && !far) {
          const int2 at = row_of(r);
          const long long ob = static_cast<long long>(at.x) * a.heads + at.y;
          uint16_t* out = static_cast<uint16_t*>(a.out) + ob * D + d;
          if constexpr (kDT == 2)
            *reinterpret_cast<uint32_t*>(out) = pack_out(a.type, acc[0], acc[1]);
          else
            *out = static_cast<uint16_t>(pack_out(a.type, acc[0], 0.f));
          if (a.lse && d == 0) a.lse[ob] = kv_log_sum(v.x, v.y, kROff);
        } else {
#pragma unroll
          for (int y = 0; y < kDT; ++y) mine[r * D + d + y] = acc[y];
          if (d == 0) reinterpret_cast<float2*>(mine + kRows * D)[r] = v;
        }
      }
      __syncthreads();
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll 1
      for (int r0 = 8 * n; r0 < 8 * n + 8 && r0 < R; r0 += kMergeRows) merge_rows(r0, o[n]);
    if (far) {
      // the pages left out join what has been written beside them
      for (int r = warp; r < R; r += kRW) {
        const FarRow<D> f = far_row<D>(
            a, smem + L::kQOff + r * L::kQStride, qscale[r] * a.scale_log2,
            p_first + kv_token(a, r), b, hk, pages,
            s_begin < u_begin ? static_cast<int>(u_begin - s_begin) : 0,
            static_cast<int>(e_here - s_begin));
        float* to = mine + r * D + lane * (D / 32);
        float2* at = reinterpret_cast<float2*>(mine + kRows * D) + r;
        const float2 v = *at;
        const float top = fmaxf(v.y == 0.f ? -INFINITY : v.x, f.ref);
        const float base = top == -INFINITY ? 0.f : top;
        const float w0 = v.y == 0.f ? 0.f : v.y * exp2f(v.x - base);
        const float w1 = f.sum * exp2f(f.ref - base), l = w0 + w1;
        const float f0 = l == 0.f ? 0.f : w0 / l, f1 = l == 0.f ? 0.f : w1 / l;
        const int2 row = row_of(r);
        const long long ob = static_cast<long long>(row.x) * a.heads + row.y;
        __syncwarp();
#pragma unroll
        for (int y = 0; y < D / 32; ++y) {
          const float x = to[y] * f0 + f.o[y] * f1;
          if (whole)
            static_cast<uint16_t*>(a.out)[ob * D + lane * (D / 32) + y] =
                static_cast<uint16_t>(pack_out(a.type, x, 0.f));
          else
            to[y] = x;
        }
        if (lane == 0) {
          if (!whole)
            *at = make_float2(base, l);
          else if (a.lse)
            a.lse[ob] = kv_log_sum(base, l, kROff);
        }
      }
      __syncthreads();  // the queries have been read
    }
    if (!whole) {
      // the last of the segment's CTAs adds the parts in their order, a row per
      // warp
      const int parts = range_of(s_end - 1) - first + 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        s_last = atomic_add_acq_rel_gpu(&a.tickets[first], 1) == parts - 1;
      __syncthreads();
      if (s_last) {
        if (threadIdx.x == 0) a.tickets[first] = 0;
        constexpr int kV = D / 32;
        for (int r = warp; r < R; r += kRW) {
          float top = -INFINITY, l = 0.f, acc[kV];
#pragma unroll
          for (int y = 0; y < kV; ++y) acc[y] = 0.f;
#pragma unroll 1
          for (int p0 = 0; p0 < parts; p0 += 32) {
            // a part per lane: its weight, 0 if its rows saw nothing
            const int n = parts - p0 < 32 ? parts - p0 : 32;
            float2 ms = make_float2(-INFINITY, 0.f);
            if (lane < n)
              ms = __ldcg(reinterpret_cast<const float2*>(part_of(first + p0 + lane) + kRows * D) +
                          r);
            float now = ms.y == 0.f ? -INFINITY : ms.x;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, k));
            now = fmaxf(now, top);
            const float base = now == -INFINITY ? 0.f : now;
            const float w = ms.y == 0.f ? 0.f : ms.y * exp2f(ms.x - base);
            const float old = exp2f(top - base);
            float all = w;
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) all += __shfl_xor_sync(0xffffffffu, all, k);
            l = l * old + all;
            top = now;
#pragma unroll
            for (int y = 0; y < kV; ++y) acc[y] *= old;
            constexpr int kAtOnce = 16;  // parts whose loads are in flight
#pragma unroll 1
            for (int p1 = 0; p1 < n; p1 += kAtOnce) {
              float v[kAtOnce][kV];
#pragma unroll
              for (int p = 0; p < kAtOnce; ++p) {
                const float* src = part_of(first + p0 + p1 + p) + r * D;
#pragma unroll
                for (int y = 0; y < kV; ++y) v[p][y] = 0.f;
                if (p1 + p < n) {
                  if constexpr (kV == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                    v[p][0] = x.x, v[p][1] = x.y, v[p][2] = x.z, v[p][3] = x.w;
                  } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                    v[p][0] = x.x, v[p][1] = x.y;
                  }
                }
              }
#pragma unroll
              for (int p = 0; p < kAtOnce; ++p) {
                const float f = __shfl_sync(0xffffffffu, w, p1 + p);
#pragma unroll
                for (int y = 0; y < kV; ++y)
                  if (f != 0.f) acc[y] = fmaf(f, v[p][y], acc[y]);
              }
            }
          }
          const int2 at = row_of(r);
          const long long ob = static_cast<long long>(at.x) * a.heads + at.y;
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + ob * D) +
                          lane * (kV / 2);
#pragma unroll
          for (int y = 0; y < kV; y += 2)
            out[y / 2] = pack_out(a.type, acc[y] * inv, acc[y + 1] * inv);
          if (a.lse && lane == 0) a.lse[ob] = kv_log_sum(top, l, kROff);
        }
      }
      __syncthreads();
    }
    if (u >= u_end && extra > 0) {
      const int n = s_next;
      if (n >= extra) break;
      range = static_cast<int>(ctas) + n;
      u_begin = u = c0 = c1 = fixed + n * per2;
      u_end = U < u_begin + per2 ? U : u_begin + per2;
    }
  }
  // no copy of this warp outlives it
  for (; used < issued; ++used)
    if (!mbar_wait_clk(&full[used % L::kStages], (used / L::kStages) & 1, a.err)) break;
}

template <int D, int NT>
cudaError_t launch_one(const CUtensorMap* tm, const Kv8Args& a, int max_rows, int num_sms,
                       cudaStream_t stream, int* launches) {
  cudaLaunchAttribute attr[1];
  for (int b0 = 0; b0 < a.seqs; b0 += kKvSeqsPerLaunch) {
    Kv8Args p = a;
    p.seqs = a.seqs - b0 < kKvSeqsPerLaunch ? a.seqs - b0 : kKvSeqsPerLaunch;
    p.table += static_cast<size_t>(b0) * a.width;
    p.lens += b0;
    p.starts += b0;
    const int grid = num_sms < kSmallTMaxCtas ? num_sms : kSmallTMaxCtas;
    const cudaLaunchConfig_t cfg =
        pdl_launch_config(attr, dim3(grid), dim3(kRW * 32), RL<D, NT>::kAlloc, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_rows_kernel<D, NT>, *tm, p, max_rows,
                                             a.seqs == 1 ? grid / a.hkv : 0);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

size_t kv8_rows_partial_bytes(int dim) {
  // two parts a range: each CTA's, and as many short ones
  static_assert(2 * kSmallTMaxCtas <= kQueue, "tickets");
  return static_cast<size_t>(2 * kSmallTMaxCtas) * 2 * kKvFewRowsLong * (dim + 2) * sizeof(float);
}

cudaError_t kv8_rows_set_attributes() {
  const auto allow = [](auto kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = allow(kv8_rows_kernel<64, 1>, RL<64, 1>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_rows_kernel<64, 2>, RL<64, 2>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_rows_kernel<64, 3>, RL<64, 3>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_rows_kernel<128, 3>, RL<128, 3>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_rows_kernel<128, 1>, RL<128, 1>::kAlloc);
  if (e == cudaSuccess) e = allow(kv8_rows_kernel<128, 2>, RL<128, 2>::kAlloc);
  return e;
}

cudaError_t launch_kv8_rows(const CUtensorMap* tm, const Kv8Args& a, int max_rows, int num_sms,
                            cudaStream_t stream, int* launches) {
  // as many tiles of rows as the largest of the kernel's sequences can have
  const long long most = static_cast<long long>(a.max_new) * a.group;
  const int tiles = static_cast<int>(((most < max_rows ? most : max_rows) + 7) / 8);
  const bool wide = a.dim == 128;
  const auto launch = tiles == 1   ? (wide ? launch_one<128, 1> : launch_one<64, 1>)
                      : tiles == 2 ? (wide ? launch_one<128, 2> : launch_one<64, 2>)
                                   : (wide ? launch_one<128, 3> : launch_one<64, 3>);
  return launch(tm, a, max_rows, num_sms, stream, launches);
}

}  // namespace tern
