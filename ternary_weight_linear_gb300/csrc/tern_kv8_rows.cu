// tern_kv8_attention for sequences with few query rows per key-value head
// (decode and speculative verify): bound by the bytes of the cache.
//
// The rows of a sequence that share a key-value head (new tokens x heads of
// the group) form one tile of 16 or 32 rows, so every cache byte is read once
// for all of them.  Per 64-token page the warp computes, with m16n8k16 fp16
// tensor instructions and fp32 sums,
//   S = Q Kc^T,  s = S * (softmax_scale * log2(e) * k_scale * 2^-a(row))
//   p = 2^(s + log2 f - max + 14),   O += P (2^(e - E) Vc),   l += p / f
// with Q scaled by 2^a per row into fp16, Kc and Vc the int8 codes (exact in
// fp16) and v_scale = 2^e f.  The running maximum and the running exponent E
// rescale O when they grow.
//
// Why these instructions: a page is 16 KB for 16 rows, 8.4 MFLOP at most, an
// eighth of what the SM's HBM share would allow even on the warp-level path,
// whose operands come straight from registers: codes go from shared memory
// to the operand registers with 1.25 (keys) and 1.5 (values) instructions per
// element and are never written back, as an operand in shared memory would
// need.  The contraction order is free, so a lane's operand elements are the
// 32 (16) consecutive bytes it loads: position 2t, 2t+1, 2t+8, 2t+9 of step j
// is element 32t + 4j + 0..3 of the row.
//
// Work: all (sequence, head, page) units of the launch in one line, cut into
// equal ranges, one persistent CTA of eight warps per SM.  Each warp takes
// every eighth half-page of its CTA's range through its own ring of TMA
// boxes (32 tokens of keys and of values a stage), so no barrier between
// warps stands in the loop; at a segment's end the warps' (max, sum, O) are
// merged through shared memory.  Segments cut by a range's end go to the
// workspace, and the last CTA to finish one adds its parts in CTA order.
#include "tern_kv8.cuh"

namespace tern {
namespace {

constexpr int kRW = 8;        // warps
constexpr int kHalf = 32;     // tokens of a stage
constexpr int kRecs = 256;    // pages whose records are held at a time
constexpr float kPOff = 14.f;  // weights are up to 2^14 (times f < 2): fp16's range below
                               // is then 2^-38 of a row's largest weight

template <int D, int MT>
struct RL {
  static constexpr int kRows = 16 * MT;
  static constexpr int kStage = 2 * kHalf * D;  // bytes: keys, then values
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRing = kRW * kStages * kStage;  // 1024-aligned stages
  static constexpr int kQStride = 2 * D + 16;           // bytes of a staged query row
  static constexpr int kQOff = kRing;
  static constexpr int kMergeOff = kQOff + kRows * kQStride;  // [kRW][4][D] fp32
  static constexpr int kMlOff = kMergeOff + kRW * 4 * D * 4;  // [kRW][kRows] (max, sum)
  static constexpr int kQScaleOff = kMlOff + kRW * kRows * 8;  // [kRows] 2^-a
  static constexpr int kExpOff = kQScaleOff + kRows * 4;       // [kRW] E
  static constexpr int kRecOff = kExpOff + kRW * 4;            // [kRecs] row, ks, vs
  static constexpr int kSeqOff = kRecOff + kRecs * 12 + 8;     // see SeqTab
  static constexpr int kBarOff = kSeqOff + kKvSeqsPerLaunch * 20 + 16;
  static constexpr int kBytes = kBarOff + kRW * kStages * 8;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kQOff % 16 == 0 && kMergeOff % 16 == 0 && kBarOff % 8 == 0 && kSeqOff % 8 == 0,
                "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

// Units before each sequence of the launch, and the sequences' entries.
struct SeqTab {
  long long* before;  // [seqs + 1]
  int *len, *m, *row0;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_out(const Kv8Args& a, long long i, float v) {
  uint16_t* o = static_cast<uint16_t*>(a.out);
  o[i] = a.type == TERN_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                             : __half_as_ushort(__float2half_rn(v));
}

template <int D, int MT>
__global__ void __launch_bounds__(kRW * 32, 1)
    kv8_rows_kernel(const __grid_constant__ CUtensorMap tm, const Kv8Args a, int max_rows) {
  using L = RL<D, MT>;
  constexpr int kW = D / 16;   // words of a lane per key row: 8 or 4 (k steps)
  constexpr int kNT = D / 8;   // output column tiles
  constexpr int kVW = D / 32;  // words of a lane per value row: 4 or 2
  grid_dependents_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff) + warp * L::kStages;
  uint8_t* ring = smem + warp * (L::kStages * L::kStage);
  float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  float* qscale = reinterpret_cast<float*>(smem + L::kQScaleOff);
  int* wexp = reinterpret_cast<int*>(smem + L::kExpOff);
  // first row of the page's keys in the codes' tensor map, with a bit for each
  // half that some row sees; -1 for a page out of range
  int* rec_page = reinterpret_cast<int*>(smem + L::kRecOff);
  float* rec_ks = reinterpret_cast<float*>(rec_page + kRecs);
  float* rec_vs = rec_ks + kRecs;
  SeqTab sq;
  sq.before = reinterpret_cast<long long*>(smem + L::kSeqOff);
  sq.len = reinterpret_cast<int*>(sq.before + kKvSeqsPerLaunch + 1);
  sq.m = sq.len + kKvSeqsPerLaunch;
  sq.row0 = sq.m + kKvSeqsPerLaunch;
  __shared__ int s_last;

  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    prefetch_tensormap(&tm);
  }
  grid_dependency_wait();  // every input, the output and the workspace belong to earlier work

  // ---- the launch's units: (sequence, row tile, head, page), pages fastest
  for (int b = threadIdx.x; b < a.seqs; b += kRW * 32) {
    const KvSeq s = kv_seq(a, b);
    if (!s.ok && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
    const long long rows = static_cast<long long>(s.m) * a.group;
    long long u = 0;
    if (s.ok && s.m > 0 && rows <= max_rows)
      u = static_cast<long long>(kv_pages(a, s.len - s.m, s.len - 1).count) * a.hkv *
          ((rows + L::kRows - 1) / L::kRows);
    sq.before[b + 1] = u;
    sq.len[b] = s.len;
    sq.m[b] = s.m;
    sq.row0[b] = s.row0;
  }
  __syncthreads();
  if (warp == 0) {
    // running sums of 32 sequences at a time
    long long carry = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
      const int b = b0 + lane;
      long long v = b < a.seqs ? sq.before[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      __syncwarp();
      if (b < a.seqs) sq.before[b + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) sq.before[0] = 0;
  }
  __syncthreads();
  const long long U = sq.before[a.seqs];
  const long long per = (U + gridDim.x - 1) / gridDim.x;  // units of a CTA
  const long long u_end = U < (blockIdx.x + 1ll) * per ? U : (blockIdx.x + 1ll) * per;
  const long long u_begin = static_cast<long long>(blockIdx.x) * per;
  if (u_begin >= u_end) return;

  // the sequence of unit u
  auto seq_of = [&](long long u) {
    int lo = 0, hi = a.seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sq.before[mid + 1] > u) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };

  // ---- state of the current segment (one sequence, row tile and head)
  uint32_t qf[MT == 1 ? kW : 1][4];  // (one tile) the query fragments
  float o[MT][kNT][4];
  float mx[MT][2], sum[MT][2], cs[MT][2];
  int pos[MT][2];  // the rows' positions; -1: no row
  int E = -127;

  unsigned issued = 0, used = 0;  // stages of this warp so far
  bool ok = true;

  long long c0 = u_begin;  // first unit whose record is held
  long long c1 = u_begin;
  long long pre = 0;  // next half-page (2 * unit + half) this warp requests

  auto issue_ahead = [&]() {
    // (whole warp) request half-pages until the ring is full
    while (pre < 2 * c1 && issued - used < L::kStages) {
      const int i = static_cast<int>((pre >> 1) - c0);
      const int rec = rec_page[i];
      const int half = static_cast<int>(pre & 1);
      if (rec >= 0 && ((rec >> half) & 1)) {
        if (lane == 0) {
          const int s = issued % L::kStages;
          const int row = (rec & ~(kBlk - 1)) + half * kHalf;
          mbar_arrive_expect_tx(&full[s], L::kStage);
          tma_load_2d(ring + s * L::kStage, &tm, 0, row, &full[s]);
          tma_load_2d(ring + s * L::kStage + kHalf * D, &tm, 0, row + a.hkv * kBlk, &full[s]);
        }
        ++issued;
      }
      pre += kRW;
    }
  };

  long long u = u_begin;
  while (u < u_end) {
    // ---- the segment that starts (or continues) at unit u
    const int b = seq_of(u);
    const int len = sq.len[b], m = sq.m[b];
    const int p_first = len - m, p_last = len - 1;
    const KvPages pages = kv_pages(a, p_first, p_last);
    const int np = pages.count;
    const long long seg = (u - sq.before[b]) / np;  // row tile * hkv + head
    const int hk = static_cast<int>(seg % a.hkv), rt = static_cast<int>(seg / a.hkv);
    const long long s_begin = sq.before[b] + seg * np, s_end = s_begin + np;
    const long long e_here = s_end < u_end ? s_end : u_end;
    const long long left = static_cast<long long>(m) * a.group - 1ll * rt * L::kRows;
    const int R = left < L::kRows ? static_cast<int>(left) : L::kRows;
    auto row_base = [&](int r) -> long long {  // element of q for row r of the tile
      const int rr = rt * L::kRows + r;
      return static_cast<long long>(sq.row0[b] + rr / a.group) * a.ld +
             static_cast<long long>(hk * a.group + rr % a.group) * a.hd;
    };
    auto out_base = [&](int r) -> long long {  // row of out
      const int rr = rt * L::kRows + r;
      return static_cast<long long>(sq.row0[b] + rr / a.group) * a.heads + hk * a.group +
             rr % a.group;
    };

    // queries: each warp scales some rows by a power of two into fp16
    for (int r = warp; r < L::kRows; r += kRW) {
      float v[D / 32];
      float big = 0.f;
      uint32_t raw[D / 64];
#pragma unroll
      for (int e = 0; e < D / 64; ++e) raw[e] = 0u;
      if (r < R) {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + row_base(r) + lane * (D / 32);
        if constexpr (D == 128) {
          const uint2 w = *reinterpret_cast<const uint2*>(src);
          raw[0] = w.x, raw[1] = w.y;
        } else {
          raw[0] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        unpack16(raw[e], a.type, v[2 * e], v[2 * e + 1]);
        big = fmaxf(big, fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
      // largest element into [2^14, 2^15); the two steps keep the factors in range
      int ex = static_cast<int>((__float_as_uint(big) >> 23) & 0xFF) - 127;
      if (big == 0.f) ex = 14;
      const float up1 = __uint_as_float(static_cast<uint32_t>((14 - ex) / 2 + 127) << 23);
      const float up2 =
          __uint_as_float(static_cast<uint32_t>((14 - ex) - (14 - ex) / 2 + 127) << 23);
      uint32_t* dst = reinterpret_cast<uint32_t*>(smem + L::kQOff + r * L::kQStride);
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        // 8-byte unit w of the row sits at w ^ (w / (units / 2))
        const int word = lane * (D / 64) + e;
        const int unit = word >> 1;
        const int at = ((unit ^ (unit / (D / 8))) << 1) | (word & 1);
        dst[at] = half2_bits(v[2 * e] * up1 * up2, v[2 * e + 1] * up1 * up2);
      }
      if (lane == 0) qscale[r] = 1.0f / up1 / up2;
    }

    // the rest of the segment in this CTA's range, in pieces whose page
    // records fit
    bool first_piece = true;
    while (u < e_here) {
      if (u >= c1) {
        // records of the next units of the range (all segments): where the
        // pages lie, which halves any row sees, and the scales
        c0 = u;
        c1 = u_end < c0 + kRecs ? u_end : c0 + kRecs;
        for (int i = threadIdx.x; i < static_cast<int>(c1 - c0); i += kRW * 32) {
          const long long uu = c0 + i;
          const int bb = seq_of(uu);
          const int ll = sq.len[bb], mm = sq.m[bb];
          const KvPages pp = kv_pages(a, ll - mm, ll - 1);
          const long long in = uu - sq.before[bb];
          const int lp = pp.page(static_cast<int>(in % pp.count));
          const int hh = static_cast<int>((in / pp.count) % a.hkv);
          const int page = a.table[static_cast<size_t>(bb) * a.width + lp];
          int rec = -1;
          if (page < 0 || page >= a.pages) {
            atomicOr(a.err, kErrIndex);
          } else {
            rec = (page * 2 * a.hkv + hh) * kBlk;
            for (int hf = 0; hf < 2; ++hf) {
              const int j0 = lp * kBlk + hf * kHalf;
              if (kv_any(a, ll - mm, ll - 1, j0, j0 + kHalf - 1)) rec |= 1 << hf;
            }
            const float* sc = a.scales + (static_cast<size_t>(page) * 2) * a.hkv + hh;
            rec_ks[i] = sc[0];
            rec_vs[i] = sc[a.hkv];
          }
          rec_page[i] = rec;
        }
        __syncthreads();
        pre = 2 * c0 + warp;
        issue_ahead();
      }
      if (first_piece) {
        __syncthreads();  // queries staged
        first_piece = false;
        if constexpr (MT == 1) {
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            const int unit = (D / 16) * t + j;
            const int at = (unit ^ (unit / (D / 8))) * 8;
            const uint2 x = *reinterpret_cast<const uint2*>(smem + L::kQOff + g * L::kQStride + at);
            const uint2 y =
                *reinterpret_cast<const uint2*>(smem + L::kQOff + (g + 8) * L::kQStride + at);
            qf[j][0] = x.x, qf[j][2] = x.y, qf[j][1] = y.x, qf[j][3] = y.y;
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = mt * 16 + g + 8 * x;
            mx[mt][x] = -INFINITY;
            sum[mt][x] = 0.f;
            cs[mt][x] = qscale[r] * a.scale_log2;
            pos[mt][x] = r < R ? p_first + (rt * L::kRows + r) / a.group : -1;
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[mt][n][x] = 0.f;
        }
        E = -127;
      }
      const long long piece = e_here < c1 ? e_here : c1;
      // this warp's half-pages of [u, piece): those congruent to its number
      long long h = 2 * u;
      h += (warp + 2 * c0 - h) & (kRW - 1);
      for (; h < 2 * piece && ok; h += kRW) {
        const int i = static_cast<int>((h >> 1) - c0);
        const int half = static_cast<int>(h & 1);
        const int rec = rec_page[i];
        if (rec < 0 || !((rec >> half) & 1)) continue;
        const int s = used % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait_clk(&full[s], (used / L::kStages) & 1, a.err));
        if (!ok) break;
        const uint8_t* kb = ring + s * L::kStage;
        const uint8_t* vb = kb + kHalf * D;
        const int j0 = pages.page(static_cast<int>((h >> 1) - s_begin)) * kBlk + half * kHalf;
        const float ks = rec_ks[i];
        const VScale vs = split_vscale(rec_vs[i]);

        // S = Q Kc^T for 32 tokens
        float sc[MT][4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x) sc[mt][n][x] = 0.f;
          uint32_t w[kW];
          const int row = 8 * n + g;
          if constexpr (D == 128) {
            const uint8_t* kr = kb + row * D;
            const uint4 x = lds_v4(kr + (((2 * t) ^ g) << 4));
            const uint4 y = lds_v4(kr + (((2 * t + 1) ^ g) << 4));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
          } else {
            const uint4 x = lds_v4(kb + row * D + ((t ^ ((g >> 1) & 3)) << 4));
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < kW; ++j) {
            uint32_t b0, b1;
            codes_to_half(w[j], b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (MT == 1) {
                mma_16816(sc[mt][n], qf[j], b0, b1);
              } else {
                const int unit = (D / 16) * t + j;
                const int at = (unit ^ (unit / (D / 8))) * 8;
                const uint8_t* qr = smem + L::kQOff + (mt * 16 + g) * L::kQStride + at;
                const uint2 x = lds_v2(qr);
                const uint2 y = lds_v2(qr + 8 * L::kQStride);
                const uint32_t af[4] = {x.x, y.x, x.y, y.y};
                mma_16816(sc[mt][n], af, b0, b1);
              }
            }
          }
        }

        // softmax of the half-page
        const bool all = kv_all(a, p_first, p_last, j0, j0 + kHalf - 1);
        const int En = vs.e > E ? vs.e : E;
        const float escale = En == E ? 1.f : exp2f(static_cast<float>(E - En));
        const float lf = log2f(vs.f), rf = 1.0f / vs.f;
        uint32_t pf[MT][2][4];
        bool grew = En != E;
        float alpha[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float c = cs[mt][x] * ks;
            float big = -INFINITY;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float v = sc[mt][n][2 * x + y] * c;
                if (!all && !kv_sees(a, pos[mt][x], j0 + 8 * n + 2 * t + y)) v = -INFINITY;
                sc[mt][n][2 * x + y] = v;
                big = fmaxf(big, v);
              }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const float now = fmaxf(mx[mt][x], big);
            const float ref = now == -INFINITY ? 0.f : now;
            alpha[mt][x] = exp2_approx(mx[mt][x] - ref);
            grew = grew || now > mx[mt][x];
            mx[mt][x] = now;
            float part = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float v = sc[mt][n][2 * x + y];
                // (a masked token's weight is 0 even where f is NaN)
                const float p = v == -INFINITY ? 0.f : exp2_approx((v - ref) + (kPOff + lf));
                sc[mt][n][2 * x + y] = p;
                part += p;
              }
            sum[mt][x] = sum[mt][x] * alpha[mt][x] + (part == 0.f ? 0.f : part * rf);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            pf[mt][k][0] = half2_bits(sc[mt][2 * k][0], sc[mt][2 * k][1]);
            pf[mt][k][1] = half2_bits(sc[mt][2 * k][2], sc[mt][2 * k][3]);
            pf[mt][k][2] = half2_bits(sc[mt][2 * k + 1][0], sc[mt][2 * k + 1][1]);
            pf[mt][k][3] = half2_bits(sc[mt][2 * k + 1][2], sc[mt][2 * k + 1][3]);
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float f0 = alpha[mt][0] * escale, f1 = alpha[mt][1] * escale;
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              o[mt][n][0] *= f0;
              o[mt][n][1] *= f0;
              o[mt][n][2] *= f1;
              o[mt][n][3] *= f1;
            }
          }
          E = En;
        }

        // O += P Vc 2^(e - E)
        const uint32_t hp = half_pow2(vs.e - E);
        const uint32_t vmul = hp | (hp << 16);
        uint32_t vadd;  // -1152 * 2^(e - E), exact
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(vadd) : "r"(vmul), "r"(0xE480E480u));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[4][kVW];  // tokens 2t, 2t+1, 2t+8, 2t+9 of the step's 16
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 16 * k + 2 * t + (x & 1) + 8 * (x >> 1);
            if constexpr (D == 128) {
              const uint4 v = lds_v4(vb + row * D + ((g ^ (row & 7)) << 4));
              w[x][0] = v.x, w[x][1] = v.y, w[x][2] = v.z, w[x][3] = v.w;
            } else {
              const uint2 v =
                  lds_v2(vb + row * D + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
              w[x][0] = v.x, w[x][1] = v.y;
            }
          }
#pragma unroll
          for (int q = 0; q < kVW; ++q) {
            const uint32_t w0 = w[0][q] ^ 0x80808080u, w1 = w[1][q] ^ 0x80808080u;
            const uint32_t w2 = w[2][q] ^ 0x80808080u, w3 = w[3][q] ^ 0x80808080u;
            const uint32_t lo[2] = {__byte_perm(w0, w1, 0x5140), __byte_perm(w2, w3, 0x5140)};
            const uint32_t hi[2] = {__byte_perm(w0, w1, 0x7362), __byte_perm(w2, w3, 0x7362)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t bf[2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t c =
                    __byte_perm(e < 2 ? lo[x] : hi[x], 0x64646464u, (e & 1) ? 0x4342 : 0x4140);
                asm("fma.rn.f16x2 %0, %1, %2, %3;"
                    : "=r"(bf[x])
                    : "r"(c), "r"(vmul), "r"(vadd));
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_16816(o[mt][4 * q + e], pf[mt][k], bf[0], bf[1]);
            }
          }
        }
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
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sum[mt][x] += __shfl_xor_sync(0xffffffffu, sum[mt][x], 1);
        sum[mt][x] += __shfl_xor_sync(0xffffffffu, sum[mt][x], 2);
        if (t == 0) ml[warp * L::kRows + mt * 16 + g + 8 * x] = make_float2(mx[mt][x], sum[mt][x]);
      }
    if (lane == 0) wexp[warp] = E;
    const bool whole = s_begin >= u_begin && s_end <= u_end;
    const long long cta_first = s_begin / per, cta_last = (s_end - 1) / per;
    const int parts = static_cast<int>(cta_last - cta_first + 1);
    auto part_of = [&](long long cta) {  // the partial results of the segment in that CTA
      return a.partials + (2 * cta + (cta == cta_first ? 1 : 0)) * (L::kRows * (D + 2));
    };
    float* mine = part_of(blockIdx.x);
    for (int r0 = 0; r0 < R; r0 += 4) {
      // rows r0 .. r0 + 3 of every warp
      const int mt = r0 >> 4, x = (r0 >> 3) & 1;
      if ((g >> 2) == ((r0 >> 2) & 1)) {
        float* dst = merge + (warp * 4 + (g & 3)) * D + (D / 4) * t;
#pragma unroll
        for (int m2 = 0; m2 < MT; ++m2)
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2)
            if (m2 == mt && x2 == x) {
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
                dst[n] = o[m2][n][2 * x2];
                dst[kNT + n] = o[m2][n][2 * x2 + 1];
              }
            }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 4 * D; i += kRW * 32) {
        const int r = r0 + i / D, d = i % D;
        if (r < R) {
          float big = -INFINITY;
          int Em = -127;
#pragma unroll
          for (int w = 0; w < kRW; ++w) {
            big = fmaxf(big, ml[w * L::kRows + r].x);
            Em = max(Em, wexp[w]);
          }
          const float ref = big == -INFINITY ? 0.f : big;
          float acc = 0.f, l = 0.f;
#pragma unroll
          for (int w = 0; w < kRW; ++w) {
            const float2 v = ml[w * L::kRows + r];
            if (v.x != -INFINITY || v.y != 0.f) {
              const float f = exp2f(v.x - ref);
              l += v.y * f;
              acc += merge[(w * 4 + i / D) * D + d] * (f * exp2f(static_cast<float>(wexp[w] - Em)));
            }
          }
          const float val = l == 0.f ? 0.f : acc / l * exp2f(static_cast<float>(Em));
          if (whole) {
            const long long ob = out_base(r);
            store_out(a, ob * D + d, val);
            if (a.lse && d == 0)
              a.lse[ob] = l == 0.f ? -INFINITY : (big - kPOff + log2f(l)) * 0.6931471805599453f;
          } else {
            mine[r * D + d] = val;
            if (d == 0)
              reinterpret_cast<float2*>(mine + L::kRows * D)[r] = make_float2(big, l);
          }
        }
      }
      __syncthreads();
    }
    if (!whole) {
      // the last of the segment's CTAs adds the parts in CTA order
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        s_last = atomic_add_acq_rel_gpu(&a.tickets[cta_first], 1) == parts - 1;
      __syncthreads();
      if (s_last) {
        if (threadIdx.x == 0) a.tickets[cta_first] = 0;
        for (int i = threadIdx.x; i < R * D; i += kRW * 32) {
          const int r = i / D, d = i % D;
          float big = -INFINITY;
          for (int p = 0; p < parts; ++p)
            big = fmaxf(big, __ldcg(part_of(cta_first + p) + L::kRows * D + 2 * r));
          const float ref = big == -INFINITY ? 0.f : big;
          float acc = 0.f, l = 0.f;
          for (int p = 0; p < parts; ++p) {
            const float* src = part_of(cta_first + p);
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src + L::kRows * D) + r);
            if (v.y != 0.f) {
              const float f = v.y * exp2f(v.x - ref);
              l += f;
              acc = fmaf(f, __ldcg(src + r * D + d), acc);
            }
          }
          const long long ob = out_base(r);
          store_out(a, ob * D + d, l == 0.f ? 0.f : acc / l);
          if (a.lse && d == 0)
            a.lse[ob] = l == 0.f ? -INFINITY : (big - kPOff + log2f(l)) * 0.6931471805599453f;
        }
      }
      __syncthreads();
    }
  }
  // no copy of this warp outlives it
  for (; used < issued; ++used)
    if (!mbar_wait_clk(&full[used % L::kStages], (used / L::kStages) & 1, a.err)) break;
}

template <int D, int MT>
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
        pdl_launch_config(attr, dim3(grid), dim3(kRW * 32), RL<D, MT>::kAlloc, stream);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_rows_kernel<D, MT>, *tm, p, max_rows);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

size_t kv8_rows_partial_bytes(int dim) {
  return static_cast<size_t>(kSmallTMaxCtas) * 2 * 32 * (dim + 2) * sizeof(float);
}

cudaError_t kv8_rows_set_attributes() {
  cudaError_t e = cudaSuccess;
#define TERN_ROWS_ATTR(D, MT)                                                   \
  if (e == cudaSuccess)                                                         \
    e = cudaFuncSetAttribute(kv8_rows_kernel<D, MT>,                            \
                             cudaFuncAttributeMaxDynamicSharedMemorySize, RL<D, MT>::kAlloc);
  TERN_ROWS_ATTR(64, 1)
  TERN_ROWS_ATTR(64, 2)
  TERN_ROWS_ATTR(128, 1)
  TERN_ROWS_ATTR(128, 2)
#undef TERN_ROWS_ATTR
  return e;
}

cudaError_t launch_kv8_rows(const CUtensorMap* tm, const Kv8Args& a, int max_rows, int num_sms,
                            cudaStream_t stream, int* launches) {
  const bool one = a.max_new * a.group <= 16;
  if (a.dim == 128)
    return one ? launch_one<128, 1>(tm, a, max_rows, num_sms, stream, launches)
               : launch_one<128, 2>(tm, a, max_rows, num_sms, stream, launches);
  return one ? launch_one<64, 1>(tm, a, max_rows, num_sms, stream, launches)
             : launch_one<64, 2>(tm, a, max_rows, num_sms, stream, launches);
}

}  // namespace tern
