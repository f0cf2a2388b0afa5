// The few-row attention's arithmetic on half-pages of 32 tokens, with m16n8k16
// fp16 tensor instructions and fp32 sums, and what its kernels need of a page.
//
// Transposed: tokens (and then the elements of the output) are the operand of 16
// rows, tiles of eight query rows the one of eight.  The contraction order is
// free, so a lane's operand elements are the 32 (16) consecutive bytes it loads:
// position 2t, 2t+1, 2t+8, 2t+9 of step j is element 32t + 4j + 0..3 of the row.
// (Lane 4 g + t of a warp: group g, place t.)
#pragma once

#include "tern_kv8.cuh"

namespace tern {

constexpr int kHalf = 32;     // tokens of a half-page
constexpr float kROff = 10.f, kRLazy = 4.f;
// Value scales of 2^-38 to 2^38 (and 0) have their logarithm in the weights'
// exponents; blocks of others are left to far_row.  (The least weight that the
// sum must have, 2^(10 - 76) times 2^-40 beside the largest, is a normal number.)
constexpr float kMinScale = 3.637978807091713e-12f, kMaxScale = 274877906944.f;
// Whether a block is left to far_row.
__device__ __forceinline__ bool far_scales(float ks, float vs) {
  return good_scales(ks, vs) && vs != 0.f && !(vs >= kMinScale && vs <= kMaxScale);
}
constexpr float kCodeUp = 16777216.f;        // 2^24
constexpr uint32_t kNeg128 = 0x80808080u;   // a pair of -128 * 2^-24 in fp16

// What a half-page's arithmetic needs of its page, in one 16-byte load.
struct __align__(16) PageRec {
  float ks, lv;  // scale of the keys; log2 of the scale of the values
  float rv;      // 1 over the latter, or NaN where the scales cannot be used
  float any;     // 1, or 0 where the values have no part in the output
};
__device__ __forceinline__ PageRec page_rec(float ks, float vs) {
  PageRec rec = {0.f, 0.f, 1.f, 0.f};
  // (a value scale of 0 weighs as the least, so that its block hardly raises a
  // row's reference; scales that cannot be used keep out of the arithmetic)
  const bool good = good_scales(ks, vs);
  rec.ks = good ? ks : 0.f;
  if (!good) {
    rec.rv = __uint_as_float(0x7FC00000u);
  } else if (!far_scales(ks, vs)) {
    const float v = fmaxf(vs, kMinScale);
    rec.lv = log2f(v);
    rec.rv = 1.0f / v;
    rec.any = vs != 0.f ? 1.f : 0.f;
  }
  return rec;
}
// Beside it, the first row of the page's keys in the codes' tensor map (a
// multiple of 64) with these bits (no kMHalf where it is left to far_row), or -1
// for a page out of range.
enum : int {
  kMHalf = 1,  // << half: some row sees a token of the half
  kMAll = 4    // << half: every row sees all of them
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The bytes of u (codes + 128) that sel picks, as a pair in fp16: kBiased the
// subnormals (code + 128) 2^-24, a byte beside a zero byte; otherwise the codes
// themselves, from 1024 + (code + 128).  Both are exact.
template <bool kBiased>
__device__ __forceinline__ uint32_t code_pair(uint32_t u, uint32_t sel) {
  if (kBiased) return __byte_perm(u, 0u, sel);
  const uint32_t v = __byte_perm(u, 0x64646464u, sel);
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x64806480u));
  return d;
}
// The transpose of the warp's 8 x 8 matrix of 16-bit elements (lane 4 i + j
// holds elements 2 j and 2 j + 1 of row i).
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One tile of rows takes the codes as biased subnormals, which saves an
// instruction per pair, and products of all -128 for the bias; with two tiles the
// values' separate sums would not fit the registers.
constexpr bool biased(int tiles) { return tiles == 1; }

// Element unit j of a lane's part of the staged query 8 n + g.
template <int D>
__device__ __forceinline__ uint2 staged_query(const uint8_t* q, int n, int j, int g, int t) {
  const int unit = (D / 16) * t + j;
  return lds_v2(q + (8 * n + g) * (2 * D + 16) + (unit ^ (unit / (D / 8))) * 8);
}

// What the scores of a tile of queries start from: -128 * 2^-24 times the sums
// of the rows' queries.
template <int D, bool kBiased, typename Query>
__device__ __forceinline__ void query_bias(const Query& query, float (&s0)[4]) {
  const uint32_t neg128[4] = {kNeg128, kNeg128, kNeg128, kNeg128};
#pragma unroll
  for (int x = 0; x < 4; ++x) s0[x] = 0.f;
#pragma unroll
  for (int j = 0; kBiased && j < D / 16; ++j) {
    const uint2 q = query(j);
    mma_16816(s0, neg128, q.x, q.y);
  }
}

// The keys' codes (in shared memory as a tensor map's swizzled box) of a lane:
// tokens g, 8 + g, 16 + g, 24 + g.
template <int D>
__device__ __forceinline__ void half_keys(const uint8_t* kb, int g, int t,
                                          uint32_t (&kw)[4][D / 16]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint8_t* kr = kb + (8 * n + g) * D;
    if constexpr (D == 128) {
      const uint4 x = lds_v4(kr + (((2 * t) ^ g) << 4));
      const uint4 y = lds_v4(kr + (((2 * t + 1) ^ g) << 4));
      kw[n][0] = x.x, kw[n][1] = x.y, kw[n][2] = x.z, kw[n][3] = x.w;
      kw[n][4] = y.x, kw[n][5] = y.y, kw[n][6] = y.z, kw[n][7] = y.w;
    } else {
      const uint4 x = lds_v4(kr + ((t ^ ((g >> 1) & 3)) << 4));
      kw[n][0] = x.x, kw[n][1] = x.y, kw[n][2] = x.z, kw[n][3] = x.w;
    }
  }
}

// S^T = Kc Q^T for 32 tokens, two tiles of 16 side by side.
template <int D, int NT, typename Query>
__device__ __forceinline__ void half_scores(const uint32_t (&kw)[4][D / 16],
                                            const float (&s0)[NT][4], float (&sc)[NT][2][4],
                                            const Query& query) {
  constexpr int kW = D / 16;  // words of a lane per key row (k steps)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) sc[n][i][x] = s0[n][x];
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    uint2 q[NT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t af[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t u = kw[2 * i + x][j] ^ 0x80808080u;
        af[x] = code_pair<biased(NT)>(u, 0x4140);
        af[x + 2] = code_pair<biased(NT)>(u, 0x4342);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (i == 0) q[n] = query(n, j);
        mma_16816(sc[n][i], af, q[n].x, q[n].y);
      }
    }
  }
}

// Scores of tokens (32 from j0) that the rows at pos do not see: -inf.
template <int NT>
__device__ __forceinline__ void half_mask(const Kv8Args& a, const int (&pos)[NT][2], int j0, int g,
                                          float (&sc)[NT][2][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t see = static_cast<uint32_t>(kv_mask(a, pos[n][x], j0)) >> g;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!(see & (1u << (8 * k)))) sc[n][k >> 1][2 * (k & 1) + x] = -INFINITY;
    }
}

// The values' codes: tokens 2t, 2t+1, 2t+8, 2t+9 of each step's 16.
template <int D>
__device__ __forceinline__ void half_values(const uint8_t* vb, int g, int t,
                                            uint32_t (&vw)[2][4][D / 32]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t(&w)[4][D / 32] = vw[k];
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
  }
}

// The online softmax of a half-page: its scores sc to weights, with the rows' references
// and sums, and the output so far where a reference rises.  cs: what a row's scores are
// times, but for the key scale.
template <int D, int NT>
__device__ __forceinline__ void half_softmax(const PageRec& rec, const float (&cs)[NT][2],
                                             float (&sc)[NT][2][4], float (&ref)[NT][2],
                                             float (&sum)[NT][2], float (&o)[NT][D / 16][4]) {
  constexpr float kUp = biased(NT) ? kCodeUp : 1.f;  // 1 over the codes' unit
  bool raise = false;
  float c[NT][2], big[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // (a scale of 0 must not turn a masked -inf into a NaN)
      c[n][x] = fmaxf(cs[n][x] * rec.ks * kUp, 1e-37f);
      big[n][x] = fmaxf(fmaxf(sc[n][0][x], sc[n][0][x + 2]), fmaxf(sc[n][1][x], sc[n][1][x + 2]));
      raise = raise || fmaf(big[n][x], c[n][x], rec.lv) > ref[n][x] + kRLazy;
    }
  if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float scale[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = fmaf(big[n][x], c[n][x], rec.lv);  // -inf: no visible token
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        scale[x] = 1.f;
        if (top > ref[n][x] + kRLazy) {
          scale[x] = exp2_approx(ref[n][x] - top);  // 0 for the row's first
          sum[n][x] *= scale[x];
          ref[n][x] = top;
        }
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][i][x] *= scale[x & 1];
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float add = kROff + rec.lv - (ref[n][x] == -INFINITY ? 0.f : ref[n][x]);
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int y = x; y < 4; y += 2) {
          sc[n][i][y] = exp2_approx(fmaf(sc[n][i][y], c[n][x], add));
          part += sc[n][i][y];
        }
      // (scales that cannot be used: the rows that see the page, and only they, become
      // NaN)
      if (big[n][x] != -INFINITY) sum[n][x] = fmaf(part, rec.rv, sum[n][x]);
    }
  }
}

// O^T += Vc^T P^T, the weights P in the scores' place, times any (a pair of 1 or 0
// in fp16).
template <int D, int NT>
__device__ __forceinline__ void half_products(const float (&sc)[NT][2][4], uint32_t any,
                                              const uint32_t (&vw)[2][4][D / 32],
                                              float (&o)[NT][D / 16][4]) {
  constexpr bool kBiased = biased(NT);
  const uint32_t neg128[4] = {kNeg128, kNeg128, kNeg128, kNeg128};
  uint2 pf[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      auto mul = [&](uint32_t p) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(any));
        return r;
      };
      pf[n][i].x = transposed(mul(half2_bits(sc[n][i][0], sc[n][i][1])));
      pf[n][i].y = transposed(mul(half2_bits(sc[n][i][2], sc[n][i][3])));
    }
  float oc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int x = 0; x < 4; ++x) oc[n][x] = 0.f;
#pragma unroll
    for (int k = 0; kBiased && k < 2; ++k) mma_16816(oc[n], neg128, pf[n][k].x, pf[n][k].y);
  }
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    // elements 4 q to 4 q + 3 of the lane's group of D / 8, two at a time
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float od[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) od[n][x] = kBiased ? oc[n][x] : o[n][2 * q + i][x];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t(&w)[4][D / 32] = vw[k];
        const uint32_t sel = i ? 0x7362 : 0x5140;
        const uint32_t u0 = __byte_perm(w[0][q], w[1][q], sel) ^ 0x80808080u;
        const uint32_t u1 = __byte_perm(w[2][q], w[3][q], sel) ^ 0x80808080u;
        const uint32_t af[4] = {code_pair<kBiased>(u0, 0x4140), code_pair<kBiased>(u0, 0x4342),
                                code_pair<kBiased>(u1, 0x4140), code_pair<kBiased>(u1, 0x4342)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_16816(od[n], af, pf[n][k].x, pf[n][k].y);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          float(&to)[4] = o[n][2 * q + i];
          if (kBiased)
            unpair_f32(add_pair(pair_f32(to[x], to[x + 1]), pair_f32(od[n][x], od[n][x + 1])),
                       to[x], to[x + 1]);
          else
            to[x] = od[n][x], to[x + 1] = od[n][x + 1];
        }
    }
  }
}

// A row's softmax over some pages: l = sum 2^(ref - kROff), and the row's output
// of them (elements lane * D / 32 on).
template <int D>
struct FarRow {
  float ref, sum, o[D / 32];
};
// The row at position p over those pages [begin, end) of the segment's list whose
// value scales are out of [kMinScale, kMaxScale], by a warp: a token per lane for
// the scores, elements per lane for the output, which has a reference of its own
// (it follows the largest weight times value scale).  Such blocks are rare: what
// counts is that there is little code.  query: the staged row; c: what a score
// is times, but for the key scale.
template <int D, typename Pages>
__device__ __forceinline__ FarRow<D> far_row(const Kv8Args& a, const uint8_t* query, float c, int p,
                                             int b, int hk, const Pages& pages, int begin,
                                             int end) {
  const int lane = threadIdx.x & 31;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int kV = D / 32;
  FarRow<D> f;
  f.ref = -INFINITY;
  f.sum = 0.f;
#pragma unroll
  for (int y = 0; y < kV; ++y) f.o[y] = 0.f;
  float unit = -INFINITY;
#pragma unroll 1
  for (int i0 = begin; i0 < end; i0 += 32) {
    // a page per lane: is it one?
    int page = -1, lp = 0;
    float ks = 0.f, vs = 0.f;
    if (i0 + lane < end) {
      lp = pages.page(i0 + lane);
      page = a.table[static_cast<size_t>(b) * a.width + lp];
      if (page >= 0 && page < a.pages) {
        const float* sc = a.scales + static_cast<size_t>(page) * 2 * a.hkv + hk;
        ks = sc[0], vs = sc[a.hkv];
      }
    }
#pragma unroll 1
    for (unsigned set = __ballot_sync(kAll, far_scales(ks, vs)); set; set &= set - 1) {
      const int from = __ffs(set) - 1;
      const size_t at = static_cast<size_t>(__shfl_sync(kAll, page, from)) * 2 * a.hkv + hk;
      const float ck = fmaxf(c * __shfl_sync(kAll, ks, from), 1e-37f);
      const float lv = log2f(__shfl_sync(kAll, vs, from));
      const uint64_t see = kv_mask(a, p, __shfl_sync(kAll, lp, from) * kBlk);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int8_t* kr = a.codes + (at * kBlk + half * kHalf + lane) * D;
        float s = 0.f;
#pragma unroll 1
        for (int e = 0; e < D; e += 4) {
          const uint2 q = lds_v2(query + ((e / 4) ^ (e / 4 / (D / 8))) * 8);
          const char4 k = *reinterpret_cast<const char4*>(kr + e);
          float q0, q1, q2, q3;
          unpack16(q.x, TERN_F16, q0, q1);
          unpack16(q.y, TERN_F16, q2, q3);
          s = fmaf(q0, k.x, fmaf(q1, k.y, fmaf(q2, k.z, fmaf(q3, k.w, s))));
        }
        s = (see >> (half * kHalf + lane)) & 1 ? s * ck : -INFINITY;
        float top = s;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, k));
        if (!__any_sync(kAll, s != -INFINITY)) continue;
        if (top > f.ref) {
          f.sum *= exp2_approx(f.ref - top);
          f.ref = top;
        }
        if (top + lv > unit) {
          const float less = exp2_approx(unit - (top + lv));
          unit = top + lv;
#pragma unroll
          for (int y = 0; y < kV; ++y) f.o[y] *= less;
        }
        f.sum += exp2_approx(s - f.ref + kROff);
        const float w = exp2_approx(s + lv - unit);
        const int8_t* vr = a.codes + ((at + a.hkv) * kBlk + half * kHalf) * D + lane * kV;
#pragma unroll 1
        for (int j = 0; j < kHalf; ++j) {
          const float wj = __shfl_sync(kAll, w, j);
#pragma unroll
          for (int y = 0; y < kV; ++y) f.o[y] = fmaf(wj, vr[j * D + y], f.o[y]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) f.sum += __shfl_xor_sync(kAll, f.sum, k);
  const float one = f.sum == 0.f ? 0.f : exp2f(unit - f.ref + kROff) / f.sum;
#pragma unroll
  for (int y = 0; y < kV; ++y) f.o[y] *= one;
  return f;
}

}  // namespace tern
