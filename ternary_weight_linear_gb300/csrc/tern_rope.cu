// tern_rope: rotary positions of the rows of [T][heads][dim], and the host's
// tables of frequencies.
//   (u, v) -> m (u cos - v sin, u sin + v cos),  angle = position * freq
// for the pairs of a head's first `rotary` elements, the others as they are.
//
// A thread holds a unit of eight elements (four pairs) of a row in registers,
// computes its four turns once and applies them to that unit of several heads of
// the token.  Every element is read and written once: a prompt is bound by HBM, a
// decode step by one load after the position's.  Several heads a thread where
// that leaves work for all SMs: a turn costs some 30 instructions, a unit's loads
// and stores 4.  (Units of sixteen elements, at 61 registers, kept 14 warps an SM:
// 15.4 us for 2048 tokens of 56 heads in bf16, 11.4 here, 0.76 of the copy rate;
// the issue slots were 61 % busy at 12.6.  One or two heads a token leave the turns alone:
// 65536 tokens of one head 13.2 us, their bytes 4.9.)
#include <math.h>

#include "tern_device.cuh"
#include "tern_rope.cuh"

namespace tern {
namespace {

template <int TYPE, int OUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeRows a) {
  grid_dependents_launch();
  // x: units of a head; y: heads; z: tokens
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.z + threadIdx.z;
  const RopeUnit unit(a.rope, threadIdx.x);
  grid_dependency_wait();  // the inputs and the output come from earlier work
  if (t >= a.T) return;
  float2 turn[4];
  for (int h0 = threadIdx.y; h0 < a.heads; h0 += kRopeBatch * blockDim.y) {
    RopeHeads<TYPE> x;
    x.load(unit, a.x, t * a.ld, a.hd, h0, blockDim.y, a.heads);
    if (h0 == threadIdx.y && unit.pair >= 0)
      rope_turns(a.rope, unit.pair, a.positions[t], turn);
    x.template store<OUT>(a.rope, unit, turn, a.out, t * a.out_ld, a.out_hd, h0, blockDim.y,
                          a.heads);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeRows& a, int num_sms, cudaStream_t stream) {
  const int units = a.dim / 8;
  // One head a thread until every SM has its threads, then four and more, in CTAs of 128
  // threads.  With one and four: 32 tokens of 48 heads of 128 2.07 and 2.20 us, 256 of
  // 40 3.17 and 3.29, 8192 of 8 13.1 and 7.5.  2048 of 56 heads take 12.1 with 14 of them
  // side by side, 11.2 with 8, 11.6 with 4, 16.6 with 2.
  const long long all = static_cast<long long>(a.T) * a.heads * units;
  const int each = all < static_cast<long long>(num_sms) * 2048 ? 1 : 4;
  int lanes = (a.heads + each - 1) / each;
  const int most = (each == 1 ? kRopeThreads : 128) / units;  // (at least one)
  if (lanes > most) lanes = most;
  int tokens = 128 / (units * lanes);
  if (tokens < 1) tokens = 1;
  if (tokens > a.T) tokens = a.T;
  if (tokens > 64) tokens = 64;  // (a block's third extent)
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_launch_config(attr, dim3((a.T - 1) / tokens + 1), dim3(units, lanes, tokens), 0, stream);
#define TERN_ROPE_CASE(TYPE, OUT) \
  if (a.type == TYPE && a.out_type == OUT) return cudaLaunchKernelEx(&cfg, rope_kernel<TYPE, OUT>, a);
  TERN_ROPE_CASE(TERN_F32, TERN_F32)
  TERN_ROPE_CASE(TERN_F32, TERN_BF16)
  TERN_ROPE_CASE(TERN_F32, TERN_F16)
  TERN_ROPE_CASE(TERN_BF16, TERN_F32)
  TERN_ROPE_CASE(TERN_BF16, TERN_BF16)
  TERN_ROPE_CASE(TERN_BF16, TERN_F16)
  TERN_ROPE_CASE(TERN_F16, TERN_F32)
  TERN_ROPE_CASE(TERN_F16, TERN_BF16)
  TERN_ROPE_CASE(TERN_F16, TERN_F16)
#undef TERN_ROPE_CASE
  return cudaErrorInvalidValue;
}

void rope_frequencies(int rotary, double base, int scaling, double factor, double trained,
                      double low, double high, uint64_t* freq, float* magnitude) {
  const double kTurn = 6.283185307179586;
  double grow = 1.0;
  if (scaling == TERN_ROPE_BASE) base *= pow(factor, static_cast<double>(rotary) / (rotary - 2));
  // the pairs (as real numbers) that turn `high` and `low` times in the trained
  // context
  double first = 0, last = 0;
  if (scaling == TERN_ROPE_RAMP) {
    const double per = rotary / (2 * log(base));
    first = floor(per * log(trained / (kTurn * high)));
    last = ceil(per * log(trained / (kTurn * low)));
    if (first < 0) first = 0;
    if (last > rotary - 1) last = rotary - 1;
    grow = 0.1 * log(factor) + 1.0;
  }
  for (int i = 0; i < rotary / 2; ++i) {
    double theta = pow(base, -2.0 * i / rotary);
    double keep = 1.0;  // share of the frequency that is not slowed
    if (scaling == TERN_ROPE_LINEAR) keep = 0.0;
    if (scaling == TERN_ROPE_BANDS) keep = (trained * theta / kTurn - low) / (high - low);
    if (scaling == TERN_ROPE_RAMP)
      keep = 1.0 - (i - first) / (last - first > 0.001 ? last - first : 0.001);
    keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
    theta *= keep + (1.0 - keep) / factor;
    // (base > 1 and factor >= 1: at most a radian, 0.16 of 2^64)
    freq[i] = static_cast<uint64_t>(ldexp(theta / kTurn, 64));
  }
  *magnitude = static_cast<float>(grow);
}

}  // namespace tern
