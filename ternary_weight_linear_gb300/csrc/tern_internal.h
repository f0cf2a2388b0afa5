// Internal interface between the C-ABI layer (tern_api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tern {

// Small-T rungs (T <= 16): k per pipeline stage.  Token tiles are TT = 1, 4,
// 8 or 16 tokens.
constexpr int kSTStageK = 1024;  // 256 packed bytes per row: two 128-byte TMA boxes
// Grid cap of the small-T kernel (one CTA per SM).
constexpr int kSmallTMaxCtas = 160;
// Most activation blocks the one-token kernel keeps resident in shared memory
// (one per distinct k stage a CTA visits); a one-token call that needs more
// runs on the four-token tile.
constexpr int kSmallTX1MaxSlots = 8;

// Workspace layout shared by all rungs: a synchronisation area of kSyncBytes
// (the small-T kernels' ticket counters, one int per CTA, which must hold
// zeros when a call starts; every call leaves them zeroed again), followed by
// the rung's scratch.
constexpr size_t kSyncBytes = 4096;
static_assert(kSmallTMaxCtas * sizeof(int) <= kSyncBytes, "sync area");

// Partial row sums of a TT tile's row blocks split between CTAs:
// [kSmallTMaxCtas][2][TT][128] fp32.
size_t smallt_partials_bytes(int tt);
// Scratch after the sync area for a TT tile and K: the partial sums, then
// (TT > 1) the activation blocks built by the prep kernel.
size_t smallt_work_bytes(int tt, int K);
// Rows per CTA row block (the TMA box height).
int smallt_rows(int tt);
// Token tile of a T = 1 call: 1 when the one-token kernel's resident
// activation blocks fit for (K, N) on num_sms SMs, else 4.
int smallt_gemv_tile(int K, int N, int num_sms);
cudaError_t smallt_set_attributes();
// Launch the small-T kernel(s) for tokens [tok0, tok0 + Tt) with Tt <= tt.
// tmW: Wp's tensor map; sync: the zeroed sync area; work:
// smallt_work_bytes(tt, K) bytes.  act: how the activations are staged
// (kActExact: exact bf16 pieces; kActRotated: the same for the
// Hadamard-rotated activations, K % 1024 == 0; kActInt8: per-token int8
// codes, the s8 definition; kActCodes: the s8 definition on the caller's codes
// and token scales, x unused).  Adds the number of kernels launched to
// *launches.
enum : int { kActExact = 0, kActRotated = 1, kActInt8 = 2, kActCodes = 3 };
struct ActCodes {
  const int8_t* q = nullptr;       // [T][K]
  const float* x_scale = nullptr;  // [T]
};
cudaError_t launch_smallt(int tt, const CUtensorMap* tmW, const uint32_t* Wp,
                          const uint16_t* scales, const uint16_t* x, const ActCodes& codes,
                          int* sync, uint8_t* work, float* y, int K, int N, int tok0, int Tt,
                          int num_sms, int act, int* err, cudaStream_t stream, int* launches);

// s8 rung: tiles of 128 weight rows x 128 tokens on tcgen05.
constexpr int kS8TileN = 128;
constexpr int kS8TileT = 128;
constexpr int kS8SmallTileT = 32;  // token tile of the s8 rung for T <= 32
// Chunked last wave of the s8 rung: at most this many group ranges per tile;
// the chunks' partial sums take kS8PartialBytes of workspace after the
// pieces, and their tickets the synchronisation area.
constexpr int kS8FoldWarps = 8;                          // warps folding the accumulators
constexpr int kS8YBoxT = kS8TileT * 4 / kS8FoldWarps;   // tokens per fold warp's output box
constexpr int kS8MaxChunks = 4;

// Work split of the prefill rungs (s8, bf16): P CTAs walk nfull whole tiles,
// then the rest of the tiles as `chunks` group ranges each.  Chunking applies
// when the rest fills at most half a wave, so that a fraction of a tile per
// CTA finishes the call instead of a whole tile on few SMs.
struct TileSplit {
  int P, nfull, chunks;
};
inline TileSplit tile_split(int tiles, int G, int num_sms) {
  TileSplit sp;
  const int rounds = tiles / num_sms;
  const int rest = tiles - rounds * num_sms;
  sp.nfull = tiles;
  sp.chunks = 1;
  if (rest > 0 && 2 * rest <= num_sms) {
    int c = num_sms / rest;
    if (c > kS8MaxChunks) c = kS8MaxChunks;
    if (c > G / 2) c = G / 2;
    if (c >= 2) {
      sp.nfull = rounds * num_sms;
      sp.chunks = c;
    }
  }
  const int items = sp.nfull + (tiles - sp.nfull) * sp.chunks;
  sp.P = items < num_sms ? items : num_sms;
  return sp;
}
// (at most 160 chunk items, each kS8FoldWarps blocks of kS8YBoxT x 32 floats)
constexpr size_t kS8PartialBytes =
    static_cast<size_t>(160) * kS8FoldWarps * kS8YBoxT * 32 * sizeof(float);
cudaError_t s8_set_attributes();
// Token tile the s8 rung uses for T tokens (the pieces' tensor maps' box
// height): kS8SmallTileT for T <= kS8SmallTileT, else kS8TileT.
int s8_token_tile(int T);
// Stage ring of the s8 kernel: 12 for the small token tile; for the 128-token
// tile 4, or kS8DeepStages when the piece blocks (2 T K bytes, all read while
// a wave of CTAs crosses one row block) take more than half of the L2.
constexpr int kS8DeepStages = 6;
int s8_stages(int T, int K, size_t l2_bytes);

// bf16 rung: x reordered for the MMA (xp [T][K] bf16, optionally rotated
// first), then tiles of 128 weight rows x 128 tokens on tcgen05 kind::f16.
// tmW as for s8; tmX: xp as bytes [T][2K], box 128 B x 128 rows, 128-byte
// swizzle; tmY as for s8 (or null).
cudaError_t launch_interleave(const uint16_t* x, uint16_t* xp, int T, int K, int rotate,
                              int num_sms, cudaStream_t stream);
cudaError_t launch_bf16(const CUtensorMap* tmW, const CUtensorMap* tmX, const CUtensorMap* tmY,
                        const uint16_t* scales, float* y, int T, int K, int N, int* tickets,
                        float* partials, int num_sms, int* err, cudaStream_t stream);
cudaError_t bf16_set_attributes();
// tmW: packed weights, box 32 B x kS8TileN rows, no swizzle.  tmP1 / tmP2:
// the two fp8 activation pieces [T][K], box 128 B x s8_token_tile(T) rows,
// 128-byte swizzle.  y: fp32 [T][N], stored directly.  x_scale: [T] floats,
// readable up to T rounded up to 4.
cudaError_t launch_s8(const CUtensorMap* tmW, const CUtensorMap* tmP1, const CUtensorMap* tmP2,
                      const uint16_t* scales, const float* x_scale, float* y, int T, int K, int N,
                      int* tickets, float* partials, int num_sms, size_t l2_bytes, int* err,
                      cudaStream_t stream);

// Launch configuration of a programmatic dependent launch (the kernel may
// start while the previous kernel in the stream finishes; it waits for that
// kernel's results with griddepcontrol.wait).  attr: one attribute slot.
inline cudaLaunchConfig_t pdl_launch_config(cudaLaunchAttribute* attr, dim3 grid, dim3 block,
                                            size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Pack and quantise.
cudaError_t launch_pack(const int8_t* W, uint32_t* Wp, int K, int N, int* bad, int num_sms,
                        cudaStream_t stream);
cudaError_t launch_quant_s8(const uint16_t* x, int8_t* q, float* xs, int T, int K,
                            cudaStream_t stream);
// The s8 rung's activations: the int8 codes split into two exact e4m3 pieces.
// rotate: quantise the blockwise Hadamard rotation of x (K % 1024 == 0,
// K <= kRotateMaxK: the rotated row is staged in shared memory).
cudaError_t launch_quant_pieces(const uint16_t* x, uint8_t* p1, uint8_t* p2, float* xs, int T,
                                int K, int rotate, int num_sms, int* err, cudaStream_t stream);
// The same pieces of the caller's codes, and a copy of its token scales.
cudaError_t launch_code_pieces(const int8_t* q, const float* x_scale, uint8_t* p1, uint8_t* p2,
                               float* xs, int T, int K, int num_sms, cudaStream_t stream);
cudaError_t quant_set_attributes();

// Base-3 packed weights (26 bytes per 128-weight group) -> 2-bit codes.
cudaError_t launch_repack_t5(const uint8_t* P, uint32_t* Wp, int K, int N, int* bad,
                             cudaStream_t stream);
// Blockwise (1024) Hadamard rotation of bf16 activations; xr may equal x.
constexpr int kRotBlock = 1024;
// Largest K for which tern_linear can stage rotated activations (the s8
// rung keeps a rotated token row in shared memory).
constexpr int kRotateMaxK = 65536;
cudaError_t launch_rotate_bf16(const uint16_t* x, uint16_t* xr, int T, int K,
                               cudaStream_t stream);

// Residual addition, root-mean-square norm and int8 codes of [T][K] rows;
// see tern_add_rmsnorm_s8.  K <= kNormMaxK.
constexpr int kNormMaxK = 32768;
struct NormArgs {
  const void* x;
  long long x_ld;  // elements
  int x_type;
  const void* residual;  // may be null
  void* residual_out;    // may be null
  int residual_type;
  const void* weight;
  int weight_type;
  float eps;
  int8_t* q;       // may be null
  float* x_scale;  // with q
  uint16_t* y;     // may be null
  int T, K;
};
cudaError_t launch_add_rmsnorm_s8(const NormArgs& a, cudaStream_t stream);

// The int8 cache (see tern_kv8_cache) and one call's rows.
struct Kv8Args {
  int8_t* codes;
  float* scales;
  const int* table;
  const int* lens;
  const int* starts;
  int pages, seqs, width, hkv, dim;
  int type;           // of q, or of k and v
  long long ld, hd;   // row and head strides in elements
  int rows, max_new;
  // append
  const void *k, *v;
  // attention
  const void* q;
  int heads, group;  // query heads; query heads per key-value head
  unsigned group_mul, group_shift;
  int window, sinks;
  float scale_log2;  // softmax scale * log2(e)
  void* out;
  float* lse;
  int* tickets;
  float* partials;
  int* err;
};
// n / group = (high half of n * mul + n) >> shift for n < 2^31: with shift =
// ceil(log2 group), mul = floor(2^32 (2^shift - group) / group) + 1.
inline void kv8_set_group(Kv8Args* a, int group) {
  a->group = group;
  a->group_shift = 0;
  while ((1u << a->group_shift) < static_cast<unsigned>(group)) ++a->group_shift;
  a->group_mul = static_cast<unsigned>(((1ull << 32) * ((1ull << a->group_shift) - group)) / group +
                                       1);
}
cudaError_t launch_kv8_append(const Kv8Args& a, cudaStream_t stream, int* launches);

// Attention of sequences with few query rows per key-value head (new tokens *
// group), at most max_rows; the others are left to the prompt kernel.  tm: the
// codes as bytes [pages * 2 * hkv * 64][dim], box dim x kKvRowsBox rows,
// swizzle of the row's width.
constexpr int kKvRowsBox = 32;
// Query rows per key-value head (new tokens times group) up to which a
// sequence takes the few-row kernel.  Measured, that kernel and the one on the
// tensor cores: 9.3 and 16.6 us (one token over 777, 6 rows), 181 and 630 us
// (32 single tokens, 544000 cached).
constexpr int kKvFewRows = 16;
// The same where no sequence has more and each SM gets at least kKvLongPages
// pages: its three tiles of eight rows.  At 24 rows of 4 sequences: 71 and 90
// us (105 pages an SM), 48 and 53 (53), 36.6 and 34.6 (26); at 20 rows under a
// window 36.9 and 34.9 (28).  (With longer sequences in the batch the single
// tokens among them would pay for the third tile.)
constexpr int kKvFewRowsLong = 24, kKvLongPages = 40;
constexpr int kKvSeqsPerLaunch = 128;  // sequences of one launch
size_t kv8_rows_partial_bytes(int dim);
cudaError_t kv8_rows_set_attributes();
cudaError_t launch_kv8_rows(const CUtensorMap* tm, const Kv8Args& a, int max_rows, int num_sms,
                            cudaStream_t stream, int* launches);

// Attention of sequences with at least min_rows query rows per key-value
// head, on the tensor cores.  tickets: kSmallTMaxCtas zeroed ints.
size_t kv8_prompt_partial_bytes(int dim);
cudaError_t kv8_prompt_set_attributes();
// Whether the kernel's grid holds the blocks of rows of such a call.
bool kv8_prompt_fits(int max_new, int group, int kv_heads, int seqs);
cudaError_t launch_kv8_prompt(const Kv8Args& a, int min_rows, float* partials, int* tickets,
                              int num_sms, cudaStream_t stream, int* launches);

// Diagnostic: one kernel whose bounded wait runs out (which = 0: an mbarrier
// phase nobody completes; 1: a device counter nobody raises) and records the
// timeout in *err.
cudaError_t launch_wait_timeout_probe(int which, int* err, cudaStream_t stream);

}  // namespace tern
