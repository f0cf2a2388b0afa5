/*
 * tern.h — C ABI of the ternary-weight linear layer for one GB300 (sm_103a).
 *
 * The layer computes y = x W^T for ternary weights W in {-1, 0, +1} with one
 * fp16 scale per 128 consecutive weights along K, for T tokens of bf16
 * activations.  Three token bands, each served by its own kernel ("rung"):
 *   T = 1        decode GEMV                           rung "gemv"
 *   T = 2..8     speculative-verify small-T tile       rung "small_t"
 *   T = 9..16    two small-T token tiles per weight    rung "small_t_tiled"
 *   T >= 17      int8 per-token activations ("s8")     rung "s8"
 * The band map, the env override and the per-rung probe follow the rung map
 * and the probe discipline of the "ninfer-perf-tuning" skill page, section 2
 * ("which rung ran" and its rung-map table); the format follows the "NInfer
 * sm_89 fork" write-up, section 9 item 2 (ternary codes plus one FP16 scale
 * per 128 weights; int8 activations with m16n8k32 int8 MMA for prefill).
 *
 * Conventions for every entry point
 *  - All array arguments are DEVICE pointers of the current CUDA device, owned
 *    by the caller.  The library never allocates or frees device memory.
 *  - `stream` is a cudaStream_t (passed as void*; NULL = legacy default
 *    stream).  Calls are asynchronous on that stream and never synchronise.
 *  - Row-major, densely packed layouts; element types are given as bit
 *    patterns so that this header needs no CUDA headers:
 *      bf16 = uint16_t (upper half of an IEEE fp32), fp16 = uint16_t (IEEE
 *      binary16), fp32 = float.
 *  - Every pointer must be 16-byte aligned (TERN_EALIGN otherwise).
 *  - Errors are returned as a negative tern_status; nothing aborts.  Launch
 *    failures return TERN_ECUDA.  Asynchronous device-side failures (a bounded
 *    wait that ran out) are recorded in a per-device error word read by
 *    tern_device_status().
 *
 * Packed weight layout (this library's format; the pages pack base-3 trits
 * five to a byte, this format spends 2 bits per weight on sign and magnitude):
 *   Wpacked is uint32 [N][K/16], i.e. K/4 bytes per row.  Byte b of row n
 *   (little-endian bytes within the words) holds weights k = 4b .. 4b+3.
 *   Weight i of a byte has its "nonzero" bit at bit P[i] and its "negative"
 *   bit at bit P[i] + 2, with P = {0, 1, 4, 5}; each nibble thus reads
 *   [nz_lo, nz_hi, neg_lo, neg_hi] from bit 0 up:
 *       (nz, neg) = (0, 0) -> 0,  (1, 0) -> +1,  (1, 1) -> -1,  (0, 1) invalid.
 *   tern_pack never writes the invalid pair; the linear kernels decode it as 0.
 *   The bit order lets the kernels turn a byte into the fp8 e4m3 encoding of
 *   w/8 with one shift and one AND.
 * Scales: fp16 [N][K/128], scale (n, g) applies to k in [128g, 128g+128).
 *
 * Beside the layer, the operators that stand between two such layers of a
 * decoder: tern_add_rmsnorm_s8 (residual, norm and int8 codes),
 * tern_linear_s8 (the layer on such codes), tern_kv8_append and
 * tern_kv8_attention (a paged int8 cache of keys and values and the attention
 * that reads it).
 */
#ifndef TERN_H_
#define TERN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TERN_OK = 0,
  TERN_EINVAL = -1,   /* bad size / null pointer / unsupported shape */
  TERN_EALIGN = -2,   /* a pointer is not 16-byte aligned */
  TERN_ENOSPACE = -3, /* workspace smaller than tern_linear_workspace_bytes() */
  TERN_ENODEV = -4,   /* no usable sm_103 device current */
  TERN_ECUDA = -5,    /* a CUDA runtime call or launch failed */
  TERN_ETIMEOUT = -6, /* a device-side bounded wait ran out (see tern_device_status) */
  TERN_EINDEX = -7    /* a kernel met a page, length or row index out of range and
                         skipped it (see tern_device_status) */
} tern_status;

/* Element types of the operators that take more than one. */
typedef enum {
  TERN_F32 = 0,
  TERN_BF16 = 1,
  TERN_F16 = 2
} tern_type;

/* Rung identifiers (tern_select_rung / tern_last_rung_id). */
typedef enum {
  TERN_RUNG_GEMV = 0,
  TERN_RUNG_SMALL_T = 1,
  TERN_RUNG_SMALL_T_TILED = 2,
  TERN_RUNG_S8 = 3,
  TERN_RUNG_BF16 = 4  /* exact bf16 prefill rung; chosen by TERN_RUNG=bf16 or,
                         for T >= TERN_S8_MIN_T, TERN_PREFILL=bf16 */
} tern_rung;

/* Pack ternary int8 weights into the 2-bit layout above.
 *   W        device int8 [N][K], values in {-1, 0, +1}
 *   Wpacked  device uint32 [N][K/16], written
 *   K, N     K > 0 and K % 16 == 0; N > 0
 *   bad_count optional device int32; if not NULL, the number of inputs outside
 *            {-1, 0, +1} is ADDED to *bad_count (those inputs are packed as 0).
 * Format: "NInfer sm_89 fork" write-up, section 9 item 2 (ternary codes with
 * per-128 fp16 scales), 2-bit reading of its base-3 digit. */
int tern_pack(const int8_t* W, uint32_t* Wpacked, int K, int N, int* bad_count,
              void* stream);

/* Per-token int8 quantisation of bf16 activations ("s8" rung input).
 *   x        device bf16 [T][K]
 *   q        device int8 [T][K], written: clamp(rint(x / x_scale), -127, 127),
 *            rint = round to nearest even
 *   x_scale  device fp32 [T], written: max_k |x[t][k]| / 127 (IEEE fp32
 *            division); a token whose absmax is 0 gets x_scale 0 and q 0.
 *   T > 0, K > 0, K % 16 == 0.
 * Source: int8 activations for the prefill rung, "NInfer sm_89 fork" write-up
 * section 9 item 2 and the "s8" rung of the "ninfer-perf-tuning" skill page
 * section 2; absmax/127 with round-to-nearest-even is the reading of
 * "quantised per token". */
int tern_quant_act_s8(const uint16_t* x, int8_t* q, float* x_scale, int T,
                      int K, void* stream);

/* Convert base-3 packed weights (five per byte) to the 2-bit layout above.
 *   Pt5      device uint8 [N][K/128][26], read-only.  Each 128-weight group
 *            takes 26 bytes; byte j of a group holds the group's weights
 *            5j .. 5j+4 as the base-3 number sum_i (w_i + 1) * 3^i, the first
 *            weight least significant.  The last byte holds three weights;
 *            its two upper digits are padding and are ignored.  Bytes above
 *            242 are invalid: their weights are written as 0.
 *   Wpacked  device uint32 [N][K/16], written
 *   K, N     K > 0 and K % 128 == 0; N > 0
 *   bad_count optional device int32; if not NULL, the number of invalid bytes
 *            is ADDED to *bad_count.
 * The scales keep their [N][K/128] fp16 array.  This is a one-time,
 * memory-bound conversion for weights stored in the base-3 format; the
 * linear kernels read the 2-bit layout.
 * Format: "NInfer sm_89 fork" write-up, section 9 item 2 (base-3 codes,
 * five weights per byte, one FP16 scale per 128 weights, 1.75 bits per
 * weight: 26 bytes + 2 bytes of scale per 128 weights). */
int tern_repack_t5(const uint8_t* Pt5, uint32_t* Wpacked, int K, int N,
                   int* bad_count, void* stream);

/* Blockwise Hadamard rotation of bf16 activations:
 *   xr[t][1024 b + i] = bf16( 1/32 * sum_j (-1)^popcount(i & j) x[t][1024 b + j] )
 * for each 1024-wide block b of each token t (the orthonormal Sylvester
 * Hadamard matrix of order 1024), computed in fp32 and rounded to bf16 with
 * round-to-nearest-even.  Each output differs from the exact rotation by at
 * most half a bf16 step plus the fp32 sum error bound
 * 10 * 2^-24 * sum_j |x[t][1024 b + j]| / 32, so it is the exact value's own
 * bf16 rounding except where that value lies within the sum bound of a
 * rounding boundary.
 *   x        device bf16 [T][K], read-only
 *   xr       device bf16 [T][K], written; may be x itself (in place),
 *            otherwise it must not overlap x
 *   T > 0, K > 0, K % 1024 == 0.
 * Source: the Hadamard rotation that the "NInfer sm_89 fork" write-up
 * (section 9 item 2) fuses into the activation quantisation, over the
 * (1024-block, token) pairs of the "ninfer-perf-tuning" skill page's
 * section 6 budget table. */
int tern_rotate_bf16(const uint16_t* x, uint16_t* xr, int T, int K,
                     void* stream);

/* Bytes of the synchronisation area at the start of every workspace. */
#define TERN_SYNC_BYTES 4096u

/* Bytes of device workspace tern_linear needs for (T, K, N); the value covers
 * every rung: the synchronisation area, then for the s8 rung the int8 codes
 * split into two fp8 pieces (2 T K bytes) and the token scales, or for the
 * small-T rungs the partial row sums of row blocks that two or more CTAs
 * share and the activation blocks built per call.
 * Host-only; 0 for T < 1 or K < 1. */
size_t tern_linear_workspace_bytes(int T, int K, int N);

/* y = x W^T with group scales:
 *   y[t][n] = sum_g s[n][g] * sum_{k in g} w[n][k] * x[t][k]
 * on the bf16-activation rungs (T <= 16), and on the s8 rung (T >= 17)
 *   q, xs = tern_quant_act_s8(x)
 *   acc[t][n][g] = sum_{k in g} q[t][k] * w[n][k]   (exact integers)
 *   y[t][n]      = xs[t] * sum_g s[n][g] * acc[t][n][g]   (fp32).
 * Precision of the bf16 rungs, for every finite input: each bf16 x is cut
 * into three fp8 e5m2 pieces at a power-of-two scale per token and
 * 128-group, exactly for every element within 21 binades of the group's
 * largest, so those products w * x are formed exactly on the tensor cores.
 * The few elements further down (leftovers) are handled per row block: if
 * the bound s * sum|x| of every leftover group of a row block adds up to at
 * most 2^-11 of the row block's partial sum, they are left out, otherwise
 * they are multiplied exactly on the CUDA cores.  Beside the fp32 sums'
 * rounding the error is therefore at most 2^-11 * sum|s w x|, inside
 * |y - y_exact| <= 1e-3 * sum|s w x| + 1e-6.  Row blocks that need their
 * leftovers added read them twice (extra time, same result).
 * Results are bit-for-bit reproducible from call to call on every rung: rows
 * whose sums several CTAs share are added in a fixed CTA order.
 *   Wpacked  device uint32 [N][K/16] (layout above), read-only
 *   scales   device fp16 [N][K/128], read-only
 *   x        device bf16 [T][K], read-only
 *   y        device fp32 [T][N], written (fully overwritten)
 *   T >= 1, K >= 128 with K % 128 == 0, N >= 1
 *   workspace, workspace_bytes: device scratch of at least
 *            tern_linear_workspace_bytes(T, K, N) bytes, 16-byte aligned
 *            (TERN_ENOSPACE if smaller).  Its first TERN_SYNC_BYTES bytes are
 *            a synchronisation area (ticket counters with which the CTAs of a
 *            launch agree which of them adds up the rows they share; no CTA
 *            ever waits for another) owned by the library: zero it once
 *            before the workspace's first use (e.g. with cudaMemset), then
 *            leave it alone; every call that completes without a device-side
 *            error leaves it zeroed again.  After TERN_ETIMEOUT from
 *            tern_device_status, zero it again.  The rest of the workspace is
 *            scratch whose contents on entry are ignored.  The workspace must
 *            not be used by anything else (nor by another tern_linear call)
 *            until the call's work on `stream` has finished.
 * The small-T kernels use programmatic dependent launch: a kernel may start
 * while the previous kernel on the stream finishes, and it then already
 * reads Wpacked and scales (never x) before that kernel has completed.  So
 * Wpacked and scales must not be written by a kernel that launches its
 * dependents early and may still be running; a kernel launched without
 * programmatic dependent launch (any other library's kernel, and this
 * library's tern_pack and tern_repack_t5) has completed before the next
 * kernel starts.
 * x, y and the workspace are touched only after the previous kernel has
 * completed.
 * With TERN_ROTATE=1 in the environment the layer runs on the blockwise
 * Hadamard rotation of x (the operation of tern_rotate_bf16: each 1024-wide
 * block of each token rotated and rounded once to bf16) instead of x itself,
 * for weights stored in the rotated basis.  Every rung rotates inside its own
 * activation staging (x is never written and no extra call is made); K must
 * then be a multiple of 1024 and at most 65536, else TERN_EINVAL.  The
 * rotation's fp32 sums may round an element the other way where its exact
 * value lies within tern_rotate_bf16's stated bound of a bf16 rounding
 * boundary; otherwise the result is that of tern_linear on tern_rotate_bf16's
 * output.  Source: the rotation the "NInfer sm_89 fork" write-up (section 9
 * item 2) fuses into the activation quantisation.
 * With TERN_DECODE_ACT=int8 the T <= 16 rungs compute the s8 definition
 * instead (per-token int8 codes as tern_quant_act_s8 makes them, exact
 * integer group sums, y = xs * sum_g s * acc, held to the s8 rung's bars):
 * the int8-activation decode path of the "NInfer sm_89 fork" write-up
 * (section 9 item 2).  It has no rotated form (TERN_ROTATE with it:
 * TERN_EINVAL on those rungs).
 * The bf16 rung (TERN_RUNG=bf16, or TERN_PREFILL=bf16 for the s8 band)
 * computes the bf16-rung definition above on tcgen05 kind::f16: weights as
 * bf16 +-1, activations as they are, every product exact, fp32 sums; no
 * activation quantisation (its workspace holds x reordered for the MMA).
 * The rung is chosen from T (see tern_select_rung); TERN_RUNG forces one.
 * Every rung is correct for every T. */
int tern_linear(const uint32_t* Wpacked, const uint16_t* scales,
                const uint16_t* x, float* y, int T, int K, int N,
                void* workspace, size_t workspace_bytes, void* stream);

/* The layer on int8 codes and token scales that the caller already has
 * (tern_quant_act_s8's or tern_add_rmsnorm_s8's):
 *   acc[t][n][g] = sum_{k in g} q[t][k] * w[n][k]   (exact integers)
 *   y[t][n]      = x_scale[t] * sum_g s[n][g] * acc[t][n][g]   (fp32),
 * the s8 definition at every T, without quantising again.  T <= 16 runs on
 * the small-T rungs' kernels, T >= 17 on the s8 rung's; TERN_RUNG forces a
 * rung as for tern_linear (bf16 has no such form: TERN_EINVAL).  Codes have no
 * rotated form either: with TERN_ROTATE, TERN_EINVAL.  TERN_PREFILL and
 * TERN_DECODE_ACT do not apply.
 *   q        device int8 [T][K], any value of -128..127
 *   x_scale  device fp32 [T]
 *   the others and the workspace as for tern_linear. */
int tern_linear_s8(const uint32_t* Wpacked, const uint16_t* scales,
                   const int8_t* q, const float* x_scale, float* y, int T,
                   int K, int N, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Residual addition, root-mean-square norm and int8 codes of token rows:
 *   r = x + residual, rounded to the residual's type (r = x without one)
 *   y = r * weight / sqrt(mean_k(r^2) + eps)             (fp32)
 *   x_scale[t] = max_k |y[t][k]| / 127                   (IEEE division)
 *   q[t][k]    = clamp(rint(y / x_scale), -127, 127), to nearest even;
 *                a token whose y is all zeros gets x_scale 0 and q 0.
 *   x        device [T][K] of x_type (TERN_F32, as tern_linear writes it, or
 *            TERN_BF16); row t starts at element t * x_ld (x_ld >= K, rows
 *            16-byte aligned)
 *   residual device [T][K] of residual_type (TERN_BF16 or TERN_F32), or NULL
 *   residual_out device [T][K] of residual_type, written with r; may be
 *            residual itself, may be NULL; NULL when residual is
 *   weight   device [K] of weight_type (TERN_BF16 or TERN_F32)
 *   q, x_scale device int8 [T][K] and fp32 [T], written; both or neither NULL
 *   y        device bf16 [T][K], written with y rounded once (what the
 *            bf16-activation rungs take), or NULL; q or y must be given
 *   T >= 1; K > 0, K % 16 == 0, K <= 32768; eps >= 0.
 * The statistics are fp32.  A row that holds an infinity or a NaN, in r or in
 * y, gives unspecified codes and a scale that is not finite or 0. */
int tern_add_rmsnorm_s8(const void* x, int x_type, long long x_ld,
                        const void* residual, void* residual_out,
                        int residual_type, const void* weight, int weight_type,
                        float eps, int8_t* q, float* x_scale, uint16_t* y,
                        int T, int K, void* stream);

/* ---------------------------------------------------------------- int8 cache
 * A paged cache of keys and values in int8.  A page holds TERN_KV8_BLOCK
 * tokens of one sequence, keys and values of every head, and is the block
 * that shares a scale: one fp32 scale for each (page, keys | values, head).
 *   codes   device int8 [pages][2][kv_heads][TERN_KV8_BLOCK][head_dim],
 *           keys at [0], values at [1] of the second index
 *   scales  device fp32 [pages][2][kv_heads], not negative (the append writes
 *           none that are; the attention reads a negative one as NaN); a stored
 *           value is scale * code
 *   page_table  device int32 [seqs][table_width]: page of tokens
 *           [64 j, 64 j + 64) of each sequence; entries past a sequence's
 *           last token are not read
 *   seq_lens    device int32 [seqs]: tokens of each sequence, the new ones
 *           included
 *   row_start   device int32 [seqs + 1], ascending: the new tokens of sequence
 *           b are rows [row_start[b], row_start[b + 1]) of q, k and v; they
 *           are its last tokens, in order
 * pages * 2 * kv_heads * 64, table_width * 64, table_width * kv_heads and
 * rows * heads / kv_heads have to fit in 31 bits (TERN_EINVAL).
 * Sequences may be empty and may have no new tokens.  These arrays are read
 * on the device, so a captured call can be replayed with other contents.  A
 * sequence whose entries are inconsistent (a length that is negative or does
 * not fit table_width, more new tokens than tokens or than max_new, rows
 * outside [0, rows)) is skipped and its rows of the output are left as they
 * are; a page outside [0, pages) is skipped, as if its tokens were masked;
 * both are recorded for tern_device_status (TERN_EINDEX).  */
#define TERN_KV8_BLOCK 64

typedef struct {
  int8_t* codes;
  float* scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* row_start;
  int pages, seqs, table_width;
  int kv_heads, head_dim; /* head_dim 64 or 128 */
} tern_kv8_cache;

/* Write the new keys and values of every sequence into the cache.  For each
 * page that receives new tokens, keys and values apart, and each head:
 *   s = max(s_old if the page holds older tokens, max |new| / 127)  (fp32,
 *       IEEE division);
 *   where s > s_old, the older tokens' codes become rint(code * (s_old / s));
 *   new codes are clamp(rint(x / s), -127, 127), rint to nearest even.
 * So a code is rounded once more at each growth: a token's error is at most half
 * the sum of the scales that its block has had since it was written.  For 64
 * normal tokens appended one by one (some 5 growths) the root mean square error
 * of the first sixteen is 1.6 times that of the same tokens appended together,
 * and 2.5 times where the magnitudes grow fourfold on the way (some 16).
 * Codes of the page's slots past the last token are left as they are; the
 * scale of a page without older tokens is overwritten whatever it held.  An
 * infinite or NaN input makes its block's scale NaN (the block's values then
 * read as NaN), and no other block's.
 *   k, v    device [rows][kv_heads][head_dim] of `type` (TERN_F32, TERN_BF16
 *           or TERN_F16); row r, head h start at element r * ld + h * hd
 *           (k and v have the same strides); every start 16-byte aligned
 *   rows    rows of k and v; 0: nothing is done
 *   max_new at least the most new tokens of a sequence, and at least 1 where
 *           there are rows (sizes the grid)
 * No two sequences of a call may share a page that receives new tokens. */
int tern_kv8_append(const tern_kv8_cache* cache, const void* k, const void* v,
                    int type, long long ld, long long hd, int rows,
                    int max_new, void* stream);

/* Bytes of device workspace tern_kv8_attention needs for `rows` query rows of
 * `seqs` sequences (the synchronisation area, then partial results of
 * sequences that several CTAs share).  Host-only; 0 for sizes out of range. */
size_t tern_kv8_attention_workspace_bytes(int seqs, int rows, int heads,
                                          int kv_heads, int head_dim);

/* Attention of the new tokens of every sequence over the cache (which must
 * already hold them).  Query row i of the m new rows of a sequence of n tokens
 * stands at position p = n - m + i and sees the tokens j <= p with, if window
 * > 0, j > p - window or j < sinks:
 *   o[row][h] = sum_j softmax_j(softmax_scale q[row][h] . k_j) v_j,
 * k_j and v_j the cache's scale * code of key-value head h / (heads /
 * kv_heads).  Codes and scales of blocks that a row does not see do not enter
 * its result, whatever they hold, nor do the codes of tokens that it does not
 * see in a block that it does.
 *   q       device [rows][heads][head_dim] of `type` (TERN_BF16 or TERN_F16);
 *           row r, head h start at element r * ld + h * hd, 16-byte aligned
 *   rows    rows of q; 0: nothing is done
 *   out     device [rows][heads][head_dim] of `type`, dense, written
 *   lse     device fp32 [rows][heads], written with log sum_j exp(s_j)
 *           (natural logarithm), or NULL
 *   heads   a multiple of kv_heads, at most 64 times as many
 *   max_new at least the most new tokens of a sequence, and at least 1 where
 *           there are rows; ceil(max_new * heads / kv_heads / 256) * kv_heads *
 *           seqs has to stay below 2^31 - 1000 (TERN_EINVAL).  It and
 *           table_width, which the launch knows alone, choose the kernels: a
 *           decode step whose max_new is the call's rows takes a launch more and
 *           wider tiles than one with max_new 1
 *   window  0 (none) or the tokens that a row sees, itself included
 *   sinks   first tokens that stay visible outside the window (>= 0)
 *   softmax_scale > 0, and times log2(e) a finite float
 *   workspace as for tern_linear: zero its first TERN_SYNC_BYTES once.
 * Numbers: q is scaled by a power of two per row and held in fp16 (a bf16 or
 * fp16 element is exact down to 2^-31 of the row's largest), codes are exact in
 * fp16, products and sums are fp32, some of them of code + 128 with the 128s
 * taken off the sum: the roundings of a score follow 128 k_scale sum |q|, and
 * those of an output 128 v_scale sum p, a few 2^-24 of them.  The weights are
 * rounded to fp16 for their products with the values (relative 2^-11, down to
 * 2^-24 of the row's largest weight, or weight times v_scale); their sum is fp32
 * and unrounded.  Value scales may lie any number of powers of two apart, which
 * costs time: more than 2^8 within a block of prompt rows, or out of 2^-38 to
 * 2^38.  Results are bit-for-bit reproducible. */
int tern_kv8_attention(const tern_kv8_cache* cache, const void* q, int type,
                       long long ld, long long hd, int rows, int heads,
                       int max_new, int window, int sinks, float softmax_scale,
                       void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Bytes of the fixed device scratch tern_linear_small_t_noalloc uses. */
#define TERN_NOALLOC_SCRATCH_BYTES (8u << 20)

/* tern_linear for T = 1..16 without a caller workspace and without allocating.
 *
 * The pages have no counterpart of this call; it exists for callers that
 * cannot allocate device memory or hand over a workspace: plug-in interfaces
 * that pass only input and output buffers, engines that reserve all device
 * memory at start-up and forbid allocation afterwards, and latency-critical
 * code where cudaMalloc / cudaFree would synchronise the device.
 *
 *   Wpacked, scales, x, y, T, K, N, stream: as for tern_linear.
 *   1 <= T <= 16 (TERN_EINVAL otherwise).  The rung comes from T alone:
 *   "gemv" at T = 1, "small_t" at T = 2..8, "small_t_tiled" at T = 9..16; the
 *   environment overrides of tern_linear do not apply.
 *
 * Scratch.  The call's workspace (the synchronisation area, partial sums and
 * activation blocks) lives in one file-scope device array of
 * TERN_NOALLOC_SCRATCH_BYTES (8 MiB) inside the library; every GPU that loads
 * the library holds it until the process exits.  A call whose workspace does
 * not fit returns TERN_ENOSPACE before any device work: K <= 479232 for
 * T = 1..4, K <= 219136 for T = 5..8 and K <= 118784 for T = 9..16.  The call
 * allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 * routine.
 *
 * Set-up.  The first call on a device (with that device current) looks up the
 * array's device address with cudaGetSymbolAddress and performs the library's
 * per-device set-up (kernel attributes); make that first call before any
 * stream capture.
 *
 * Sharing.  Every call on a device uses the same array, and the array keeps
 * the last call's contents.  The array is zero when the library loads; its
 * synchronisation area is left valid by every call that completes without a
 * device-side error, and every other byte a call reads it has written first,
 * so nothing needs clearing between calls.  When tern_device_status reports
 * TERN_ETIMEOUT it also zeroes the array's synchronisation area on that
 * device.  Calls whose work overlaps on the GPU (e.g. on two streams without
 * ordering between them) race on the array and give wrong results: order
 * them on one stream or with events. */
int tern_linear_small_t_noalloc(const uint32_t* Wpacked, const uint16_t* scales,
                                const uint16_t* x, float* y, int T, int K, int N,
                                void* stream);

/* Diagnostic of the failure path.  Launches one small kernel whose bounded
 * wait can never be satisfied, using the same wait code as the layer's
 * kernels:
 *   which = 0  an mbarrier phase that nothing completes
 *   which = 1  a device counter that nothing raises (a wait in global
 *              memory, the form a wait on another CTA would take)
 * After the wait limit (2 s) the kernel records the timeout in the device
 * error word and returns: nothing faults or hangs, and the context stays
 * usable.  tern_device_status() on the same stream then returns
 * TERN_ETIMEOUT and clears the word.  which outside {0, 1}: TERN_EINVAL.
 * For tests and health checks only; never needed on the layer's path. */
int tern_selftest_wait_timeout(int which, void* stream);

/* Rung the dispatcher picks for T (after env overrides).  Host-only. */
int tern_select_rung(int T);

/* Name of a rung id ("gemv", "small_t", "small_t_tiled", "s8", "bf16"), or "?". */
const char* tern_rung_name(int rung);

/* Rung launched by this thread's last successful tern_linear, or -1 / "none". */
int tern_last_rung_id(void);
const char* tern_last_rung(void);

/* Number of kernels this thread's last successful tern_linear,
 * tern_linear_s8, tern_linear_small_t_noalloc, tern_add_rmsnorm_s8,
 * tern_kv8_append or tern_kv8_attention launched: per token tile of the bandwidth
 * rungs one main kernel, plus the activation-prep kernel where the tile
 * uses one; 2 on the s8 rung (activation pieces, then the GEMM).  0 before
 * any call.  Host-only; for benchmarks and tests. */
int tern_last_launches(void);

/* Static text for a tern_status. */
const char* tern_status_string(int status);

/* Re-read the environment (TERN_RUNG, TERN_SMALL_T_MAX, TERN_TILED_MAX,
 * TERN_S8_MIN_T, TERN_PREFILL, TERN_ROTATE, TERN_DECODE_ACT, TERN_DEBUG,
 * TERN_DEBUG_MIN_T, TERN_DEBUG_BUDGET).  The
 * environment is otherwise read once per process, on first use. */
void tern_reload_env(void);

/* Synchronises `stream`, then returns and clears the current device's
 * asynchronous error word: TERN_OK, or TERN_ETIMEOUT if a kernel's bounded
 * wait ran out since the last call (in which case it also zeroes the
 * synchronisation area of tern_linear_small_t_noalloc's scratch, if that
 * scratch is set up on this device), or TERN_EINDEX if a cache kernel skipped
 * an index that was out of range. */
int tern_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TERN_H_ */
