/*
 * sage_sparse.h -- block-sparse attention for video diffusion transformers and
 * the steps before it, in the library of sage.h (same conventions, status codes
 * and modes):
 *   sage_qk_norm_rope      the projections' q and k -> normalised and rotated,
 *                          in the layouts the attention calls read;
 *   sage_select_blocks     the key blocks each query block attends to, by the
 *                          scores of pooled queries and keys;
 *   sage_attn_fwd_sparse   attention over those blocks, in every mode of
 *                          sage_attn_fwd.
 * Block-sparse attention is named as an acceleration of video DiTs by the
 * overview at cloud.baidu.com/article/9430832; the scheme here is this
 * library's.  All calls are asynchronous on `stream`, allocate nothing, keep
 * nothing between calls and can be captured into a CUDA graph after one eager
 * call per device.  Forward only.
 */
#ifndef SAGE_SPARSE_H
#define SAGE_SPARSE_H

#include "sage.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm of queries and keys and the position rotation, one pass over the data.
 *
 * q, k      bf16, token n of batch b at (b * N + n) * stride elements, its H * d
 *           channels contiguous (heads in order); q_stride, k_stride >= H * d and
 *           multiples of 8, so slices of one fused projection are read in place.
 *           One of q and k may be NULL (with its output): cross attention
 *           rotates them apart.
 * norm      SAGE_NORM_NONE   y = x
 *           SAGE_NORM_RMS    y = x / sqrt(mean(x^2) + eps) * w
 *           SAGE_NORM_LAYER  y = (x - mean) / sqrt(mean((x - mean)^2) + eps) * w + b
 *           A vector whose mean square plus eps is 0 gives 0 before b.
 * scope     SAGE_NORM_SCOPE_HEAD: over the d channels of each head, w and b [d];
 *           SAGE_NORM_SCOPE_ALL: over the token's H * d channels, w and b [H * d].
 * wq, bq, wk, bk  weights, w_dtype SAGE_DTYPE_BF16 or SAGE_DTYPE_F32, 16-byte
 *           aligned; NULL means 1 and 0.  Must be NULL for SAGE_NORM_NONE; b must
 *           be NULL for SAGE_NORM_RMS.
 * eps       finite, >= 0.
 * rope      SAGE_ROPE_NONE, SAGE_ROPE_INTERLEAVED (pairs of channels 2i, 2i + 1)
 *           or SAGE_ROPE_HALF (pairs i, i + d/2):
 *             (a, b) -> (a cos - b sin, a sin + b cos), cos and sin from row
 *           n - rope_begin, column i of
 * cos, sin  device fp32 [rope_len, d/2], 16-byte aligned (NULL without rope).
 *           Tokens outside [rope_begin, rope_begin + rope_len) are normalised
 *           only (text tokens, padding); the range must lie within [0, N].
 * q_out, k_out  bf16.  out_ranks 0: [B, H, N, d], as sage_attn_fwd reads it.
 *           out_ranks P >= 1: [P][B][N][H/P][d], the send layout of the Ulysses
 *           exchange for this rank's N tokens (sage_ulysses_permute,
 *           SAGE_ULYSSES_SEND); P must divide H.  P = 1 is [B, N, H, d].
 *           An output must not overlap an input or the other output, except
 *           q_out == q (k_out == k) with out_ranks 1 and stride H * d: in place.
 *
 * Arithmetic in fp32, one rounding to bf16.  d 64 or 128, H * d <= 16384, B <=
 * 65535, B * N < 2^31.  Errors: SAGE_EINVAL (sizes, strides, pointers, overlap,
 * arguments that do not belong together), SAGE_EUNSUPPORTED (d, H * d, device).
 */
#define SAGE_NORM_NONE 0
#define SAGE_NORM_RMS 1
#define SAGE_NORM_LAYER 2
#define SAGE_NORM_SCOPE_HEAD 0
#define SAGE_NORM_SCOPE_ALL 1
#define SAGE_ROPE_NONE 0
#define SAGE_ROPE_INTERLEAVED 1
#define SAGE_ROPE_HALF 2
#define SAGE_NORM_MAX_WIDTH 16384
int sage_qk_norm_rope(const void* q, const void* k, long long q_stride, long long k_stride, const void* wq,
                      const void* bq, const void* wk, const void* bk, int w_dtype, const float* cos,
                      const float* sin, int B, int N, int H, int d, int norm, int scope, double eps, int rope,
                      int rope_begin, int rope_len, void* q_out, void* k_out, int out_ranks, void* stream);

/*
 * The key blocks of every 128-token query block, by a cheap score.  With
 * nT = ceil(N/128) and blocks of 128 tokens (the last one of the real rows only):
 *   qbar[i], kbar[j] = the mean of a block's rows, summed in fp64 (rows r, r + 8, r + 16, ..
 *                      for each r < 8, then the eight sums; exact, whatever the order, where a
 *                      channel's nonzero values lie within a factor of 2^38), rounded to fp32;
 *   s[i][j] = sum over the d channels of qbar[i] * kbar[j], in fp64.
 * Row i keeps the min(keep, nT) blocks of largest s, ties to the lower index;
 * the blocks j < first and those with |i - j| <= window rank above all others
 * (window -1: none), and first + 2 * window + 1 must not exceed keep unless
 * keep >= nT.  A score that is not a number ranks last.
 *
 * q, k      bf16 [B, H, N, d]
 * lists     int32 [B, H, nT, keep]: the kept blocks in ascending order, -1 behind
 * counts    int32 [B, H, nT]: how many
 * scratch   at least sage_select_scratch_bytes(B, H, N, d) bytes, 16-byte
 *           aligned.  Calls that overlap on the GPU need a scratch each.
 * lists, counts and scratch must not overlap each other or q and k.
 * nT at most SAGE_SELECT_MAX_BLOCKS (a row of scores stays in shared memory);
 * more is SAGE_EUNSUPPORTED (sage_select_scratch_bytes: 0).  Errors otherwise as
 * sage_quantize_qk.
 */
#define SAGE_SELECT_MAX_BLOCKS 6016
size_t sage_select_scratch_bytes(int B, int H, int N, int d);
int sage_select_blocks(const void* q, const void* k, int B, int H, int N, int d, int keep, int first, int window,
                       int32_t* lists, int32_t* counts, void* scratch, size_t scratch_bytes, void* stream);

/*
 * O_i = softmax(Q_i K_L^T / sqrt(d)) V_L for every 128-row query block i, L the
 * keys of the blocks lists[b][h][i][0 .. counts[b][h][i] - 1], walked in that
 * order; an empty list gives rows of 0.  A block listed twice counts twice.
 * mode as in sage_attn_fwd; in the INT8/FP8 modes the statistics of the prepass
 * (the K mean, the V scales) are those of the whole sequence.  A list of all
 * blocks in ascending order gives the bits of sage_attn_fwd (with
 * SAGE_COEFF_DIVIDE).
 *
 * q, k, v, o  bf16 [B, H, N, d]; o and the workspace must not overlap each other
 *           or the other buffers
 * lists     int32 [B, H, nT, width], width >= 1 (sage_select_blocks' keep, or any)
 * counts    int32 [B, H, nT], 0 .. width
 * coeff     how the INT8/FP8 modes round the quantization coefficients scale =
 *           amax / top and top / amax (top 127 or 448).  SAGE_COEFF_DIVIDE: correctly
 *           rounded divisions, the codes of sage_quantize_qk.
 *           SAGE_COEFF_RECIPROCAL: amax * fl(1 / top) and fl(1 / amax) * top, the
 *           codes that a torch program gets on the GPU from amax / 127.0 and
 *           127.0 / amax (a division by a number, or of one, is a product with a
 *           rounded reciprocal there); a code at a rounding border may differ.
 * workspace as in sage_attn_fwd (sage_workspace_bytes, 256-byte aligned, zero
 *           status word before the first call).  In every mode calls that overlap
 *           on the GPU need a workspace each, and so do graphs that are replayed
 *           at once: the counter that hands out the work lies in it.
 * The lists are read on the device: an index outside [0, nT) adds nothing,
 * whatever the tensors hold, a count outside [0, width] is clamped, and
 * sage_status() on the workspace then returns SAGE_EINVAL.
 */
#define SAGE_COEFF_DIVIDE 0
#define SAGE_COEFF_RECIPROCAL 1
int sage_attn_fwd_sparse(const void* q, const void* k, const void* v, void* o, int B, int H, int N, int d, int mode,
                         const int32_t* lists, const int32_t* counts, int width, int coeff, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Test hook of the bounded waits: sage_attn_fwd_sparse with a wait that no one
 * satisfies and a limit of `timeout_cycles` SM clocks, so that the kernel
 * records SAGE_ETIMEOUT in the workspace's status word and returns.
 */
int sage_dbg_sparse_forced_timeout(const void* q, const void* k, const void* v, void* o, int B, int H, int N, int d,
                                   int mode, const int32_t* lists, const int32_t* counts, int width, int coeff,
                                   void* workspace, size_t workspace_bytes, long long timeout_cycles, void* stream);

#ifdef __cplusplus
}
#endif

#endif
