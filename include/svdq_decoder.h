/*
 * svdq_decoder.h — C ABI of what a decoding step needs between its projections, on MI355X
 * (gfx950), exported by libsvdq.so beside the functions of svdq.h and svdq_serve.h: the
 * root-mean-square norm with the residual's addition, to 16 bits or to 8 with a scale for each
 * row; the product of 8-bit integers with scales for each row and column, for any number of rows;
 * rotary positions; and sampling from logits with given random numbers.
 *
 * svdq.h's activations are quantized in groups of 64 with a low-rank branch beside them, for 4-bit
 * weights.  Layers that are kept at 8 bits on both sides (W8A8, SmoothQuant's setting in DCMP's
 * list of methods) need no branch and one scale per row, which the norm before them computes on
 * the way; q and k are rotated by the positions that kv_block_plan wrote before kv_block_append and
 * kv_block_attention; the tokens drawn from the vocabulary projection's logits are what the next
 * kv_block_plan is called for.
 *
 * The conventions are those of svdq_serve.h: device pointers owned by the caller, synchronous
 * validation with nothing launched on error, the status codes, svdq_last_error, asynchronous work
 * on `stream` that can be captured into a graph.  A dtype argument is SVDQ_OUT_BF16 or
 * SVDQ_OUT_FP32 (enum svdq_out_dtype).
 */
#ifndef SVDQ_DECODER_H
#define SVDQ_DECODER_H

#include <stddef.h>
#include <stdint.h>

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_DECODER_VERSION 1

/* SVDQ_DECODER_VERSION of the built library. */
int svdq_decoder_version(void);

/*
 * svdq_rms_norm — h = fl32(x + residual), residual_out = h rounded to its dtype,
 *     y = h / sqrt(mean(h^2) + eps) gamma,
 * rounded to bf16, or to 8 bits with a scale for each row:
 *     s = fl32(max |y| / 127),  c = clamp(rne(fl32(y / s)), -127, 127), 0 where s = 0.
 * y is computed in fp32 from h before residual_out's rounding; a row's sum of squares neither
 * overflows nor vanishes, whatever its magnitude; a row of zeros gives zeros.  A row with a NaN or
 * an infinity has the scale NaN (infinity / infinity) and the codes 0; other rows are not touched
 * by it.  (h gamma is rounded to fp32 before it is divided; where that leaves fp32's range for all of a row, the row
 * is scaled by a power of two first.)
 *   x          [M, K] of x_dtype, 16B, rows x_stride elements apart (a multiple of 8, from K to 2^31)
 *   residual   [M, K] of residual_dtype (16B), or NULL: h = x.  residual_out likewise, or NULL
 *              where it is not needed; it may be residual itself, and is NULL without a residual
 *   gamma      fp32 [K] 16B, or NULL for ones;  0 <= eps <= 3e38
 *   y          bf16 [M, K] 16B;  codes  int8 [M, K] 16B, scales  fp32 [M]: y or NULL, codes and
 *              scales or both NULL, at least one of the two
 *   0 <= M <= 2^24, 8 <= K <= 2^20, K % 8 == 0.  Nothing else overlaps.
 */
int svdq_rms_norm(const void* x, int x_dtype, int64_t x_stride, const void* residual,
                  int residual_dtype, void* residual_out, const float* gamma, int M, int K,
                  float eps, uint16_t* y, int8_t* codes, float* scales, void* stream);

/*
 * svdq_quantize_rows — the 8 bits of svdq_rms_norm without the norm: y = fl32(x factor) (x where
 * factor is NULL).  For activations that no norm precedes, and for weights [N, K], whose rows are
 * the columns of the product.  A row with a NaN has the scale NaN, one with an infinity the scale
 * infinity, and the codes 0.
 *   x as for svdq_rms_norm;  factor  fp32 [K] 16B or NULL;  codes, scales as there
 */
int svdq_quantize_rows(const void* x, int x_dtype, int64_t x_stride, const float* factor, int M,
                       int K, int8_t* codes, float* scales, void* stream);

/*
 * svdq_pack_w8a8 — relayout of a weight's codes for svdq_w8a8_gemm (offline; the codes need not be
 * kept).  Unit (t, u) of 1024 bytes, at (t K / 64 + u) * 1024, holds columns 16 t .. + 15 at
 * k = 64 u .. + 63 as 64 pieces of 16 bytes: piece l has column 16 t + l % 16 and
 * k = 64 u + 16 (l / 16) .. + 15.  Columns past N are 0.
 *   codes      int8 [N, K] 16B;  container  int8 [svdq_w8a8_container_bytes(N, K)] 16B
 *   1 <= N <= 2^24, K % 64 == 0, 64 <= K <= 64 * 2047 (the size is 0 outside these limits)
 */
size_t svdq_w8a8_container_bytes(int N, int K);
int svdq_pack_w8a8(const int8_t* codes, int N, int K, int8_t* container, void* stream);

/*
 * svdq_w8a8_gemm — Y[m, n] = sx[m] sw[n] sum_k qx[m, k] qw[n, k] + bias[n].
 * The sum is exact (int32: |codes| <= 128 and K < 2^17), and so does not depend on how it is
 * divided; it is rounded to fp32, multiplied by sx and then by sw in fp32, the bias is added, and
 * the result is rounded to Y's dtype.  A row whose sx is NaN (or infinite with a sum of 0) is NaN.
 *   qx         int8 [M, K] 16B;  sx  fp32 [M]
 *   container  as written by svdq_pack_w8a8 16B;  sw  fp32 [N]
 *   bias       bf16 [N] or NULL;  Y  [M, N], bf16 or fp32 by out_dtype, 16B
 *   workspace  device scratch of svdq_w8a8_workspace_bytes(M, N, K) bytes (16B; may be NULL when
 *              that is 0), no initialization needed, rewritten by every call; calls that share one
 *              workspace must not overlap in time
 *   0 <= M <= 2^24, N and K as svdq_pack_w8a8, M N <= 2^40.
 */
size_t svdq_w8a8_workspace_bytes(int M, int N, int K);
int svdq_w8a8_gemm(const int8_t* qx, const float* sx, const int8_t* container, const float* sw,
                   const uint16_t* bias, int M, int N, int K, void* Y, int out_dtype,
                   void* workspace, void* stream);

/*
 * svdq_rope — rotary positions on the first rot_dim channels of every head of q and k: the pairs
 * (a, b) of channels i and i + rot_dim / 2, or 2 i and 2 i + 1 where `interleaved`, become
 *     scale (a cos t - b sin t),  scale (a sin t + b cos t),  t = positions[row] freqs[i];
 * channels from rot_dim on are copied.  t is formed and reduced in fp64, off by at most |t| 2^-51,
 * so a far position is as exact as a near one; sines, cosines and products are in fp32, rounded once
 * to bf16.
 *   q       [rows, heads, dim] of x_dtype, rows q_stride elements apart; k likewise with kv_heads
 *           (slices of a fused projection need no copy); kv_heads may be 0 with k and k_out NULL
 *   q_out, k_out  bf16, rows q_out_stride and k_out_stride elements apart; either may be its input
 *           where x_dtype is SVDQ_OUT_BF16 and the strides agree, otherwise they do not overlap it
 *   positions  int32 [rows] (as written by kv_block_plan);  freqs  fp64 [rot_dim / 2], in radians
 *           per position, finite
 *   scale   at most 3e38 either way; 1, or the factor of a scheme for long contexts
 *   rows >= 0, heads >= 1, kv_heads >= 0, (heads + kv_heads) rows <= 2^27, heads and kv_heads
 *   <= 65535; dim % 8 == 0, dim <= 1024; rot_dim % 16 == 0, 16 <= rot_dim <= dim; strides a multiple
 *   of 8, from heads * dim to 2^31; all pointers but positions 16B.
 */
int svdq_rope(const void* q, int64_t q_stride, int heads, const void* k, int64_t k_stride,
              int kv_heads, int x_dtype, int rows, int dim, int rot_dim, int interleaved,
              const int32_t* positions, const double* freqs, float scale, uint16_t* q_out,
              int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride, void* stream);

/*
 * svdq_sample — one token per row of logits, from one given random number per row.  With
 * zmax the row's largest logit, the weights are whole numbers,
 *     w_i = rne(2^40 exp((z_i - zmax) / temperature))   (in fp64: 2^-41 of the largest rounds to 0),
 * so that their sums are exact and the result does not depend on the order of adding.  In the order
 * of falling logits (the lower index first among equal ones)
 *     top_k > 0:  the first top_k stay (all where top_k <= 0);
 *     top_p < 1:  of these, those before which less than fl64(top_p * their sum) stands, and the first;
 *     min_p > 0:  of these, those with w_i >= min(min_p, 1) 2^40.
 * The token is the first, in the vocabulary's order, up to and with which more than
 * min(floor(fl64(W u)), W - 1) of the remaining sum W stands; share is w / W.  A temperature that
 * is not > 0 means the largest logit (the first of equal ones), with the share 1.
 * Logits of -infinity are never drawn; where the largest is +infinity, only such logits are.  A row
 * with a NaN, or with nothing above -infinity, gets the token -1 and the share 0.
 *   logits       [rows, vocab] of logits_dtype, rows logits_stride elements apart (from vocab to 2^31),
 *                aligned to an element
 *   temperature  fp32 [rows];  uniform  fp32 [rows], in [0, 1) (clamped to it; NaN counts as 0)
 *   top_k        int32 [rows] or NULL;  top_p, min_p  fp32 [rows] or NULL (NaN: no limit)
 *   tokens       int32 [rows];  share  fp32 [rows] or NULL
 *   workspace    device scratch of svdq_sample_workspace_bytes(rows, vocab) bytes (16B), no
 *                initialization needed, rewritten by every call; calls that share one workspace
 *                must not overlap in time
 *   0 <= rows <= 65535, 1 <= vocab <= 2^22.
 * Over a vocabulary of more than 2048, some rows are searched by one workgroup, which takes 6 to 20 times
 * as long (64 rows of 131072: 126 - 467 us instead of 15 - 47):
 *   - a top-k of more than 512, or of more than the row has parts (512 at most, of neighbouring logits) with
 *     anything above -infinity in them: a mask that leaves fewer than top_k tokens is such a row;
 *   - a limit that falls among thousands of equal logits;
 *   - a top-p, without a top-k, with more than 4096 logits (2048 in a chunk of the row) in the bin that its
 *     limit falls into.  A bin is 1/72 of the temperature wide: flat rows at high temperatures have such bins.
 */
size_t svdq_sample_workspace_bytes(int rows, int vocab);
int svdq_sample(const void* logits, int logits_dtype, int64_t logits_stride, int rows, int vocab,
                const float* temperature, const float* uniform, const int32_t* top_k,
                const float* top_p, const float* min_p, int32_t* tokens, float* share,
                void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_DECODER_H */
