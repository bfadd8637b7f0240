/*
 * svdq_serve.h — C ABI of the decoding step on MI355X (gfx950), exported by libsvdq.so beside
 * the functions of svdq.h: the SVDQuant linear layer on few rows with 16-bit activations, and a
 * paged KV cache held in 8 bits with a scale for each block of tokens and head (its block tables
 * and slot maps, the append, the read-back and the attention over it).
 *
 * svdq.h's per-channel INT8 cache takes its statistics over every token of the call, so it cannot
 * take one more token, and its attention reads one dense sequence.  Here a block of tokens of one
 * head has its own scale, so tokens are appended as they come (VARC "INT8 KV cache quantization":
 * the cache is the memory of autoregressive decoding), and a batch of ragged requests shares one
 * pool of blocks.
 *
 * The conventions are those of svdq.h (device pointers owned by the caller, synchronous
 * validation with nothing launched on error, the status codes, svdq_last_error, asynchronous
 * work on `stream`), with these additions:
 *   - A block size bs is 16, 32, 64 or 128 tokens; dim is 64 or 128.
 *   - The cache of `num_blocks` blocks is four arrays:
 *       k_codes  uint8 [num_blocks, kv_heads, bs, dim]     code c + 128, c in [-127, 127]  16B
 *       v_codes  uint8 [num_blocks, kv_heads, dim, bs]     (channels before tokens)        16B
 *       k_scale  fp32 [num_blocks, kv_heads];  v_scale likewise      value = c * scale
 *     Blocks need no initialization before their first append.
 *   - A slot is block * bs + offset (int64); a slot outside [0, num_blocks * bs) marks a row
 *     without a token, which is skipped.
 *   - Values on the device (lengths, tables, slots) cannot be validated before the launch; the
 *     kernels keep every access inside the arrays whatever these hold.
 */
#ifndef SVDQ_SERVE_H
#define SVDQ_SERVE_H

#include <stddef.h>
#include <stdint.h>

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_SERVE_VERSION 1

/* SVDQ_SERVE_VERSION of the built library. */
int svdq_serve_version(void);

/*
 * svdq_pack_w4a16 — relayout of svdq_pack_weights' INT4 codes and scales for svdq_w4a16_gemv
 * (offline weight preparation; the codes and scales are copied, not rounded, and wq need not be
 * kept).  Unit (t, s) of the container, at (t ceil(K / 512) + s) * 4352 bytes, holds columns
 * 16 t .. + 15 and the 64-groups g = 8 s .. + 7: for each pair of groups 64 lanes of 16 bytes
 * (lane l: column 16 t + l % 16, the 8 bytes of wq with k = 64 g + 16 (l / 16) .. + 15 of the even,
 * then of the odd group), then the scales fp16 [16 columns][8 groups]; what lies past N or K is 0.
 *   wq         uint8 [N, K/2] (16B), w_scales  fp16 [K/64, N], as written by svdq_pack_weights
 *   container  uint8 [svdq_w4a16_container_bytes(N, K)]  16B
 *   1 <= N <= 2^24, K % 64 == 0, 64 <= K <= 64 * 65535 (the size is 0 outside these limits).
 */
size_t svdq_w4a16_container_bytes(int N, int K);
int svdq_pack_w4a16(const uint8_t* wq, const uint16_t* w_scales, int N, int K, uint8_t* container,
                    void* stream);

/*
 * svdq_w4a16_gemv — the linear layer on few rows (decoding: 1 to 64 tokens), with the INT4
 * weights of svdq_pack_weights and the activations kept at 16 bits (no activation codes), in
 * fp32:
 *     X^ = fl32(X * inv_lambda),  T = X^ L1,
 *     Y[m, n] = sum_g s_w[g, n] sum_{k in g} X^[m, k] qw[n, k] + (T L2)[m, n] + bias[n].
 *   X           bf16 [M, K]  16B;  inv_lambda  fp32 [K]  16B
 *   L1p         bf16 [r, K] (16B), L2p  bf16 [N, r] (16B), as for svdq_quantize_act and
 *               svdq_w4a4_gemm; may be NULL when r == 0
 *   container   as written by svdq_pack_w4a16  16B
 *   bias        bf16 [N] or NULL
 *   Y           [M, N], bf16 or fp32 by out_dtype (enum svdq_out_dtype)
 *   workspace   device scratch of svdq_w4a16_workspace_bytes(M, N, K, r, out_dtype) bytes (16B),
 *               no initialization needed, rewritten by every call; calls that share one
 *               workspace must not overlap in time
 *   0 <= M <= 64 (more rows: svdq_w4a4_gemm), 1 <= N <= 2^24, K % 64 == 0,
 *   64 <= K <= 64 * 65535, 0 <= r <= 128, r % 16 == 0.
 * For SVDQ_OUT_BF16 an activation enters the products rounded to 11 significant bits, for
 * SVDQ_OUT_FP32 to 22 (of values within 2^24 of the largest of its row's 512), and T's sums enter
 * the second product of the low-rank branch with 16 or 24; every product with a 4-bit code is exact
 * and every sum is in fp32.  A row with a NaN is NaN, one with an infinity has no finite output.
 */
size_t svdq_w4a16_workspace_bytes(int M, int N, int K, int r, int out_dtype);
int svdq_w4a16_gemv(const uint16_t* X, const float* inv_lambda, const uint16_t* L1p,
                    const uint8_t* container, const uint16_t* L2p, const uint16_t* bias, int M,
                    int N, int K, int r, void* Y, int out_dtype, void* workspace, void* stream);

/*
 * kv_block_plan — the bookkeeping of one step, on the device: from each request's cached tokens
 * (ctx) and new tokens (new) the blocks it needs more, taken off the end of the free list in the
 * requests' order, and a position and a slot for every new row.
 *   ctx_lens, new_lens   int32 [requests] (negative values count as 0)
 *   block_tables         int32 [requests, width], in and out: entry j of a request holds its
 *                        tokens [j bs, (j + 1) bs); the entries of blocks it holds are read, the
 *                        ones of new blocks are written, no other is touched
 *   free_blocks          int32 [free_capacity]; the first *free_count entries are free blocks
 *   free_count           int32 [1] (clamped to [0, free_capacity])
 *   cu_rows              int32 [requests + 1]: row range [cu_rows[b], cu_rows[b + 1]) of request b
 *   seq_lens             int32 [requests]: ctx + new, or ctx where the status is not 0
 *   positions            int32 [rows]: ctx + i for row i of a request, 0 behind the last request
 *   slots                int64 [rows]: the row's slot, -1 behind the last request and where the
 *                        status is not 0
 *   status               int32 [requests]: 0, or why the request got nothing this step:
 *                        1 the free list does not hold its blocks (nor then those of any later
 *                        request that needs one), 2 its tokens do not fit `width` blocks, 3 its
 *                        rows do not fit `rows`
 *   free_count_out       int32 [1]: what is left
 *   0 <= requests <= 2^20, 1 <= width, requests * width < 2^31, 0 <= rows <= 2^30,
 *   free_capacity >= 0.  No output overlaps an input or another output: workgroups read the lengths
 *   and the count at their own time (free_count_out that is free_count, and seq_lens or status that is
 *   one of the lengths, are refused).
 */
int kv_block_plan(const int32_t* ctx_lens, const int32_t* new_lens, int requests,
                  int32_t* block_tables, int width, int block_size, const int32_t* free_blocks,
                  int free_capacity, const int32_t* free_count, int32_t* cu_rows,
                  int32_t* seq_lens, int rows, int32_t* positions, int64_t* slots,
                  int32_t* status, int32_t* free_count_out, void* stream);

/*
 * kv_block_release — gives the blocks of finished requests back: the ceil(len / bs) blocks of
 * every request with done != 0 go to the end of the free list, in the requests' order (those
 * that no longer fit free_capacity are dropped), their table entries become -1 and their lengths
 * 0; the other requests keep theirs.
 *   seq_lens  int32 [requests];  done  uint8 [requests]
 *   block_tables  int32 [requests, width], in and out;  free_blocks  int32 [free_capacity], in
 *   and out;  free_count  int32 [1];  seq_lens_out  int32 [requests];  free_count_out  int32 [1]
 *   Limits as kv_block_plan.  seq_lens_out and free_count_out may not be their inputs.
 */
int kv_block_release(const int32_t* seq_lens, const uint8_t* done, int requests,
                     int32_t* block_tables, int width, int block_size, int32_t* free_blocks,
                     int free_capacity, const int32_t* free_count, int32_t* seq_lens_out,
                     int32_t* free_count_out, void* stream);

/*
 * kv_block_append — writes the K and V rows of new tokens into their slots.  For each block and
 * head with new tokens, amax over their values:
 *     s = max(s_old, fl32(amax / 127))   (s_old = 0 where the block's first token is among them),
 *     c = clamp(rne(fl32(x / s)), -127, 127), 0 where s = 0,
 * and where s > s_old the codes of the block's earlier tokens become rne(fl32(c fl32(s_old / s))).
 * A NaN among the values makes s NaN, an infinity makes it infinite (as does either in s_old); the new
 * codes are 0 then, and every token of that block and head reads as NaN until the block is begun anew.
 *   k, v     bf16 [rows, kv_heads, dim], 16B, rows k_stride / v_stride elements apart (a
 *            multiple of 8, at least kv_heads dim: slices of a fused projection need no copy)
 *   slots    int64 [rows], as written by kv_block_plan: the rows of one block must stand
 *            together, their offsets ascending by one (otherwise that block's contents are
 *            unspecified)
 *   rows >= 0, 1 <= kv_heads <= 65535, rows kv_heads <= 2^27, num_blocks >= 1; the cache may
 *   exceed 4 GiB.
 */
int kv_block_append(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                    const int64_t* slots, int rows, int kv_heads, int dim, int block_size,
                    int num_blocks, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
                    float* v_scale, void* stream);

/*
 * kv_block_read — the values the cache holds at `slots`: bf16(fl32(c s)) per element.  Rows
 * without a token are left as they were.
 *   slots    int64 [rows], in any order, repeats allowed
 *   k_out, v_out   bf16 [rows, kv_heads, dim]  16B
 *   Limits as kv_block_append.
 */
int kv_block_read(const int64_t* slots, int rows, int kv_heads, int dim, int block_size,
                  int num_blocks, const uint8_t* k_codes, const uint8_t* v_codes,
                  const float* k_scale, const float* v_scale, uint16_t* k_out, uint16_t* v_out,
                  void* stream);

/*
 * kv_block_attention — attention of ragged rows over the block cache.  Request b has the query
 * rows [cu_rows[b], cu_rows[b + 1]) and seq_lens[b] cached tokens, the rows' own among them; with
 * h' = h kv_heads / heads the cached head of query head h,
 *     out[i, h, :] = softmax_t(sm_scale q[i, h, :] . K[t, h', :]) V[t, h', :]
 * over the tokens t < seq_lens[b], and with `causal` only t <= seq_lens[b] - n + j for the j-th
 * of the request's n rows (also where the batch's `rows` end before the last of them).  A row with
 * no token gives 0; rows at or behind cu_rows[requests] are left as they were; tokens of a block whose
 * table entry is outside [0, num_blocks) are left out.  Scores, maxima, sums and outputs are in fp32; a
 * weight enters the product with V rounded to fp16 (11 bits, of weights times V scale down to 2^-24 of
 * the row's largest; what is below 2^-35 of it counts in the sum alone).
 * Blocks' V scales may lie as far apart as appends can make them, zero and subnormal ones among
 * them: one under 2^-80 of the largest of the request's and head's blocks may count as that, which
 * moves an output by less than 2^-56 of the largest |V|.  A block that an append gave a NaN or infinite
 * scale makes the rows that see it NaN, and no others.
 *   q        bf16 [rows, heads, dim], 16B, rows q_stride elements apart (as k_stride)
 *   block_tables   int32 [requests, width];  seq_lens  int32 [requests] (clamped to
 *            [0, width bs]);  cu_rows  int32 [requests + 1], ascending
 *   max_rows the most rows that any request has (a request's rows beyond it are left as they
 *            were); 1 for plain decoding.  It chooses the kernel for the whole batch: decoding
 *            requests and prompts in one call cost several times what a call for each kind does
 *   out      bf16 [rows, heads, dim]  16B
 *   workspace   device scratch of kv_block_attention_workspace_bytes(...) bytes (16B; may be
 *            NULL when that is 0), no initialization needed, rewritten by every call; calls that
 *            share one workspace must not overlap in time.  The size is that of the call's own
 *            arguments: a smaller batch can need more (its tokens are spread over more
 *            workgroups), so a workspace for several batches takes the largest of their sizes
 *   0 <= requests <= 65535, 0 <= rows <= 2^24, 1 <= max_rows <= 2^24, heads % kv_heads == 0,
 *   heads / kv_heads <= 128, requests kv_heads ceil(max_rows heads / kv_heads / n) < 2^23 with
 *   n = 16 where max_rows heads / kv_heads <= 16, else at least 32; width >= 1,
 *   requests * width < 2^31, width * bs <= 2^30, sm_scale finite.
 */
size_t kv_block_attention_workspace_bytes(int requests, int rows, int max_rows, int heads,
                                          int kv_heads, int dim, int width, int block_size);
int kv_block_attention(const uint16_t* q, int64_t q_stride, const uint8_t* k_codes,
                       const uint8_t* v_codes, const float* k_scale, const float* v_scale,
                       const int32_t* block_tables, int width, const int32_t* seq_lens,
                       const int32_t* cu_rows, int requests, int rows, int max_rows, int heads,
                       int kv_heads, int dim, int block_size, int num_blocks, int causal,
                       float sm_scale, uint16_t* out, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_SERVE_H */
