// Host-side launchers of the decoding step's kernels (declared to users in svdq_serve.h).
// Arguments are validated by the C ABI layer before any of these is called; each returns
// hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace svdq {

size_t w4a16_container_bytes(int N, int K);
hipError_t launch_w4a16_pack(const uint8_t* wq, const uint16_t* w_scales, int N, int K,
                             uint8_t* container, hipStream_t stream);

size_t w4a16_workspace_bytes(int M, int N, int K, int r, int out_fp32);
hipError_t launch_w4a16_gemv(const uint16_t* X, const float* inv_lambda, const uint16_t* L1p,
                             const uint8_t* container, const uint16_t* L2p, const uint16_t* bias,
                             int M, int N, int K, int r, void* Y, int out_fp32, void* workspace,
                             hipStream_t stream);

hipError_t launch_kv_block_plan(const int32_t* ctx, const int32_t* add, int requests,
                                int32_t* tables, int width, int bs, const int32_t* free_blocks,
                                int capacity, const int32_t* free_count, int32_t* cu,
                                int32_t* seq, int rows, int32_t* positions, int64_t* slots,
                                int32_t* status, int32_t* free_out, hipStream_t stream);

hipError_t launch_kv_block_release(const int32_t* seq, const uint8_t* done, int requests,
                                   int32_t* tables, int width, int bs, int32_t* free_blocks,
                                   int capacity, const int32_t* free_count, int32_t* seq_out,
                                   int32_t* free_out, hipStream_t stream);

// the cache's arrays and sizes, as in svdq_serve.h
struct BlockCacheView {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  int heads, dim, bs, num_blocks;
};

hipError_t launch_kv_block_append(const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                  int64_t v_stride, const int64_t* slots, int rows,
                                  const BlockCacheView& c, hipStream_t stream);

hipError_t launch_kv_block_read(const int64_t* slots, int rows, const BlockCacheView& c,
                                uint16_t* k_out, uint16_t* v_out, hipStream_t stream);

struct BlockAttention {
  const uint16_t* q;
  int64_t q_stride;
  BlockCacheView cache;
  const int32_t* tables;
  int width;
  const int32_t* seq;
  const int32_t* cu;
  int requests, rows, max_rows, heads, causal;
  float sm_scale;
  uint16_t* out;
  float* ws;
};

bool kv_block_attention_fits(int requests, int max_rows, int heads, int kv_heads, int dim);
size_t kv_block_attention_ws_bytes(int requests, int rows, int max_rows, int heads, int kv_heads,
                                   int dim, int width, int bs);
hipError_t launch_kv_block_attention(const BlockAttention& a, hipStream_t stream);

}  // namespace svdq
