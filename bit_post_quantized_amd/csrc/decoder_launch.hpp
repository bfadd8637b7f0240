// Host-side launchers of the kernels declared to users in svdq_decoder.h.  Arguments are validated
// by the C ABI layer before any of these is called; each returns hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace svdq {

// a NULL `y` or `codes` is not written; `norm` 0: y = x gamma (residual NULL then)
struct NormRows {
  const void* x;
  int64_t x_stride;
  const void* residual;
  void* residual_out;
  const float* gamma;
  int M, K, norm;
  float eps;
  uint16_t* y;
  int8_t* codes;
  float* scales;
};
hipError_t launch_norm_rows(const NormRows& a, int x_fp32, int residual_fp32, hipStream_t stream);

size_t w8a8_container_bytes(int N, int K);
hipError_t launch_w8a8_pack(const int8_t* codes, int N, int K, int8_t* container,
                            hipStream_t stream);
size_t w8a8_workspace_bytes(int M, int N, int K);
hipError_t launch_w8a8_gemm(const int8_t* qx, const float* sx, const int8_t* container,
                            const float* sw, const uint16_t* bias, int M, int N, int K, void* Y,
                            int out_fp32, void* workspace, hipStream_t stream);

struct RopeRows {
  const void* in[2];       // q, k
  int64_t in_stride[2];
  uint16_t* out[2];
  int64_t out_stride[2];
  int heads[2];
  int rows, dim, rot, interleaved;
  const int32_t* positions;
  const double* freqs;
  float scale;
};
hipError_t launch_rope(const RopeRows& a, int x_fp32, hipStream_t stream);

struct SampleRows {
  const void* logits;
  int64_t stride;
  int rows, vocab;
  const float* temperature;
  const float* uniform;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* share;
  void* ws;
};
size_t sample_workspace_bytes(int rows, int vocab);
hipError_t launch_sample(const SampleRows& a, int logits_fp32, hipStream_t stream);

}  // namespace svdq
