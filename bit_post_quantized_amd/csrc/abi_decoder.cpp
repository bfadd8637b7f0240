// C ABI of the operators between a decoding step's projections (declared in include/svdq_decoder.h):
// argument validation and kernel dispatch, as in abi.cpp: every argument is checked before the HIP
// runtime is touched.
#include "svdq_decoder.h"

#include <hip/hip_runtime.h>

#include "abi_status.hpp"
#include "decoder_launch.hpp"

using namespace svdq::abi;

namespace {

constexpr int kMaxRows = 1 << 24, kMaxColumns = 1 << 24, kMaxHidden = 1 << 20;
constexpr int kMaxUnits = 2047;   // of 64 k: 64 * 2047 * 128^2 < 2^31

int check_dtype(const char* name, int dtype) {
  if (dtype != SVDQ_OUT_BF16 && dtype != SVDQ_OUT_FP32)
    return fail(SVDQ_EINVAL, "%s must be SVDQ_OUT_BF16 or SVDQ_OUT_FP32", name);
  return SVDQ_OK;
}

int check_stride(const char* name, int64_t stride, long long least) {
  if (stride < least || stride % 8 != 0 || stride > (1LL << 31))
    return fail(SVDQ_ESHAPE, "%s must be a multiple of 8 elements and at least %lld (got %lld)",
                name, least, (long long)stride);
  return SVDQ_OK;
}

int check_rows(const void* x, int x_dtype, int64_t x_stride, const float* gamma, int M, int K) {
  if (M < 0) return fail(SVDQ_EINVAL, "M must be >= 0 (got %d)", M);
  if (K <= 0) return fail(SVDQ_EINVAL, "K must be positive (got %d)", K);
  if (M > kMaxRows || K > kMaxHidden || K % 8 != 0)
    return fail(SVDQ_ESHAPE, "M must be <= 2^24, K <= 2^20 and a multiple of 8 (got %d, %d)", M, K);
  if (int s = check_dtype("x_dtype", x_dtype)) return s;
  if (int s = check_stride("x_stride", x_stride, K)) return s;
  if (M > 0 && !x) return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(x) || !aligned16(gamma))
    return fail(SVDQ_EALIGN, "x, gamma and factor must be 16-byte aligned");
  return SVDQ_OK;
}

int check_weight(int N, int K) {
  if (N <= 0 || K <= 0) return fail(SVDQ_EINVAL, "N and K must be positive (got %d, %d)", N, K);
  if (K % 64 != 0 || K / 64 > kMaxUnits)
    return fail(SVDQ_ESHAPE, "K must be a multiple of 64 and at most %d (got %d)", 64 * kMaxUnits, K);
  if (N > kMaxColumns) return fail(SVDQ_ESHAPE, "N must be <= 2^24 (got %d)", N);
  return SVDQ_OK;
}

int check_product(int M, int N, int K) {
  if (int s = check_weight(N, K)) return s;
  if (M < 0) return fail(SVDQ_EINVAL, "M must be >= 0 (got %d)", M);
  if (M > kMaxRows) return fail(SVDQ_ESHAPE, "M must be <= 2^24 (got %d)", M);
  if ((long long)M * N > kMaxElems) return fail(SVDQ_ESHAPE, "problem too large");
  return SVDQ_OK;
}

int check_vocab(int rows, int vocab) {
  if (rows < 0) return fail(SVDQ_EINVAL, "rows must be >= 0 (got %d)", rows);
  if (vocab <= 0) return fail(SVDQ_EINVAL, "vocab must be positive (got %d)", vocab);
  if (rows > 65535 || vocab > (1 << 22))
    return fail(SVDQ_ESHAPE, "at most 65535 rows and a vocabulary of 2^22 (got %d, %d)", rows, vocab);
  return SVDQ_OK;
}

}  // namespace

extern "C" {

int svdq_decoder_version(void) { return SVDQ_DECODER_VERSION; }

int svdq_rms_norm(const void* x, int x_dtype, int64_t x_stride, const void* residual,
                  int residual_dtype, void* residual_out, const float* gamma, int M, int K,
                  float eps, uint16_t* y, int8_t* codes, float* scales, void* stream) {
  if (int s = check_rows(x, x_dtype, x_stride, gamma, M, K)) return s;
  if (int s = check_dtype("residual_dtype", residual_dtype)) return s;
  if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(SVDQ_EINVAL, "eps must be >= 0 and finite");
  if (residual_out && !residual) return fail(SVDQ_EINVAL, "residual_out needs a residual");
  if (!codes != !scales) return fail(SVDQ_EINVAL, "codes and scales go together");
  if (M > 0 && !y && !codes) return fail(SVDQ_EINVAL, "y or codes is required");
  if (!aligned16(residual) || !aligned16(residual_out) || !aligned16(y) || !aligned16(codes))
    return fail(SVDQ_EALIGN, "residual, residual_out, y and codes must be 16-byte aligned");
  if (M == 0) return ok();
  const svdq::NormRows a{x, x_stride, residual, residual_out, gamma, M, K, 1, eps, y, codes, scales};
  return hip_status(svdq::launch_norm_rows(a, x_dtype == SVDQ_OUT_FP32, residual_dtype == SVDQ_OUT_FP32,
                                           (hipStream_t)stream),
                    "svdq_rms_norm");
}

int svdq_quantize_rows(const void* x, int x_dtype, int64_t x_stride, const float* factor, int M,
                       int K, int8_t* codes, float* scales, void* stream) {
  if (int s = check_rows(x, x_dtype, x_stride, factor, M, K)) return s;
  if (M > 0 && (!codes || !scales)) return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(codes)) return fail(SVDQ_EALIGN, "codes must be 16-byte aligned");
  if (M == 0) return ok();
  const svdq::NormRows a{x, x_stride, nullptr, nullptr, factor, M, K, 0, 0.0f, nullptr, codes, scales};
  return hip_status(svdq::launch_norm_rows(a, x_dtype == SVDQ_OUT_FP32, 0, (hipStream_t)stream),
                    "svdq_quantize_rows");
}

size_t svdq_w8a8_container_bytes(int N, int K) {
  return check_weight(N, K) ? 0 : svdq::w8a8_container_bytes(N, K);
}

int svdq_pack_w8a8(const int8_t* codes, int N, int K, int8_t* container, void* stream) {
  if (int s = check_weight(N, K)) return s;
  if (!codes || !container) return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(codes) || !aligned16(container))
    return fail(SVDQ_EALIGN, "codes and container must be 16-byte aligned");
  return hip_status(svdq::launch_w8a8_pack(codes, N, K, container, (hipStream_t)stream),
                    "svdq_pack_w8a8");
}

size_t svdq_w8a8_workspace_bytes(int M, int N, int K) {
  return check_product(M, N, K) || M == 0 ? 0 : svdq::w8a8_workspace_bytes(M, N, K);
}

int svdq_w8a8_gemm(const int8_t* qx, const float* sx, const int8_t* container, const float* sw,
                   const uint16_t* bias, int M, int N, int K, void* Y, int out_dtype,
                   void* workspace, void* stream) {
  if (int s = check_product(M, N, K)) return s;
  if (int s = check_dtype("out_dtype", out_dtype)) return s;
  if (!container || !sw || (M > 0 && (!qx || !sx || !Y))) return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(qx) || !aligned16(container) || !aligned16(Y) || !aligned16(workspace))
    return fail(SVDQ_EALIGN, "qx, container, Y and workspace must be 16-byte aligned");
  if (M == 0) return ok();
  if (!workspace && svdq::w8a8_workspace_bytes(M, N, K) > 0)
    return fail(SVDQ_EINVAL, "workspace is required for these sizes");
  return hip_status(svdq::launch_w8a8_gemm(qx, sx, container, sw, bias, M, N, K, Y,
                                           out_dtype == SVDQ_OUT_FP32, workspace, (hipStream_t)stream),
                    "svdq_w8a8_gemm");
}

int svdq_rope(const void* q, int64_t q_stride, int heads, const void* k, int64_t k_stride,
              int kv_heads, int x_dtype, int rows, int dim, int rot_dim, int interleaved,
              const int32_t* positions, const double* freqs, float scale, uint16_t* q_out,
              int64_t q_out_stride, uint16_t* k_out, int64_t k_out_stride, void* stream) {
  if (rows < 0 || kv_heads < 0 || heads <= 0)
    return fail(SVDQ_EINVAL, "rows and kv_heads must be >= 0, heads positive (got %d, %d, %d)", rows,
                kv_heads, heads);
  if (dim <= 0 || rot_dim <= 0)
    return fail(SVDQ_EINVAL, "dim and rot_dim must be positive (got %d, %d)", dim, rot_dim);
  if (dim % 8 != 0 || dim > 1024) return fail(SVDQ_ESHAPE, "dim must be a multiple of 8, at most 1024 (got %d)", dim);
  if (rot_dim % 16 != 0 || rot_dim > dim)
    return fail(SVDQ_ESHAPE, "rot_dim must be a multiple of 16, at most dim (got %d)", rot_dim);
  if (heads > 65535 || kv_heads > 65535 || ((long long)heads + kv_heads) * rows > (1 << 27))
    return fail(SVDQ_ESHAPE, "at most 65535 heads and rows * heads <= 2^27 (got %d, %d, %d)", heads, kv_heads, rows);
  if (int s = check_dtype("x_dtype", x_dtype)) return s;
  if (int s = check_stride("q_stride", q_stride, (long long)heads * dim)) return s;
  if (int s = check_stride("q_out_stride", q_out_stride, (long long)heads * dim)) return s;
  if (kv_heads > 0) {
    if (int s = check_stride("k_stride", k_stride, (long long)kv_heads * dim)) return s;
    if (int s = check_stride("k_out_stride", k_out_stride, (long long)kv_heads * dim)) return s;
  }
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f)
    return fail(SVDQ_EINVAL, "scale must be finite");
  if (!freqs || (rows > 0 && (!q || !q_out || !positions || (kv_heads > 0 && (!k || !k_out)))))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(freqs))
    return fail(SVDQ_EALIGN, "q, k, q_out, k_out and freqs must be 16-byte aligned");
  if ((q_out == q && (x_dtype == SVDQ_OUT_FP32 || q_stride != q_out_stride)) ||
      (kv_heads > 0 && k_out == k && (x_dtype == SVDQ_OUT_FP32 || k_stride != k_out_stride)))
    return rows > 0 ? fail(SVDQ_EINVAL, "in place, x must be bf16 and the strides the same") : ok();
  if (rows == 0) return ok();
  const svdq::RopeRows a{{q, k}, {q_stride, k_stride}, {q_out, k_out}, {q_out_stride, k_out_stride},
                         {heads, kv_heads}, rows, dim, rot_dim, interleaved ? 1 : 0, positions, freqs, scale};
  return hip_status(svdq::launch_rope(a, x_dtype == SVDQ_OUT_FP32, (hipStream_t)stream), "svdq_rope");
}

size_t svdq_sample_workspace_bytes(int rows, int vocab) {
  return check_vocab(rows, vocab) || rows == 0 ? 0 : svdq::sample_workspace_bytes(rows, vocab);
}

int svdq_sample(const void* logits, int logits_dtype, int64_t logits_stride, int rows, int vocab,
                const float* temperature, const float* uniform, const int32_t* top_k,
                const float* top_p, const float* min_p, int32_t* tokens, float* share,
                void* workspace, void* stream) {
  if (int s = check_vocab(rows, vocab)) return s;
  if (int s = check_dtype("logits_dtype", logits_dtype)) return s;
  if (logits_stride < vocab || logits_stride > (1LL << 31))
    return fail(SVDQ_ESHAPE, "logits_stride must be at least vocab and at most 2^31 (got %lld)", (long long)logits_stride);
  if (rows > 0 && (!logits || !temperature || !uniform || !tokens || !workspace))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(workspace)) return fail(SVDQ_EALIGN, "workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(logits) & (logits_dtype == SVDQ_OUT_FP32 ? 3u : 1u)) != 0)
    return fail(SVDQ_EALIGN, "logits must be aligned to an element");
  if (rows == 0) return ok();
  const svdq::SampleRows a{logits, logits_stride, rows, vocab, temperature, uniform, top_k, top_p, min_p,
                           tokens, share, workspace};
  return hip_status(svdq::launch_sample(a, logits_dtype == SVDQ_OUT_FP32, (hipStream_t)stream), "svdq_sample");
}

}  // extern "C"
