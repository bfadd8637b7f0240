// C ABI of the decoding step (declared in include/svdq_serve.h): argument validation and kernel
// dispatch, as in abi.cpp: every argument is checked before the HIP runtime is touched.
#include "svdq_serve.h"

#include <hip/hip_runtime.h>

#include "abi_status.hpp"
#include "serve_launch.hpp"

using namespace svdq::abi;

namespace {

constexpr int kMaxFewRows = 64;

int check_block(int bs) {
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128)
    return fail(SVDQ_ESHAPE, "block_size must be 16, 32, 64 or 128 (got %d)", bs);
  return SVDQ_OK;
}

int check_tables(int requests, int width, int bs) {
  if (requests < 0) return fail(SVDQ_EINVAL, "requests must be >= 0 (got %d)", requests);
  if (width <= 0) return fail(SVDQ_EINVAL, "width must be positive (got %d)", width);
  if (int s = check_block(bs)) return s;
  if (requests > (1 << 20)) return fail(SVDQ_ESHAPE, "requests must be <= 2^20 (got %d)", requests);
  if ((long long)requests * width >= (1LL << 31) || (long long)width * bs > (1LL << 30))
    return fail(SVDQ_ESHAPE, "block tables too large (%d requests, %d blocks)", requests, width);
  return SVDQ_OK;
}

int check_cache(int kv_heads, int dim, int bs, int num_blocks) {
  if (kv_heads <= 0 || num_blocks <= 0)
    return fail(SVDQ_EINVAL, "kv_heads and num_blocks must be positive (got %d, %d)", kv_heads,
                num_blocks);
  if (dim != 64 && dim != 128) return fail(SVDQ_ESHAPE, "dim must be 64 or 128 (got %d)", dim);
  if (int s = check_block(bs)) return s;
  if (kv_heads > 65535) return fail(SVDQ_ESHAPE, "kv_heads must be <= 65535 (got %d)", kv_heads);
  if ((long long)num_blocks * kv_heads > kMaxElems / (bs * dim))
    return fail(SVDQ_ESHAPE, "cache too large");
  return SVDQ_OK;
}

// (a workgroup has 16 rows of a head or more, and a launch fewer than 2^24 of them)
int check_rows(int rows, int kv_heads) {
  if ((long long)rows * kv_heads > (1 << 27))
    return fail(SVDQ_ESHAPE, "rows * kv_heads must be <= 2^27 (got %d * %d)", rows, kv_heads);
  return SVDQ_OK;
}

int check_stride(const char* name, int64_t stride, long long least) {
  if (stride < least || stride % 8 != 0 || stride > (1LL << 31))
    return fail(SVDQ_ESHAPE, "%s must be a multiple of 8 elements and at least %lld (got %lld)",
                name, least, (long long)stride);
  return SVDQ_OK;
}

}  // namespace

extern "C" {

int svdq_serve_version(void) { return SVDQ_SERVE_VERSION; }

static int check_w4a16(int N, int K) {
  if (N <= 0) return fail(SVDQ_EINVAL, "N must be positive (got %d)", N);
  if (int s = check_k(K)) return s;
  if (N > (1 << 24)) return fail(SVDQ_ESHAPE, "N must be <= 2^24 (got %d)", N);
  if (K / 64 > 65535) return fail(SVDQ_ESHAPE, "K / 64 must be <= 65535 (got K = %d)", K);
  if ((long long)N * K > kMaxElems) return fail(SVDQ_ESHAPE, "problem too large");
  return SVDQ_OK;
}

size_t svdq_w4a16_workspace_bytes(int M, int N, int K, int r, int out_dtype) {
  if (M <= 0 || M > kMaxFewRows || r < 0 || r > kMaxRank || check_w4a16(N, K)) return 0;
  return svdq::w4a16_workspace_bytes(M, N, K, r, out_dtype == SVDQ_OUT_FP32);
}

size_t svdq_w4a16_container_bytes(int N, int K) {
  return check_w4a16(N, K) ? 0 : svdq::w4a16_container_bytes(N, K);
}

int svdq_pack_w4a16(const uint8_t* wq, const uint16_t* w_scales, int N, int K, uint8_t* container,
                    void* stream) {
  if (int s = check_w4a16(N, K)) return s;
  if (!wq || !w_scales || !container) return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(wq) || !aligned16(container))
    return fail(SVDQ_EALIGN, "wq and container must be 16-byte aligned");
  return hip_status(svdq::launch_w4a16_pack(wq, w_scales, N, K, container, (hipStream_t)stream),
                    "svdq_pack_w4a16");
}

int svdq_w4a16_gemv(const uint16_t* X, const float* inv_lambda, const uint16_t* L1p,
                    const uint8_t* container, const uint16_t* L2p, const uint16_t* bias, int M,
                    int N, int K, int r, void* Y, int out_dtype, void* workspace, void* stream) {
  if (M < 0) return fail(SVDQ_EINVAL, "M must be >= 0 (got %d)", M);
  if (int s = check_w4a16(N, K)) return s;
  if (int s = check_rank(r)) return s;
  if (M > kMaxFewRows)
    return fail(SVDQ_ESHAPE, "M must be <= %d (got %d; svdq_w4a4_gemm takes more rows)",
                kMaxFewRows, M);
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_FP32)
    return fail(SVDQ_EINVAL, "out_dtype must be SVDQ_OUT_BF16 or SVDQ_OUT_FP32");
  if (!inv_lambda || !container || (M > 0 && (!X || !Y || !workspace)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (r > 0 && (!L1p || !L2p)) return fail(SVDQ_EINVAL, "L1p and L2p are required when r > 0");
  if (!aligned16(X) || !aligned16(inv_lambda) || !aligned16(container) || !aligned16(workspace) ||
      (r > 0 && (!aligned16(L1p) || !aligned16(L2p))))
    return fail(SVDQ_EALIGN,
                "X, inv_lambda, container, L1p, L2p and workspace must be 16-byte aligned");
  if (M == 0) return ok();
  return hip_status(svdq::launch_w4a16_gemv(X, inv_lambda, L1p, container, L2p, bias, M, N, K, r,
                                            Y, out_dtype == SVDQ_OUT_FP32, workspace,
                                            (hipStream_t)stream),
                    "svdq_w4a16_gemv");
}

int kv_block_plan(const int32_t* ctx_lens, const int32_t* new_lens, int requests,
                  int32_t* block_tables, int width, int block_size, const int32_t* free_blocks,
                  int free_capacity, const int32_t* free_count, int32_t* cu_rows,
                  int32_t* seq_lens, int rows, int32_t* positions, int64_t* slots,
                  int32_t* status, int32_t* free_count_out, void* stream) {
  if (int s = check_tables(requests, width, block_size)) return s;
  if (rows < 0 || free_capacity < 0)
    return fail(SVDQ_EINVAL, "rows and free_capacity must be >= 0 (got %d, %d)", rows,
                free_capacity);
  if (rows > (1 << 30)) return fail(SVDQ_ESHAPE, "rows must be <= 2^30 (got %d)", rows);
  if (!free_count || !cu_rows || !free_count_out || (free_capacity > 0 && !free_blocks) ||
      (requests > 0 && (!ctx_lens || !new_lens || !block_tables || !seq_lens || !status)) ||
      (rows > 0 && (!positions || !slots)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (free_count == free_count_out)
    return fail(SVDQ_EINVAL, "free_count_out may not be free_count");
  if (requests > 0 && (seq_lens == ctx_lens || seq_lens == new_lens || status == ctx_lens || status == new_lens))
    return fail(SVDQ_EINVAL, "seq_lens and status may not be ctx_lens or new_lens");
  return hip_status(
      svdq::launch_kv_block_plan(ctx_lens, new_lens, requests, block_tables, width, block_size,
                                 free_blocks, free_capacity, free_count, cu_rows, seq_lens, rows,
                                 positions, slots, status, free_count_out, (hipStream_t)stream),
      "kv_block_plan");
}

int kv_block_release(const int32_t* seq_lens, const uint8_t* done, int requests,
                     int32_t* block_tables, int width, int block_size, int32_t* free_blocks,
                     int free_capacity, const int32_t* free_count, int32_t* seq_lens_out,
                     int32_t* free_count_out, void* stream) {
  if (int s = check_tables(requests, width, block_size)) return s;
  if (free_capacity < 0)
    return fail(SVDQ_EINVAL, "free_capacity must be >= 0 (got %d)", free_capacity);
  if (!free_count || !free_count_out || (free_capacity > 0 && !free_blocks) ||
      (requests > 0 && (!seq_lens || !done || !block_tables || !seq_lens_out)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (free_count == free_count_out || (requests > 0 && seq_lens == seq_lens_out))
    return fail(SVDQ_EINVAL, "free_count_out and seq_lens_out may not be their inputs");
  return hip_status(svdq::launch_kv_block_release(seq_lens, done, requests, block_tables, width,
                                                  block_size, free_blocks, free_capacity,
                                                  free_count, seq_lens_out, free_count_out,
                                                  (hipStream_t)stream),
                    "kv_block_release");
}

int kv_block_append(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                    const int64_t* slots, int rows, int kv_heads, int dim, int block_size,
                    int num_blocks, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
                    float* v_scale, void* stream) {
  if (rows < 0) return fail(SVDQ_EINVAL, "rows must be >= 0 (got %d)", rows);
  if (int s = check_cache(kv_heads, dim, block_size, num_blocks)) return s;
  if (int s = check_rows(rows, kv_heads)) return s;
  if (int s = check_stride("k_stride", k_stride, (long long)kv_heads * dim)) return s;
  if (int s = check_stride("v_stride", v_stride, (long long)kv_heads * dim)) return s;
  if (!k_codes || !v_codes || !k_scale || !v_scale || (rows > 0 && (!k || !v || !slots)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(v_codes))
    return fail(SVDQ_EALIGN, "k, v, k_codes and v_codes must be 16-byte aligned");
  if (rows == 0) return ok();
  const svdq::BlockCacheView c{k_codes, v_codes, k_scale, v_scale, kv_heads, dim, block_size,
                               num_blocks};
  return hip_status(
      svdq::launch_kv_block_append(k, v, k_stride, v_stride, slots, rows, c, (hipStream_t)stream),
      "kv_block_append");
}

int kv_block_read(const int64_t* slots, int rows, int kv_heads, int dim, int block_size,
                  int num_blocks, const uint8_t* k_codes, const uint8_t* v_codes,
                  const float* k_scale, const float* v_scale, uint16_t* k_out, uint16_t* v_out,
                  void* stream) {
  if (rows < 0) return fail(SVDQ_EINVAL, "rows must be >= 0 (got %d)", rows);
  if (int s = check_cache(kv_heads, dim, block_size, num_blocks)) return s;
  if (int s = check_rows(rows, kv_heads)) return s;
  if (!k_codes || !v_codes || !k_scale || !v_scale || (rows > 0 && (!slots || !k_out || !v_out)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_out) || !aligned16(v_out))
    return fail(SVDQ_EALIGN, "k_codes, v_codes, k_out and v_out must be 16-byte aligned");
  if (rows == 0) return ok();
  const svdq::BlockCacheView c{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes),
                               const_cast<float*>(k_scale), const_cast<float*>(v_scale), kv_heads,
                               dim, block_size, num_blocks};
  return hip_status(svdq::launch_kv_block_read(slots, rows, c, k_out, v_out, (hipStream_t)stream),
                    "kv_block_read");
}

static int check_attention(int requests, int rows, int max_rows, int heads, int kv_heads, int dim,
                           int width, int block_size) {
  if (int s = check_cache(kv_heads, dim, block_size, 1)) return s;
  if (int s = check_tables(requests, width, block_size)) return s;
  if (rows < 0 || max_rows <= 0 || heads <= 0)
    return fail(SVDQ_EINVAL, "rows must be >= 0, max_rows and heads positive (got %d, %d, %d)",
                rows, max_rows, heads);
  if (heads % kv_heads != 0 || heads / kv_heads > 128)
    return fail(SVDQ_ESHAPE, "heads (%d) must be 1 to 128 times kv_heads (%d)", heads, kv_heads);
  if (requests > 65535 || rows > (1 << 24) || max_rows > (1 << 24))
    return fail(SVDQ_ESHAPE, "at most 65535 requests and 2^24 rows (got %d, %d, %d)", requests,
                rows, max_rows);
  if (!svdq::kv_block_attention_fits(requests, max_rows, heads, kv_heads, dim))
    return fail(SVDQ_ESHAPE, "too many rows: %d requests of up to %d rows and %d heads", requests,
                max_rows, heads);
  return SVDQ_OK;
}

size_t kv_block_attention_workspace_bytes(int requests, int rows, int max_rows, int heads,
                                          int kv_heads, int dim, int width, int block_size) {
  if (check_attention(requests, rows, max_rows, heads, kv_heads, dim, width, block_size)) return 0;
  return svdq::kv_block_attention_ws_bytes(requests, rows, max_rows, heads, kv_heads, dim, width,
                                           block_size);
}

int kv_block_attention(const uint16_t* q, int64_t q_stride, const uint8_t* k_codes,
                       const uint8_t* v_codes, const float* k_scale, const float* v_scale,
                       const int32_t* block_tables, int width, const int32_t* seq_lens,
                       const int32_t* cu_rows, int requests, int rows, int max_rows, int heads,
                       int kv_heads, int dim, int block_size, int num_blocks, int causal,
                       float sm_scale, uint16_t* out, void* workspace, void* stream) {
  if (int s = check_attention(requests, rows, max_rows, heads, kv_heads, dim, width, block_size))
    return s;
  if (int s = check_cache(kv_heads, dim, block_size, num_blocks)) return s;
  if (int s = check_stride("q_stride", q_stride, (long long)heads * dim)) return s;
  if (!(sm_scale == sm_scale) || sm_scale > 3.0e38f || sm_scale < -3.0e38f)
    return fail(SVDQ_EINVAL, "sm_scale must be finite");
  const bool some = requests > 0 && rows > 0;
  if (!k_codes || !v_codes || !k_scale || !v_scale ||
      (some && (!q || !block_tables || !seq_lens || !cu_rows || !out)))
    return fail(SVDQ_EINVAL, "NULL pointer");
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(out) ||
      !aligned16(workspace))
    return fail(SVDQ_EALIGN, "q, k_codes, v_codes, out and workspace must be 16-byte aligned");
  if (!some) return ok();
  if (!workspace && svdq::kv_block_attention_ws_bytes(requests, rows, max_rows, heads, kv_heads,
                                                      dim, width, block_size) > 0)
    return fail(SVDQ_EINVAL, "workspace is required for these sizes");
  const svdq::BlockCacheView c{const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(v_codes),
                               const_cast<float*>(k_scale), const_cast<float*>(v_scale), kv_heads,
                               dim, block_size, num_blocks};
  const svdq::BlockAttention a{q, q_stride, c, block_tables, width, seq_lens, cu_rows, requests,
                               rows, max_rows, heads, causal, sm_scale, out,
                               static_cast<float*>(workspace)};
  return hip_status(svdq::launch_kv_block_attention(a, (hipStream_t)stream),
                    "kv_block_attention");
}

}  // extern "C"
