// Host-only driver of the validation paths of svdq_decoder.h, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_decoder_abi_cpu.py (a CPU build; no call here reaches a
// kernel launch).  Extreme sizes must give a status, or a size, without overflow.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "svdq_decoder.h"

static int failures = 0;
#define EXPECT(cond)                                                         \
  do {                                                                       \
    if (!(cond)) {                                                           \
      std::fprintf(stderr, "check failed (line %d): %s\n", __LINE__, #cond); \
      ++failures;                                                            \
    }                                                                        \
  } while (0)

int main() {
  void* p = reinterpret_cast<void*>(0x10000);
  auto u16 = [&] { return static_cast<uint16_t*>(p); };
  auto i8 = [&] { return static_cast<int8_t*>(p); };
  auto f32 = [&] { return static_cast<float*>(p); };
  auto f64 = [&] { return static_cast<double*>(p); };
  auto i32 = [&] { return static_cast<int32_t*>(p); };
  const int ends[] = {INT_MIN, -1, 0, 1, 64, 65, 1 << 20, 1 << 24, INT_MAX / 64 * 64, INT_MAX};
  for (int M : ends)
    for (int K : ends) {
      EXPECT(svdq_rms_norm(p, 0, LLONG_MIN, p, 1, p, f32(), M, K, 0.0f, u16(), i8(), f32(), nullptr) != SVDQ_OK);
      EXPECT(svdq_rms_norm(p, 0, LLONG_MAX, p, 1, p, f32(), M, K, 0.0f, u16(), i8(), f32(), nullptr) != SVDQ_OK);
      EXPECT(svdq_quantize_rows(p, 2, 1 << 24, f32(), M, K, i8(), f32(), nullptr) != SVDQ_OK);
      (void)svdq_w8a8_container_bytes(M, K);
      EXPECT(svdq_pack_w8a8(i8(), INT_MAX, K, i8(), nullptr) != SVDQ_OK);
      (void)svdq_sample_workspace_bytes(M, K);
      EXPECT(svdq_sample(p, 0, LLONG_MAX, M, K, f32(), f32(), i32(), f32(), f32(), i32(), f32(), p, nullptr) != SVDQ_OK);
      for (int N : ends) {
        (void)svdq_w8a8_workspace_bytes(M, N, K);
        EXPECT(svdq_w8a8_gemm(i8(), f32(), i8(), f32(), nullptr, M, N, K, p, 7, p, nullptr) != SVDQ_OK);
        for (int64_t stride : {(int64_t)LLONG_MIN, (int64_t)LLONG_MAX, (int64_t)7})
          EXPECT(svdq_rope(p, stride, N, p, stride, M, 0, K, 128, 64, 0, i32(), f64(), 1.0f, u16(), stride, u16(),
                           stride, nullptr) != SVDQ_OK);
        EXPECT(svdq_rope(p, 1 << 20, 1, p, 1 << 20, 1, 0, M, K, N, 1, i32(), nullptr, 1.0f, u16(), 1 << 20, u16(),
                         1 << 20, nullptr) != SVDQ_OK);
      }
    }
  if (failures) std::fprintf(stderr, "%d check(s) failed\n", failures);
  else std::printf("all checks passed\n");
  return failures ? 1 : 0;
}
