// Host-only driver of the decoding step's validation paths, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_serve_abi_cpu.py (a CPU build; no call here reaches a
// kernel launch).  Extreme sizes must give a status, or a size, without overflow.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "svdq_serve.h"

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
  auto u8 = [&] { return static_cast<uint8_t*>(p); };
  auto u16 = [&] { return static_cast<uint16_t*>(p); };
  auto f32 = [&] { return static_cast<float*>(p); };
  auto i32 = [&] { return static_cast<int32_t*>(p); };
  auto i64 = [&] { return static_cast<int64_t*>(p); };
  const int ends[] = {INT_MIN, -1, 0, 1, 64, 65, 1 << 20, 1 << 24, INT_MAX / 64 * 64, INT_MAX};
  for (int M : ends)
    for (int K : ends) {
      (void)svdq_w4a16_workspace_bytes(M, INT_MAX, K, 128, 1);
      (void)svdq_w4a16_workspace_bytes(M, 1, K, INT_MAX, 0);
      for (int N : {INT_MIN, INT_MAX})
        EXPECT(svdq_w4a16_gemv(u16(), f32(), u16(), u8(), u16(), nullptr, M, N, K, 16, p, 0, p, nullptr) !=
               SVDQ_OK);
      (void)svdq_w4a16_container_bytes(M, K);
      EXPECT(svdq_pack_w4a16(u8(), u16(), INT_MAX, K, u8(), nullptr) != SVDQ_OK);
    }
  for (int n : ends)
    for (int w : ends)
      for (int bs : {16, 128, 17}) {
        EXPECT(kv_block_plan(i32(), i32(), n, i32(), w, bs, i32(), INT_MIN, i32(), i32(), i32(), INT_MAX,
                             i32(), i64(), i32(), i32(), nullptr) != SVDQ_OK);
        EXPECT(kv_block_release(i32(), u8(), n, i32(), w, bs, i32(), INT_MAX, i32(), i32(), i32(),
                                nullptr) != SVDQ_OK);
        for (int h : ends) {
          (void)kv_block_attention_workspace_bytes(n, 1 << 24, 1 << 24, h, h > 0 && h % 64 == 0 ? h / 64 : 1,
                                                   128, w, bs);
          EXPECT(kv_block_attention(u16(), LLONG_MAX, u8(), u8(), f32(), f32(), i32(), w, i32(), i32(), n,
                                    INT_MAX, 1, h, 1, 64, bs, INT_MAX, 1, 0.5f, u16(), p, nullptr) != SVDQ_OK);
          EXPECT(kv_block_append(u16(), u16(), LLONG_MIN, LLONG_MAX, i64(), n, h, 64, bs, w, u8(), u8(),
                                 f32(), f32(), nullptr) != SVDQ_OK);
          EXPECT(kv_block_read(i64(), n, h, 65, bs, w, u8(), u8(), f32(), f32(), u16(), u16(), nullptr) !=
                 SVDQ_OK);
        }
      }
  if (failures) std::fprintf(stderr, "%d check(s) failed\n", failures);
  else std::printf("all checks passed\n");
  return failures ? 1 : 0;
}
