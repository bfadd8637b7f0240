// What the C ABI's files share: the thread's error text and the statuses that set it.  Defined
// in abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace svdq {
namespace abi {

int fail(int status, const char* fmt, ...);
int ok();
int hip_status(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr long long kMaxElems = 1LL << 40;  // keeps every byte offset far inside size_t
constexpr int kMaxRank = 128;

int check_k(int K);
int check_rank(int r);

}  // namespace abi
}  // namespace svdq
