// What the 8-bit product chooses (csrc/w8a8_plan.hpp), built by tests/test_w8a8_plan_cpu.py: for each
// "M K N" read, or, with the argument "all", every choice over the sizes that it takes, each with one of
// the sizes that lead to it: "few <tiles of 16 rows> <tiles of 16 columns>" or "tile <rows> <columns>
// <groups of waves> <shares of K>", and " of few rows" where the first would have been possible.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>

#include "w8a8_plan.hpp"

static std::string kind(int M, int K, int N) {
  using namespace svdq::w8a8;
  const Plan p = plan(M, N, K);
  const int rt = (M + 15) / 16;
  char s[64];
  if (p.rt == 0) std::snprintf(s, sizeof s, "few %d %d", rt, few_columns(rt, (N + 15) / 16, K));
  else std::snprintf(s, sizeof s, "tile %d %d %d %d%s", 64 * p.rt, 64 * p.wn, p.groups, p.split,
                     M <= kFewRows ? " of few rows" : "");
  return s;
}

int main(int argc, char** argv) {
  if (argc > 1 && std::strcmp(argv[1], "all") == 0) {
    std::map<std::string, std::string> found;
    auto look = [&](int M, int K, int N) {
      std::string& at = found[kind(M, K, N)];
      if (at.empty()) at = std::to_string(M) + " " + std::to_string(K) + " " + std::to_string(N);
    };
    // rows and columns at tiles' ends, units of K ever farther apart
    for (int M = 1; M <= 1 << 14; M += M < 128 ? 1 : M < 1024 ? 32 : M < 4096 ? 192 : 1536)
      for (double u = 1; u <= 2047; u = std::floor(u * 1.05 + 1))
        for (double n = 1; n <= 1 << 24; n = std::floor(n * 1.04 + 1)) {
          const int N = ((int)n + 15) / 16 * 16;
          if ((long long)M * N <= 1LL << 40) look(M, 64 * (int)u, N);
        }
    for (const auto& f : found) std::printf("%s : %s\n", f.first.c_str(), f.second.c_str());
    return 0;
  }
  int M, K, N;
  while (std::scanf("%d %d %d", &M, &K, &N) == 3) std::printf("%s\n", kind(M, K, N).c_str());
  return 0;
}
