// Which kernel the 8-bit product takes, by its sizes alone (host code, also compiled by itself to check
// that the tests reach every choice).
#pragma once

#include <stdint.h>

namespace svdq {
namespace w8a8 {

constexpr int kFewRows = 64;
constexpr int kCus = 256;

struct Plan {
  int rt, wn;   // a tile of 64 rt x 64 wn; 0: few rows
  int groups;   // of waves in a workgroup, each with its units of K
  int split;
};

// Tiles of 16 columns of a workgroup for `rt` tiles of 16 rows: more of them read X less often, fewer leave more
// workgroups, and more of them on a CU.  Measured with 64 / 32 / 16 columns, us: 16 x 8192 x 28672 (rows, K, columns)
// 38 / 46 / 51, 32 x 8192 x 28672 43 / 55 / 71, one row of 4096 x 131072, where a wave has eight units in all, 93 / 78 /
// 86, of 8192 x 8192 15 / 14 / 12.
inline int few_columns(int rt, int tiles, int K) {
  if (tiles >= 4 * kCus) return rt == 1 && K <= 4096 ? 2 : 4;
  return rt > 1 && tiles >= 2 * kCus ? 2 : 1;
}

inline Plan plan(int M, int N, int K) {
  const int G = K / 64;
  Plan best{0, 0, 1, 1};
  double least = 1e30;
  const double weights = (double)N * K / 5900.0;   // ns, for memory's part
  if (M <= kFewRows) {
    // What a unit of 16 columns costs a CU, ns, by the rows and the columns of a workgroup: each wave brings X to LDS
    // for itself, which from 17 rows on may take longer than the smallest tile's way.  Measured, us: 24 / 40 / 64 rows of
    // 8192 x 28672 42 / 50 / 58 against 44 / 44 / 45 in tiles, of 4096 x 131072 101 / 121 / 136 against 92 / 93 / 98, of
    // 16384 x 1024 17 / 23 / 30 against 14 / 14 / 15, of 8192 x 8192 16 / 19 / 23 against 20 / 20 / 21, of 4096 x 4096
    // 7 / 9 / 10 against 12 / 12 / 13.
    const int rt = (M + 15) / 16, tiles = (N + 15) / 16, columns = few_columns(rt, tiles, K);
    if (rt == 1) return best;
    const double groups = (double)((tiles + columns - 1) / columns) / kCus;
    const double unit = columns == 4 ? 30 + 0.53 * M : columns == 2 ? 25 + 0.85 * M : 20 + 1.3 * M;
    const double few = groups > 1.0 ? groups * (columns * G * unit + 1000.0) : columns * G * unit;
    least = 0.97 * (few > weights ? few : weights);
  }
  // The tile and the division of K with the least time, by what a unit of K costs a CU with each tile (ns,
  // measured where all CUs are busy: small tiles read LDS and L2 more often for the same products) times the
  // items that the busiest CU has; divided sums cost a launch (the join takes 3.6 - 4.6 us for 39 x 40 to 20 x 15563
  // sums, 6.8 for 113 x 15747) and are written and read once more.  Up to 64 rows 2.5 us more are asked for.  Measured, us,
  // with 6.5 / with 4: 24 x 6144 x 14000 19.8 / 22.4, 32 x 8192 x 8192 17.5 / 20.2, 20 x 16384 x 4096 18.6 / 20.7, 64 x 4096 x 512
  // 9.1 / 10.4; the other way 40 x 8192 x 5120 24.1 / 17.4, 48 x 6144 x 6144 21.2 / 16.1, 64 x 4096 x 6144 17.0 / 14.8, where the
  // first kind has a few workgroups more than there are CUs, which its estimate does not see.  Measured,
  // us, 256 x 256 / 128 x 256 / 128 x 128 / 64 x 128, with the best division: 300 x 8192 x 28672 (M, K, N) 94 / 100 / 98 / 111,
  // 2000 x 8192 x 4096 82 / 65 / 74 / 94, 1000 x 4096 x 8192 45 / 37 / 41 / 53, 1000 x 4096 x 4096 40 / 29 / 24 / 28, 500 x
  // 12288 x 4096 46 / 39 / 39 / 37 (undivided 110 / 64 / 51 / 37), 256 x 4096 x 4096 26 / 21 / 18 / 14.  The smallest tile's
  // two groups of waves against one: 500 x 12288 x 4096 37 / 44, 256 x 4096 x 4096 14.4 / 16.6, 100 x 4096 x 12288
  // 15.3 / 17.8; for 128 x 128 no gain (39.1 / 39.0, 17.9 / 18.2, 98 / 98).
  static const struct { int rt, wn, groups; double ns; } kTiles[] = {{4, 4, 1, 860}, {2, 4, 1, 510}, {2, 2, 1, 290}, {1, 2, 2, 180}};
  for (const auto& t : kTiles) {
    if (M <= 64 * (t.rt - 1)) continue;   // (a tile half empty)
    const int64_t tiles = (int64_t)((M + 64 * t.rt - 1) / (64 * t.rt)) * ((N + 64 * t.wn - 1) / (64 * t.wn));
    for (int split = 1; split <= 8; split *= 2) {
      if (split > 1 && (tiles * split > 2 * kCus || G < 8 * split)) break;
      const int64_t rounds = (tiles * split + kCus - 1) / kCus;
      double ns = (double)rounds * ((G + split - 1) / split) * (M <= kFewRows ? 150 + 1.4 * M : t.ns);
      if (split > 1) ns += (M <= kFewRows ? 6500 : 4000) + ((double)M * N * (8 * split + 4)) / 5500;
      if (M <= kFewRows && ns < weights) ns = weights;
      if (ns < least) {
        least = ns;
        best = {t.rt, t.wn, t.groups, split};
      }
    }
  }
  return best;
}

}  // namespace w8a8
}  // namespace svdq
