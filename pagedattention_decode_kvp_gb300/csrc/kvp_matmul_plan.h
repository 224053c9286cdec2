// kvp_matmul_plan.h -- how a block-scaled matrix product is cut into tiles and CTAs: host
// code alone, without CUDA's headers.
#pragma once

namespace kvp {

constexpr int kNumSms = 152;
constexpr int kRowsB = 128;       // weight rows of a tile of the kernel for few rows
constexpr int kMaxSplits = 8;     // CTAs of a portable cluster

struct MatmulPlan {
  int tokens;                     // rows of a per tile (256: pairs of CTAs)
  int splits;                     // CTAs that share a tile's K
  int box() const { return tokens < 128 ? tokens : 128; }   // rows of a per copy (of b 128)
};

// The plan with the least time by a model of what was measured, in us: 2.6 for the start of a
// wave of CTAs (pairs: 3.5 once), a group of a CTA by its tokens and by whether its SM holds
// another CTA, the exchange of a cluster's sums, and the bytes of a and b at the rate of HBM.
// Measured and modelled (tokens x splits): 16 x 10240 x 8192 16x1 18.6 and 18.0, 16x3 16.9 and
// 15.8; 64 x 4096 x 4096 32x4 8.2 and 7.7, 64x4 8.7 and 8.5, 64x1 14.0 and 13.8; 64 x 10240 x
// 8192 64x3 19.1 and 17.9, 64x1 24.3 and 25.0; 256 x 4096 x 4096 128x2 12.9 and 12.5, pairs 17.4
// and 18.2; 517 x 4096 x 4096 128x1 27.3 and 34.0, pairs 18.6 and 18.2.
inline MatmulPlan matmul_plan(int m, int n, int groups) {
  struct Kind {
    int tokens, resident;      // rows of a per tile, CTAs of an SM
    double alone, shared;      // us a group
  };
  // clusters of 1 .. 8 CTAs that the GPU holds at a time, by the CTAs of an SM (its GPCs
  // have no multiple of most sizes: 48 clusters of 3, one CTA to an SM, take two waves).  A
  // table, so that a product has the same cut, and bits, on every board: four of them had the
  // first row's numbers, one on which clusters were counted the second's
  // (cudaOccupancyMaxActiveClusters gives the first row for both).  Where SMs lie otherwise, a
  // split may take a second wave: slower, not wrong.
  constexpr int kFit[2][kMaxSplits] = {{152, 76, 46, 36, 28, 23, 15, 15},
                                       {304, 152, 97, 74, 58, 46, 38, 36}};
  constexpr Kind kKinds[] = {{16, 2, 0.24, 0.28}, {32, 2, 0.30, 0.34}, {64, 2, 0.35, 0.58},
                             {128, 1, 0.45, 0.45}};
  const auto tiles = [](long long x, int per) { return (x + per - 1) / per; };
  MatmulPlan plan{256, 1};
  double best = 3.5 + 0.46 * groups * tiles(tiles(m, 256) * tiles(n, 256), kNumSms / 2);
  const double bytes = 2.6 + (static_cast<double>(m) + n) * groups * 128 / 6.5e6;
  for (const Kind& k : kKinds) {
    if (k.tokens / 2 >= m && k.tokens > 16) break;   // (a smaller one holds all rows)
    for (int splits = 1; splits <= kMaxSplits && (splits == 1 || 2 * splits <= groups); ++splits) {
      const long long clusters = tiles(m, k.tokens) * tiles(n, kRowsB), ctas = clusters * splits;
      const double waves = static_cast<double>(tiles(clusters, kFit[k.resident - 1][splits - 1]));
      if (splits > 1 && waves > 1) break;
      double t = waves * (2.6 + tiles(groups, splits) * (ctas > kNumSms ? k.shared : k.alone));
      if (splits > 1) t += 0.8 + 0.2 * splits + 0.006 * k.tokens * splits;
      if (t < bytes) t = bytes + (splits > 1 ? 0.1 * splits : 0.0);
      if (t < best) {
        best = t;
        plan = MatmulPlan{k.tokens, splits};
      }
    }
  }
  return plan;
}

}  // namespace kvp
