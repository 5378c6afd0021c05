// Tiling of the dense operators' few-row products (dense_few.cu).  Host only.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "tmem_share.h"

namespace moe {

constexpr int kFewBN = 128;            // rows of W a CTA (the MMA's M)
constexpr int kFewBK = 64;
constexpr int kFewMaxStages = 8;
constexpr uint32_t kFewWBytes = kFewBN * kFewBK * 2;
constexpr size_t kFewMaxSmem = 220 * 1024;

struct FewPlan {
  int tt;                  // tokens of the tile (the MMA's N)
  int stages, split;       // of a CTA's ring; CTAs of a cluster
  int tmem_cols;
  int64_t tiles;           // clusters
  int KB;                  // k-blocks in all
  size_t smem;             // dynamic shared memory of a CTA
};

// M (at most 128) tokens in `planes` planes times N rows of W (gated: of two
// matrices).  resident(split, per_sm): CTAs in clusters of `split` that are
// resident at once.
//
// CTAs an SM and CTAs a tile: what keeps most bytes in flight at once.  A CTA has at
// least two stages and six k-blocks, of many tokens (whose join costs more)
// twelve in a cluster of eight: 128 x 4096 x 5120 19 us in fours, 23 in eights, 48
// rows 15 in either.  Clusters of 1, 2, 4 or 8 (clusters of 3 fitted the SMs
// badly: 88 us where 4 took 65, one row of a 5120 / 12288 gated block; 2 took
// 75 us).
template <typename R>
inline FewPlan few_plan(int64_t M, int64_t K, int32_t N, bool gated, int planes, R resident) {
  FewPlan p{};
  const int nw = gated ? 2 : 1;
  p.tt = (int)((M + 15) / 16 * 16);
  p.KB = (int)((K + kFewBK - 1) / kFewBK);
  p.tiles = ((int64_t)N + kFewBN - 1) / kFewBN;
  const size_t stage = (size_t)nw * kFewWBytes + (size_t)planes * p.tt * kFewBK * 2;
  const size_t partial = (size_t)nw * p.tt * kFewBN * 4;
  p.tmem_cols = 32;
  while (p.tmem_cols < planes * nw * p.tt) p.tmem_cols *= 2;
  double best = 0;
  for (int per_sm = 1; per_sm <= 4; ++per_sm) {
    const size_t room = kFewMaxSmem / per_sm - (per_sm > 1 ? 2048 : 1024);       // stages or partial tile of a CTA
    const int stages = (int)std::min<size_t>(kFewMaxStages, room / stage);
    if (stages < 2 || partial > room || per_sm * p.tmem_cols > kTmemColumns) continue;
    int split = 1;
    while (split < 8 && p.tiles * split * 2 <= resident(split * 2, per_sm) &&
           p.KB / (split * 2) >= (split == 4 && p.tt > 64 ? 12 : 6))
      split *= 2;
    // (one CTA an SM leaves the next kernel's no room to start beside it)
    const double flight = (double)std::min<int64_t>(p.tiles * split, resident(split, per_sm)) * stages *
                          (per_sm == 1 ? 0.6 : 1.0);
    // (of two that keep as much, the fewer and deeper CTAs: 27 us against 45 for
    // 64 rows at 8192 x 4096, four stages and clusters of 4 against two and 8)
    if (flight > best) {
      best = flight;
      p.stages = stages;
      p.split = split;
    }
  }
  p.smem = tmem_smem(1024 + std::max(p.stages * stage, partial), p.tmem_cols);
  return p;
}

}  // namespace moe
