// Which tiles the products of the orthogonalised update take, and how their sums
// are split: plain C++ on their sizes, for the launches in zs_muon.hip.  Not
// installed; not part of the ABI.
#pragma once

#include <stdint.h>

namespace zs {
namespace ns {

constexpr int64_t kSmallSide = 128;  // matrices with both sides up to this are done by a workgroup each
inline bool one_workgroup(int64_t rows, int64_t cols) { return rows <= kSmallSide && cols <= kSmallSide; }
constexpr int64_t kSlabSide = 64;    // with the shorter up to this, by two kernels a step: S, and the rest

inline int64_t padded(int64_t n) { return (n + 31) / 32 * 32; }

enum class NsTile : int32_t { k32 = 0, k64 = 1, k128 = 2, k192 = 3, k256 = 4 };
constexpr int kTiles = 5, kTileSide[kTiles] = {32, 64, 128, 192, 256};
struct Choice {
  NsTile tile;
  int32_t splits;
  int64_t tiles;
};
inline int64_t tiles_of(int64_t m, int64_t n, int64_t side, bool triangle) {
  const int64_t tm = (m + side - 1) / side, tn = (n + side - 1) / side;
  return triangle ? tm * (tm + 1) / 2 : tm * tn;
}
// The tile and the split of a product, by the time its kernel takes (us, measured on 256 compute units): a start and an
// end, and so much a stage of 32 for a few workgroups, for 256, and for 512 where two or more fit a unit; more go in
// rounds, which overlap by half.  Split sums cost their exchange.  For example (rows x columns, product): 256 x 768, S 6.2
// in 32 x 32 tiles, 8.1 in 64 x 64; 1024 x 1024, S 10.6 / 10.6, in 128 x 128 27, in 256 x 256 64, B X 16.2 / 13.2 / 29 / 62;
// 2048 x 2048, S 46 in 64 x 64, 48 in 128 x 128, 108 in 256 x 256, B X 62 / 55 / 108; 4096 x 4096, S 332 / 213 / 205, in 192 x 192 172,
// B X 419 / 305 / 275, in 192 x 192 328.  128 x 4096, S in 32 x 32 tiles: 20.0, in 2 splits 13.1, in 4 9.4.  (Small tiles are
// bound by what a compute unit takes in, 94 bytes a ns alone and 58 with all: waves that split a workgroup's sums four ways
// took as long, 9.2 against 7.6 us at 4 x 512 x 512.)
struct TileTime {
  double start, few, full, twice;  // twice = 0: one a unit
  double exchange, exchange_each;
};
constexpr TileTime kTileTime[kTiles] = {{3.8, 0.12, 0.16, 0.22, 1.2, 0.25},
                                        {4.0, 0.175, 0.29, 0.45, 2.4, 0.35},
                                        {5.5, 0.47, 0.78, 1.17, 4.0, 0.9},
                                        {7.0, 0.83, 1.33, 0.0, 8.0, 2.0},
                                        {10.0, 1.37, 2.1, 0.0, 12.0, 3.5}};
inline double product_us(int t, int64_t groups, int64_t stages, int64_t splits) {
  const TileTime& c = kTileTime[t];
  const int64_t all = groups * splits, at_once = c.twice > 0 ? 512 : 256;
  double stage;
  if (all <= 256) {
    stage = c.few + (c.full - c.few) * (double)all / 256;
  } else if (all <= at_once) {
    stage = c.full + (c.twice - c.full) * (double)(all - 256) / 256;
  } else {
    const double rounds = 0.5 * ((double)all / (double)at_once + (double)((all + at_once - 1) / at_once));
    stage = (c.twice > 0 ? c.twice : c.full) * rounds;
  }
  return c.start + stage * (double)((stages + splits - 1) / splits) +
         (splits > 1 ? c.exchange + c.exchange_each * (double)splits : 0.0);
}
inline Choice choose(int64_t m, int64_t n, int64_t k, int64_t batch, bool triangle) {
  const int64_t stages = k / 32;
  Choice best{NsTile::k32, 1, 0};
  double least = 1e300;
  for (int t = 0; t < kTiles; ++t) {
    const int64_t tiles = tiles_of(m, n, kTileSide[t], triangle);
    for (int64_t splits = 1; splits <= 16; splits *= 2) {
      // split sums: of at most a workgroup a unit (1024 x 1024, S in 272 halves: 13.4 us, 10.6 in 136 whole ones), 4 stages
      // each at least
      if (splits > 1 && (tiles * batch * splits > 256 || stages < 4 * splits)) break;
      const double us = product_us(t, tiles * batch, stages, splits);
      if (us < least) {
        least = us;
        best = Choice{(NsTile)t, (int32_t)splits, tiles};
      }
    }
  }
  return best;
}

}  // namespace ns
}  // namespace zs
