// Which kernel a product of the gated block takes: plain C++ on its sizes, for
// the launches in zs_glu_gemm.hip.  Not installed; not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cmath>

namespace zs {

// The three products, M x N outputs over a summed axis of K:
//   kForward  a = x [M][K], b = w_gate and w_up [N][K]; out[0] = h, out[1], out[2] = gate, up (NULL: not kept)
//   kInput    a = dgate and dup [M][K], b = w_gate and w_up [K][N]; out[0] = dx, both products in one sum
//   kWeight   a = dgate and dup [K][M], b = x [K][N]; out[0], out[1] = dw_gate, dw_up (+ add[0], add[1])
enum class GluOp : int32_t { kForward = 0, kInput = 1, kWeight = 2 };

namespace glu {

constexpr int kStage = 64;  // of the summed axis a stage: 128 bytes of a row
constexpr int64_t kMostTiles = 1 << 22;  // workgroups along a grid's first axis: 2^31 threads at most

// The kernel of a product with rows on 4-byte boundaries, by the time it takes: a start, and so much a stage of 64 of the summed axis,
// between `few` for a few workgroups and `full` for as many as run at once; more go in rounds (half overlapped) with a
// start of their own.  us of the kernels, fitted to 54 shapes from 1 to 9683 tokens on 256 compute units, inputs from
// memory and outputs in 16 bits: off by 6 to 20% there.  Of calls among others they are 0.4 to 1.25 times what those take, 0.89
// forward, 0.91 input gradient and 0.78 weight gradients in the median of 88 products with sizes drawn from 1 to 16384
// tokens and 256 to 11008 features (a call's own 4 us, fp32 outputs and what is added to them are not in them).  What
// counts is the order that they put the kernels in: there the pick was 1.7, 0.8 and 1.4% behind the best kernel in
// the mean, 16, 8 and 8% at worst.  For example (predicted), forward: 1 x 11008 x 4096 39.9 by k64 (28.5), 39.6 by k128 (33.5), 41.3 by kFew
// (38.8); 333 x 11008 x 4096 85.8 by k192 (69.2), 97.1 by k128 (92.7), 97.0 by k256 (92.7); 1000 x 1371 x 1000, kept, 17.0 by k128
// (11.8), 19.8 by k64 (16.6); input gradient: 61 x 4096 x 4096 27.9 by kSplit (24.1), 35.7 by k32 (37.9); weight gradients: 61 x 4096 x
// 4096 22.4 by k128Near (22.4), 19.6 by k256 (22.6); 1025 x 1376 x 4096 in bf16 30.6 by k256 (32.4), 33.3 by k128Near (37.5), in fp32
// 33.9 and 36.5, added to fp32 sums 50.8 and 53.9.
enum class GluTile : int32_t { kAny, kThrough, kFew, kSplit, k64x32, k32, k64, k64x128, k128, k128Near, k192, k256 };
struct TileCost {
  GluTile tile;
  int bm, bn, at_once;  // sums of a workgroup; workgroups at once
  double start, few, full, round;
};
constexpr TileCost kForwardCosts[] = {{GluTile::kFew, 16, 32, 2048, 3.68, 0.089, 1.459, 0.0},
                                      {GluTile::k64x32, 64, 32, 256, 3.74, 0.200, 0.237, 1.24},
                                      {GluTile::k64, 64, 64, 512, 3.80, 0.243, 0.455, 0.40},
                                      {GluTile::k128, 128, 128, 256, 4.50, 0.324, 0.516, 2.14},
                                      {GluTile::k192, 192, 128, 512, 6.00, 0.564, 1.195, 2.32},
                                      {GluTile::k256, 256, 256, 256, 7.00, 0.972, 1.518, 3.42}};
constexpr TileCost kInputCosts[] = {{GluTile::kSplit, 16, 64, 256, 3.02, 0.124, 0.165, 1.30},
                                    {GluTile::k32, 32, 64, 512, 3.40, 0.248, 0.334, 0.72},
                                    {GluTile::k64x128, 64, 128, 256, 4.54, 0.356, 0.435, 1.48},
                                    {GluTile::k128, 128, 128, 256, 5.00, 0.452, 0.603, 2.11},
                                    {GluTile::k128Near, 128, 128, 512, 5.00, 0.647, 1.008, 2.00},
                                    {GluTile::k256, 256, 256, 256, 7.00, 1.092, 1.548, 0.99}};
constexpr TileCost kWeightCosts[] = {{GluTile::k64, 64, 64, 1024, 3.99, 0.294, 0.745, 2.01},
                                     {GluTile::k128, 128, 128, 256, 5.14, 0.406, 0.527, 2.55},
                                     {GluTile::k128Near, 128, 128, 512, 6.59, 0.460, 0.899, 3.05},
                                     {GluTile::k256, 256, 256, 256, 8.99, 1.156, 1.454, 5.34}};
inline int64_t tiles_of(int64_t M, int64_t N, int64_t bm, int64_t bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); }
// kAny: too many tiles of every kind.
template <size_t COSTS>
GluTile cheapest(const TileCost (&costs)[COSTS], int64_t M, int64_t wide, int64_t parts, int64_t stages) {
  double least = 1e300;
  GluTile best = GluTile::kAny;
  for (const TileCost& c : costs) {
    const int64_t tiles = tiles_of(M, wide, c.bm, c.bn);
    if (tiles >= kMostTiles) continue;
    const double x = (double)(parts * tiles) / c.at_once;
    const double stage = c.few + (c.full - c.few) * (x < 1 ? x : 1);
    const double us = x <= 1 ? c.start + stage * (double)stages : c.start + 0.5 * (x + std::ceil(x)) * (c.round + stage * (double)stages);
    if (us < least) least = us, best = c.tile;
  }
  return best;
}

// `direct`: rows that the direct loads to LDS take.
inline GluTile choose(GluOp op, int64_t M, int64_t N, int64_t K, bool direct) {
  const int64_t stages = (K + kStage - 1) / kStage, parts = op == GluOp::kWeight ? 2 : 1;
  if (K == 0) return GluTile::kAny;
  if (!direct) {
    const int64_t tiles = parts * tiles_of(M, N, 128, op == GluOp::kForward ? 64 : 128);
    return tiles < 64 || tiles >= kMostTiles ? GluTile::kAny : GluTile::kThrough;
  }
  switch (op) {
    case GluOp::kForward: return cheapest(kForwardCosts, M, 2 * N, 1, stages);
    case GluOp::kInput: return cheapest(kInputCosts, M, N, 1, 2 * stages);
    default: return cheapest(kWeightCosts, M, N, 2, stages);
  }
}

}  // namespace glu
}  // namespace zs
