// The products' schedule: tile shape and split of the contraction, chosen by size.
// Plain C++ (no HIP), so that it can be compiled and checked on any host.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/hclrmix.h"

namespace hc {

// Most workgroup tiles of a product whose contraction is split: one arrival
// counter each in the workspace's prefix.
constexpr int MAX_SPLIT_TILES = HCLRMIX_COUNTER_BYTES / 4;

constexpr int CUS = 256;

// A tile shape, and the times (microseconds) of its model.
struct Shape {
  int bm, bn, bk, slots;  // slots: workgroups the chip runs at once, 1 to 3 per compute unit
  double step, floor;     // one contraction step with every slot of a compute unit in use, and at least
  double fixed;           // per tile: launch, first loads, epilogue
  double join, rate;      // split tiles: per part read by the workgroup that joins it, and the rate
                          // (TB/s) at which the parts are written and read
};

// Tile shape and split of a product.
struct Plan {
  const Shape* shape;
  int tiles_m, tiles_n;
  int64_t whole, rest;  // tiles taken whole, and split
  int splits;           // parts of each split tile
  double us;            // what the model expects
};

// A shape's tiles run in rounds of `slots` workgroups. Full rounds take their tiles whole; the
// tiles left over (all of them, where there are fewer than slots) are split along the
// contraction where that ends sooner: parts run shorter, but they are written and read again,
// and the last one to arrive reads them all.
// The shapes' times were fitted to 8,500 measured combinations of shape, split and product (1 to
// 8192 rows; ten weights from 2000 x 160 to 10240 x 2560; all three operand layouts, aligned and
// not, bf16 and fp32). At the fit the model's error had a standard deviation of about 12 %, and
// the plans it picked took 3 % more time on average than the best ones measured (56 % at worst).
// The kernels have changed since, and the fit has not been repeated: the epilogue goes through
// LDS by whole rows; unaligned fp32 operands are loaded 4 bytes at a time, straight into LDS, and
// are planned with the times of aligned ones; F16's floor was set by hand (fitted: 0.175). How
// far the model is from the present kernels is not known.
inline Plan shape_plan(const Shape& sh, int64_t M, int64_t N, int64_t K, bool dual, int segments, int batch) {
  Plan p{};
  p.shape = &sh;
  const int cols = dual ? sh.bn / 2 : sh.bn;
  p.tiles_m = (int)((M + sh.bm - 1) / sh.bm);
  p.tiles_n = (int)((N + cols - 1) / cols);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * batch;
  const int64_t steps = (K + sh.bk - 1) / sh.bk * segments;
  const int64_t rounds = tiles / sh.slots, rest = tiles % sh.slots;
  auto time = [&](int64_t wgs, int64_t n) {  // of wgs workgroups of n steps
    const double full = (double)(wgs / sh.slots) * (n * sh.step + sh.fixed);
    const int64_t left = wgs % sh.slots;
    const int64_t each = (left + CUS - 1) / CUS;  // of the compute units that have most
    return full + (left ? n * std::max(sh.floor, sh.step * each * CUS / sh.slots) + sh.fixed : 0.0);
  };
  int splits = 1;
  double best = time(rest, steps);
  if (rest && rest <= MAX_SPLIT_TILES) {
    for (int s = 2; s <= 64 && 2 * s <= steps && rest * s <= 2 * sh.slots; ++s) {
      const double traffic = 8.0 * rest * s * std::min<int64_t>(sh.bm, M) * sh.bn;
      const double t = time(rest * s, (steps + s - 1) / s) + (s + 3) * sh.join + traffic / (sh.rate * 1e6);
      if (t < best) {
        best = t;
        splits = s;
      }
    }
  }
  p.splits = splits;
  p.rest = splits > 1 ? rest : 0;
  p.whole = tiles - p.rest;
  p.us = time(rounds * sh.slots, steps) + best;
  return p;
}

constexpr Shape WIDE{256, 256, 64, 256, 1.488, 0.071, 10.116, 1.738, 8.9};
constexpr Shape MID{128, 128, 64, 512, 1.211, 0.787, 4.645, 0.607, 6.5};
constexpr Shape F64{64, 64, 64, 768, 0.826, 0.347, 3.790, 0.422, 13.1};
constexpr Shape F64D{64, 128, 64, 512, 1.164, 0.694, 1.541, 0.918, 9.6};
constexpr Shape F64W{64, 256, 64, 256, 0.722, 0.735, 5.175, 0.544, 6.2};
constexpr Shape F16{16, 64, 64, 768, 0.862, 0.400, 5.099, 0.083, 7.3};
constexpr Shape F16D{16, 128, 64, 512, 1.310, 0.709, 1.857, 0.423, 3.1};
constexpr Shape F16W{16, 256, 64, 256, 0.737, 0.626, 4.047, 0.419, 2.4};
// U: 16-bit operands that are not 16-byte aligned; S: fp32, aligned or not.
constexpr Shape U128{128, 128, 64, 512, 1.682, 1.934, 4.764, 0.518, 5.0};
constexpr Shape U64{64, 64, 64, 1024, 1.908, 0.857, 4.768, 0.302, 6.7};
constexpr Shape U64D{64, 128, 64, 768, 2.191, 1.832, 2.396, 0.705, 6.7};
constexpr Shape U16{16, 64, 64, 1024, 1.829, 0.744, 4.963, 0.118, 4.2};
constexpr Shape U16D{16, 128, 64, 768, 2.700, 1.436, 2.938, 0.241, 20.0};
constexpr Shape S128{128, 128, 32, 512, 4.129, 2.306, 5.816, 0.491, 6.3};
constexpr Shape S64{64, 64, 32, 768, 1.859, 0.818, 4.282, 0.352, 9.4};
constexpr Shape S64D{64, 128, 32, 512, 2.369, 1.428, 4.227, 0.696, 10.4};
constexpr Shape S16{16, 64, 32, 768, 0.968, 0.378, 6.002, 0.093, 20.0};
constexpr Shape S16D{16, 128, 32, 512, 1.163, 0.053, 5.300, 0.182, 20.0};

// The shapes that a product may take: f(shape). few: for at most 16 rows only.
template <typename F> inline void each_shape(int dtype, bool p_trans, bool dual, bool aln, F f) {
  const bool f32 = dtype == HCLRMIX_F32, few = !p_trans;
  if (f32 || !aln) {
    f(f32 ? S128 : U128, false);
    f(f32 ? (dual ? S64D : S64) : (dual ? U64D : U64), false);
    if (few) f(f32 ? (dual ? S16D : S16) : (dual ? U16D : U16), true);
  } else {
    f(MID, false);
    f(WIDE, false);
    f(dual ? F64D : F64, false);
    if (!p_trans) f(F64W, false);
    if (few) {
      f(dual ? F16D : F16, true);
      f(F16W, true);
    }
  }
}
constexpr int64_t FEW_ROWS = 16;

inline Plan make_plan(int dtype, int64_t M, int64_t N, int64_t K, bool p_trans, bool dual, int segments, int batch,
                      bool aln) {
  Plan best{};
  each_shape(dtype, p_trans, dual, aln, [&](const Shape& s, bool few) {
    if (few && M > FEW_ROWS) return;
    const Plan p = shape_plan(s, M, N, K, dual, segments, batch);
    if (!best.shape || p.us < best.us) best = p;
  });
  return best;
}

// Floats of one split tile's part: the rows that a tile can have.
inline int64_t part_size(const Shape& sh, int64_t M) { return std::min<int64_t>(sh.bm, M) * sh.bn; }

// Bytes of split-sum scratch (without the counters) that no plan of this product exceeds, nor of
// one with fewer rows: rows are M, or K with p_trans. So it grows with the rows, though a plan's
// own need does not, and a workspace for the most rows serves every call. With more rows a split
// tile's parts never pass 2 * slots in all (fewer tiles or steps: what those allow).
inline size_t product_scratch(int dtype, int64_t M, int64_t N, int64_t K, bool p_trans, bool dual, int segments,
                              int batch) {
  if (M == 0 || K == 0) return 0;
  int64_t most = 0;
  for (int aln = 0; aln < 2; ++aln)
    each_shape(dtype, p_trans, dual, aln != 0, [&](const Shape& s, bool few) {
      const int64_t m = few ? std::min(M, FEW_ROWS) : M;
      const int cols = dual ? s.bn / 2 : s.bn;
      const int64_t tiles = (m + s.bm - 1) / s.bm * ((N + cols - 1) / cols) * batch;
      const int64_t steps = (K + s.bk - 1) / s.bk * segments;
      const int64_t splits = std::min<int64_t>(64, steps / 2);
      if (splits < 2) return;
      int64_t parts;
      if (p_trans) {  // the same tiles for any number of rows
        const int64_t rest = tiles % s.slots;
        parts = rest ? rest * std::min(splits, 2 * s.slots / rest) : 0;
      } else {
        parts = std::min<int64_t>(2 * s.slots, std::min<int64_t>(tiles, s.slots - 1) * splits);
      }
      most = std::max(most, parts * part_size(s, m) * 4);
    });
  return (size_t)most;
}

}  // namespace hc
