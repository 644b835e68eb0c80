// Which kernels the dense feed-forward block's products run in (ffn.hip): rules on sizes alone, in
// plain C++, so that they can be asked without a GPU.
#pragma once

#include <algorithm>

namespace moe {
namespace ffn {

constexpr int kPlanCus = 256;  // tiles that run at once
inline long long ceil_div(long long n, int t) { return (n + t - 1) / t; }

struct Size {  // a product of m rows (tokens, or a gradient's rows) x n columns over `steps` of K
  long long m, n;
  int steps;
};
enum Shape { kBig, kTall, kWide, kSmall, kShares };

// Tile shapes, and what a step takes when the card is full of them, in us (bytes a step 64, 48 and
// 32 KB). Measured, the whole call in us, 256 x 256 / 256 x 128 / 128 x 128: [g | u] of 2048 x 7168 x
// 2048 141 / 107 / 142 (128, 256, 512 tiles), its y 51 / 64 / 88 (224, 448, 896), dH 155 / 107 / 80 (64,
// 128, 256); [g | u] of 1777 x 4096 x 1408 80 / 53 / 72 (77, 154, 308). 128 x 256 as 256 x 128: y of
// 1920 x 4352 in the one and of 4352 x 1920 in the other, 255 tiles each, 31 and 31 us at I = 2048, 126
// and 124 at 8192.
constexpr struct {
  int bm, bn;
  float us;
} kShapes[4] = {{256, 256, 1.35f}, {256, 128, 0.95f}, {128, 256, 0.95f}, {128, 128, 0.67f}};
inline long long shape_tiles(const Size& p, int shape) {
  return ceil_div(p.m, kShapes[shape].bm) * ceil_div(p.n, kShapes[shape].bn);
}
// The shape of the fewest rounds of one tile a CU, each at its step's time.
inline Shape tile_shape(const Size& p) {
  int best = 0;
  float least = 0.f;
  long long fewest = 0;
  for (int i = 0; i < 4; ++i) {
    const long long tiles = shape_tiles(p, i);
    const float us = (float)ceil_div(tiles, kPlanCus) * kShapes[i].us;
    if (i == 0 || us < least || (us == least && tiles < fewest)) {
      best = i;
      least = us;
      fewest = tiles;
    }
  }
  return (Shape)best;
}
// When the last of n1 tiles of t1 us and then n2 of t2 is done, each taken by the CU that is free
// first.
inline float time_of(long long n1, float t1, long long n2, float t2) {
  // whole rounds of the first, and its last round on some of the CUs
  const long long r = n1 / kPlanCus, some = n1 % kPlanCus;
  float at[2] = {r * t1, (r + (some ? 1 : 0)) * t1};  // when the others and those are free
  const long long n[2] = {kPlanCus - some, some};
  float done = n1 ? at[some ? 1 : 0] : 0.f;
  while (n2 > 0) {
    const int g = n[1] && at[1] < at[0] ? 1 : 0;
    at[g] += t2;
    done = std::max(done, at[g]);
    n2 -= n[g];
  }
  return done;
}

// What else a tile costs: its start, its first loads and its epilogue.
constexpr float kTileUs = 4.f;
// What shares of K cost beyond their steps: the second kernel, and up to 10 us for a card full of sums
// to be written and read (17 MB). With 5 us for those 384 x 2048 x 1408 took 39 us forward, 31 as it is;
// 256 x 4096 x 1408 36.5 and 31, backward 52 and 46; 512 x 4096 x 4096 backward 124 and 113.
inline float shares_us(long long shares, long long tiles) {
  return shares > 1 ? 4.f + 10.f * (float)(shares * tiles) / kPlanCus : 0.f;
}
// Shares of K for few 128 x 128 tiles, of four steps at least: where the steps that are left and the
// second kernel cost the least, a step of a card that is not full 0.6 us. Unsplit and split, both
// kernels, in us: [g | u] of 128 x 7168 x 2048 73 and 24 (8 shares), of 512 tokens 74 and 49 (2); its
// dH 60 and 19 (16), 61 and 30 (4); y of 333 x 4096 x 1024, 96 tiles of 16 steps, 12 and 18.
inline int shares_of(long long tiles, int steps) {
  const int most = (int)std::min((long long)kPlanCus / std::max(tiles, 1LL), (long long)steps / 4);
  int best = 1;
  float least = 0.6f * steps;
  for (int n = 2; n <= most; ++n) {
    const float us = 0.6f * steps / n + shares_us(n, tiles);
    if (us < least) {
      least = us;
      best = n;
    }
  }
  return best;
}

// A product on its own: in shares of K (more than one), or whole tiles of a shape.
struct Plan {
  Shape shape;
  int shares;
};
inline Plan plan_of(const Size& p) {
  const int n = shares_of(shape_tiles(p, kSmall), p.steps);
  return n > 1 ? Plan{kShares, n} : Plan{tile_shape(p), 1};
}
// A pair in one launch: the rows' tiles in each shape, or in shares, with the weights' likewise; the
// pair that is done first.
struct PairPlan {
  Plan rows, dw;
};
inline PairPlan plan_of_pair(const Size& rows, const Size& dw) {
  const long long nr = shape_tiles(rows, kSmall), nw = shape_tiles(dw, kSmall);
  const int sr = shares_of(nr, rows.steps), sw = shares_of(nw, dw.steps);
  PairPlan p{};
  float least = 0.f;
  for (int i = 0; i < (sr > 1 ? 5 : 4); ++i) {
    const bool si = i == kShares;
    const long long n1 = si ? nr * sr : shape_tiles(rows, i);
    const float t1 = (si ? kShapes[kSmall].us / sr : kShapes[i].us) * rows.steps;
    for (int j = 0; j < (sw > 1 ? 5 : 4); ++j) {
      const bool sj = j == kShares;
      const long long n2 = sj ? nw * sw : shape_tiles(dw, j);
      const float t2 = (sj ? kShapes[kSmall].us / sw : kShapes[j].us) * dw.steps;
      const float join = std::max(si ? shares_us(sr, nr) : 0.f, sj ? shares_us(sw, nw) : 0.f);
      const float us = time_of(n1, kTileUs + t1, n2, kTileUs + t2) + join;
      if ((i == 0 && j == 0) || us < least) {
        least = us;
        p = {{(Shape)i, si ? sr : 1}, {(Shape)j, sj ? sw : 1}};
      }
    }
  }
  return p;
}

// Few tokens: each weight read once by a workgroup that has nothing else to wait for. It also reads
// the tokens, which come from L2 at the rate that the weights do, so this pays up to some 320 KB of
// both a CU; more is split along K. Both kernels of the forward in us, with [g | u] so (split):
// 2048 x 2048, 1 token 12 (16), 16 13 (17), 32, 192 KB, 19 (24), 64, 320 KB, 26 (28); 2048 x 4096, 24
// tokens, 320 KB, 24.6 (25.7), 32 26 (25); 7168 x 2048, 16 tokens, 448 KB, 28.6 (26.5); 4096 x 8192,
// 1 MB, 69 (56). Up to 4 tokens their part is small and large weights go faster so: 1 x 8192 x 16384
// 150 (178), but 4096 x 8192 51 (48).
// y so (split): 4096 x 2048, 16 tokens, 128 KB, 18 (22); 2048 x 4096, 16 tokens, 256 KB, 21 (21.5);
// 4096 x 8192, 512 KB, 59 (57); 64 tokens, 32 columns a workgroup, 1.5 MB, 84 (49).
constexpr long long kFewBytes = 320 << 10;
inline long long bytes_a_cu(int T, int cols, long long groups, int K) {
  return 2LL * (cols + T) * K * ceil_div(groups, kPlanCus);
}
inline bool few_gate_up(int T, int d, int I) {
  return T <= 64 && (T <= 4 || bytes_a_cu(T, 16, I / 8, d) <= kFewBytes);
}
// 32 columns of y a workgroup where that leaves 192 of them, for half the reads of A: 7168 x 2048
// 28.6 us against 29.6; 4096 columns, 128 workgroups, 20.6 against 17.8.
inline int few_down_cols(int d) { return d / 32 >= kPlanCus * 3 / 4 ? 32 : 16; }
inline bool few_down(int T, int d, int I) {
  const int cols = few_down_cols(d);
  return T <= 64 && bytes_a_cu(T, cols, d / cols, I) <= kFewBytes;
}

}  // namespace ffn
}  // namespace moe
