// Which variant of the persistent product kernel a launch takes: rules on its sizes alone, in plain C++.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMaxItems = 1 << 23;  // tiles of a launch

// As in ProductArgs: positions, output rows, experts, columns, bytes of a row, whether grouped by expert.
struct ProductSize {
  int P, R, E, N, Kb;
  bool grouped;
  // Rows that the positions can name: some of these are padding, some output rows may be no position's.
  int live() const { return P < R ? P : R; }
  // Experts that can hold one of them.
  int touched() const { return E < live() ? E : live(); }
};

// The tile of a launch: the one whose rounds over the 256 CUs take the least time, rounds counted whole up to two of
// them.  A round's cost is a 128-byte K step's time in us with all CUs busy (dense 8-bit, 8192 x 4096 x 4096: 120, 137,
// 178 and 287 us; the tiles of 128 and fewer columns run two to a CU and count half a pair's time), raised by a quarter
// for the small tiles, which read the same rows more often than a grouped launch's weight streams leave room for.  The
// narrowest tile costs half of the next, a little less where long rows hide its item changes.  Grouped launches count
// half a tile of padding per expert.  Measured, us, tiles of 256 x 256 / 128 x 256 / 64 x 128 / 32 x 128 / 32 x 64:
//   dense 8-bit, K 2048: 300 x 1024 25 / 16 / 8.2 / 6.7 / 6.5, 512 x 4096 26 / 17 / 10.1 / 13.4 / 14.6, 2048 x 2048
//   27 / 19 / 15.7 / 24 / 26, 4096 x 4096 38 / 42 / 51 / 77 / 87
//   bf16, 256 experts, top-8, K 2048, N 1024: 1 token (weights from HBM) - / - / 19 / 15.8 / 13.5, 32 tokens 93 / 67 /
//   59 / 57 / 55, 512 tokens 155 / 124 / 124 / 134 / 139, 1024 tokens 165 / 153 / 161 / 178 / 189, 2048 tokens 207 /
//   189 / 211 / 245 / 270, 8192 tokens 368 / 366 / - / - / -
//   8-bit, K 512, N 2048: 128 tokens 38 / 29 / 27 / 26 / 28, 777 tokens 57 / 46 / 43 / 51 / 56
// (128 x 128: 10% less where it makes 256 dense items, 15.0 for 2048 x 2048, and more elsewhere; not among them.)
inline int product_tile(const ProductSize& p, bool nt) {
  const struct {
    int bm, bn;
    float cost;
  } tiles[] = {
      {256, 256, 1.8f}, {128, 256, 1.1f}, {64, 128, 0.43f}, {32, 128, 0.36f}, {32, 64, p.Kb < 2048 ? 0.19f : 0.175f}};
  const int first = nt ? 1 : 0;  // below a mean of 64 rows the largest tile is never the best
  int best = 1;
  float least = 0.0f;
  for (int i = first; i < 5; ++i) {
    const int64_t cols = (p.N + tiles[i].bn - 1) / tiles[i].bn, all = ((int64_t)p.P + tiles[i].bm - 1) / tiles[i].bm;
    // far more positions than rows: the item list counts to kMaxItems (with kMaxProductOut 128 x 256 tiles stay below)
    if ((all + (p.E < p.P ? p.E : p.P)) * cols > kMaxItems) continue;
    const int64_t rows = p.grouped ? p.live() / tiles[i].bm + p.touched() / 2 + 1 : all;
    const int64_t items = rows * cols;
    const float rounds = items <= 512 ? (float)((items + 255) / 256) : (float)items / 256.0f;
    const float t = rounds * tiles[i].cost;
    if (least == 0.0f || t < least) best = i, least = t;
  }
  return best;
}

// Below a mean of 64 rows per expert a launch mostly streams weights: where they would not stay in the 256 MB
// Infinity Cache in any case, those of an expert's only tile pass the caches by, which then keep the rows of A and
// C.  With / without, us, bf16, 256 experts, top-8, K 2048, N 1024: 32 tokens 55 / 62, 512 tokens 124 / 138, 1024 tokens
// 152 / 161; at a mean of 64 189 / 189, at 256 363 / 367; 1 token, 33 MB of weights, 13.2 / 11.0 repeated, 13.3 / 13.5
// from HBM
inline bool product_streams(const ProductSize& p) {
  return p.live() / p.E < 64 && (int64_t)p.touched() * p.N * p.Kb > (128 << 20);
}

}  // namespace moe
