// product.h -- a layer's matrix product as the C entry points plan it.
#pragma once
#include "ops.h"

namespace muon {

struct Product {
  GemmArgs g{};
  int tile = kTile128;
  int loads = kStaged;
  uint64_t ws = 0;            // partials of a split contraction
  AlignArgs copy[2]{};        // of A and B, where copy_bytes > 0
  uint64_t copy_bytes[2] = {0, 0};
  bool pairs = false;         // rows 2r and 2r + 1 are added to one row of C
  uint64_t total() const { return ws + copy_bytes[0] + copy_bytes[1]; }
  uint64_t need() const { return g.m == 0 || g.n == 0 ? 0 : total(); }  // nothing to compute: nothing is used
};

// The tile and the split of p->g (m, n, k set) over `groups` groups (0: none).
void plan_product(Product* p, int dtype, bool ta, bool tb, int loads, int groups);

}  // namespace muon
