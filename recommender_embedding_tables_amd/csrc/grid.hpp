// Grids of many blocks.  Plain C++ (a host test includes it).
#pragma once

#include <cstdint>

namespace embtab {

// A launch holds fewer than 2^32 threads along x: a kernel of 256 threads a
// block goes along y too from kGridX blocks on.  Blocks past the last one are
// launched then; the kernels leave them without work.
constexpr int64_t kGridX = 1 << 23;

struct Grid {
  unsigned x, y;
};

inline Grid fold_grid(int64_t blocks) {
  if (blocks <= kGridX) return {(unsigned)blocks, 1u};
  return {(unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX)};
}

}  // namespace embtab
