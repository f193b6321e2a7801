// How attention's work is cut: arithmetic that host and kernels share, free of HIP so that it can be checked without a
// GPU at the largest arguments that a call may have.
#pragma once

#include <stdint.h>

namespace bsg {

// First tile of piece `at` of `pieces` (the end of piece at - 1): floor(at * tiles / pieces) without forming at * tiles,
// which passes 2^31 (511 pieces of 2^28 positions and more).  Pieces are one per workgroup at most, so at * pieces is small.
constexpr int piece_begin(int at, int pieces, int tiles) {
  return at * (tiles / pieces) + at * (tiles % pieces) / pieces;
}

}  // namespace bsg
