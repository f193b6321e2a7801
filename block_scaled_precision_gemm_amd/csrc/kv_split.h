// How attention's work is cut: arithmetic that host and kernels share, free of HIP so that it can be checked without a
// GPU at the largest arguments that a call may have.
#pragma once

#include <stdint.h>

namespace bsg {

constexpr int kTile = 64;  // positions of a tile
// What a unit (a block of query rows of one sequence and key/value head) costs a workgroup of the few-row kernel besides
// its tiles, in tiles: queries, the pipeline's filling, joining the waves (measured with 64 contexts up to 16384: 10 us
// for each further unit of a run, 0.7 us per tile).
constexpr int kUnitCost = 12;

// Positions that some row of a sequence sees, at most: 16 more than window and new tokens, spans starting at multiples of 16.
constexpr int64_t context_positions(int window, int max_q, int max_kv) {
  const int64_t seen = window > 0 ? (int64_t)window + max_q + 16 : max_kv;
  return seen < max_kv ? seen : max_kv;
}

// Whether the few-row kernel's 32-bit counts hold a call: the line of all units' tiles and fixed costs, and what is added
// to it (workgroups, at most one more run).  A sequence has at most one block that is not full, of 16 rows and more.
constexpr bool line_fits(int64_t tokens, int group, int64_t seqs, int kv_heads, int64_t context) {
  const int64_t units = (tokens * group / 16 + seqs) * kv_heads;
  return units * (context / kTile + 2 + kUnitCost) < ((int64_t)1 << 31) - (1 << 20);
}

// First tile of piece `at` of `pieces` (the end of piece at - 1): floor(at * tiles / pieces) without forming at * tiles,
// which passes 2^31 (511 pieces of 2^28 positions and more).  Pieces are one per workgroup at most, so at * pieces is small.
constexpr int piece_begin(int at, int pieces, int tiles) {
  return at * (tiles / pieces) + at * (tiles % pieces) / pieces;
}

}  // namespace bsg
