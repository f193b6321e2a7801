// How attention's work is cut: arithmetic that host and kernels share, free of HIP so that it can be checked without a
// GPU at the largest arguments that a call may have.
#pragma once

#include <stdint.h>

namespace bsg {

constexpr int kTile = 64;     // positions of a tile
constexpr int kFewRows = 32;  // most query rows per sequence and key/value head of the few-row kernel
// What a unit (a block of query rows of one sequence and key/value head) costs a workgroup of the few-row kernel besides
// its tiles, in tiles: queries, the pipeline's filling, joining the waves (measured with 64 contexts up to 16384: 10 us
// for each further unit of a run, 0.7 us per tile).
constexpr int kUnitCost = 12;

// A window that no context reaches (max_kv is at most 2^30) is none: differences of positions and window stay in 32 bits.
constexpr int kept_window(int window) { return window >= 1 << 30 ? 0 : window; }

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

// Rows of a workgroup of the many-row kernel: 8 waves of 32 halve the decoding per row; 4 where no sequence fills more.
constexpr int rows_waves(int max_q, int group) { return (int64_t)max_q * group > 128 ? 8 : 4; }

// Slots of row blocks where they are listed: sequence b's first.  From one sequence to the next they grow by at least
// its blocks, ceil(new tokens * group / rows), so b is found from a slot by searching the starts, without a sum over
// the sequences before it; a slot beyond its sequence's blocks has none.
constexpr int row_slot(int start, int b, int group, int rows) { return start * group / rows + b; }

// The many-row kernel's workgroups: `groups` of `width` blocks of `rows` rows.  Even batches: a group for each sequence and
// head, as wide as the longest sequence.  Uneven ones, where that would be more than twice the blocks that can exist
// (the rest only find that they have none): a group for each head, with all sequences' blocks listed.  32 heads on 8 of
// 128 dims, by groups of a sequence and listed: 8192 tokens beside 127 single ones 1034 and 736 us, 2048 beside 63 276 and
// 256 us, one of 2048 and seven of 100 143 and 125 us; 64 x 64 tokens, where the list has a slot too many for each
// sequence, 378 and 619 us.
struct RowsGrid {
  bool listed;
  int64_t groups, width;
};
constexpr RowsGrid rows_grid(int rows, int64_t tokens, int64_t seqs, int max_q, int group, int kv_heads) {
  const int64_t longest = ((int64_t)max_q * group + rows - 1) / rows, slots = tokens * group / rows + seqs;
  if (longest * seqs > 2 * slots) return {true, kv_heads, slots};
  return {false, seqs * kv_heads, longest};
}

// One token and whole prompts may share a batch: whether sequences of up to kFewRows rows are left to the few-row kernel
// (kv_attend_launch).
constexpr bool mixed_batch(int64_t tokens, int64_t seqs, int max_q, int group) {
  return group <= kFewRows && (int64_t)max_q * group > kFewRows && tokens < seqs * max_q &&
         (seqs >= 8 || (tokens - max_q) * group <= kFewRows * (seqs - 1));
}

// Whether the kernels that a call takes can count its work, and be launched: at most 2^32 - 1 threads in a grid.
constexpr bool attend_fits(int64_t tokens, int64_t seqs, int max_q, int group, int kv_heads, int64_t context) {
  if ((int64_t)max_q * group <= kFewRows) return line_fits(tokens, group, seqs, kv_heads, context);
  const int waves = rows_waves(max_q, group);
  const RowsGrid grid = rows_grid(32 * waves, tokens, seqs, max_q, group, kv_heads);
  if (grid.groups * grid.width * (64 * waves) >= (int64_t)1 << 32) return false;
  // whatever the starts say, a sequence is given to the few-row kernel with kFewRows rows at most
  const int64_t few = seqs * kFewRows / group;
  return !mixed_batch(tokens, seqs, max_q, group) || line_fits(few, group, seqs, kv_heads, context);
}

// First tile of piece `at` of `pieces` (the end of piece at - 1): floor(at * tiles / pieces) without forming at * tiles,
// which passes 2^31 (511 pieces of 2^28 positions and more).  Pieces are one per workgroup at most, so at * pieces is small.
constexpr int piece_begin(int at, int pieces, int tiles) {
  return at * (tiles / pieces) + at * (tiles % pieces) / pieces;
}

}  // namespace bsg
