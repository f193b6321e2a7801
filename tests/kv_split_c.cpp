// The arithmetic of csrc/kv_split.h for tests, built for the host.
#include "kv_split.h"

extern "C" {
int piece_begin(int at, int pieces, int tiles) { return bsg::piece_begin(at, pieces, tiles); }
int64_t context_positions(int window, int max_q, int max_kv) { return bsg::context_positions(window, max_q, max_kv); }
int line_fits(int64_t tokens, int group, int64_t seqs, int kv_heads, int64_t context) {
  return bsg::line_fits(tokens, group, seqs, kv_heads, context);
}
int unit_cost(void) { return bsg::kUnitCost; }
}
