// The arithmetic of csrc/kv_split.h for tests, built for the host.
#include "kv_split.h"

extern "C" {
int piece_begin(int at, int pieces, int tiles) { return bsg::piece_begin(at, pieces, tiles); }
int kept_window(int window) { return bsg::kept_window(window); }
int64_t context_positions(int window, int max_q, int max_kv) { return bsg::context_positions(window, max_q, max_kv); }
int line_fits(int64_t tokens, int group, int64_t seqs, int kv_heads, int64_t context) {
  return bsg::line_fits(tokens, group, seqs, kv_heads, context);
}
void rows_grid(int rows, int64_t tokens, int64_t seqs, int max_q, int group, int kv_heads, int64_t out[3]) {
  const bsg::RowsGrid g = bsg::rows_grid(rows, tokens, seqs, max_q, group, kv_heads);
  out[0] = g.listed;
  out[1] = g.groups;
  out[2] = g.width;
}
int row_slot(int start, int b, int group, int rows) { return bsg::row_slot(start, b, group, rows); }
int attend_fits(int64_t tokens, int64_t seqs, int max_q, int group, int kv_heads, int64_t context) {
  return bsg::attend_fits(tokens, seqs, max_q, group, kv_heads, context);
}
int unit_cost(void) { return bsg::kUnitCost; }
}
