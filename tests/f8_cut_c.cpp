// The choice of csrc/f8_cut.h for tests, built for the host.  gated: 1, and 2 for exact products.
#include "f8_cut.h"

extern "C" {
int cut(int gated, int64_t tokens, int64_t n, int64_t k, int cus, int64_t out[3], double* cost) {
  const bsg::F8Cut c = bsg::f8_cut(gated & 1, gated >> 1, tokens, n, k, cus);
  out[0] = (int)c.way;
  out[1] = c.tiles;
  out[2] = c.splits;
  *cost = c.cost;
  return 0;
}
int64_t tokens_at_once(int way, int64_t n, int threads) { return bsg::f8_tokens_at_once((bsg::F8Way)way, n, threads); }
void parts(int gated, int64_t max_tokens, int64_t n, int64_t k, int cus, int64_t out[2]) {
  const bsg::F8Parts p = bsg::f8_parts(gated & 1, gated >> 1, max_tokens, n, k, cus);
  out[0] = p.floats;
  out[1] = p.counters;
}
}
