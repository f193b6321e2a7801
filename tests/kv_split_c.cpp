// The arithmetic of csrc/kv_split.h for tests, built for the host.
#include "kv_split.h"

extern "C" {
int piece_begin(int at, int pieces, int tiles) { return bsg::piece_begin(at, pieces, tiles); }
}
