// How the products in E4M3 beyond 16 tokens (f8_tiled.hip, f8_pp.hip) are cut into tiles and parts of K, on the host: the kernel
// and the number of parts that take the least time by what was measured.
#pragma once

#include <stdint.h>

namespace bsg {

// The kernels' shapes of tiles: weight rows x tokens.  Gated ones hold gate's and up's rows of half as many outputs.  Wide:
// products of widened codes.
enum class F8Way : int {
  T64x32, T64x64, T128x64, T128x128, G256x32Wide, G256x64Wide, G256x64, G256x128, T64x32Wide, T64x64Wide, T128x128Wide,
  T256x256, G256x256
};

// What a shape of tile takes, in microseconds: to begin and end, a step with one workgroup on a CU and with per_cu, and joining
// parts (join + s join_each).  Measured with 61 to 2048 tokens, n and k of 512 to 8192.
struct F8Shape {
  int rows, tokens, per_cu;
  bool gated;
  double begin, step_alone, step_full, join, join_each;
};
constexpr F8Shape kF8Shapes[] = {
    {64, 32, 3, false, 3.4, 0.25, 0.42, 1.4, 0.5},    {64, 64, 3, false, 3.5, 0.33, 0.58, 1.6, 0.8},
    {128, 64, 2, false, 4.1, 0.43, 0.73, 1.0, 1.15},  {128, 128, 1, false, 4.8, 0.62, 0.62, 1.8, 1.4},
    {256, 32, 1, true, 4.5, 0.6, 0.6, 1.2, 0.8},      {256, 64, 1, true, 5.0, 1.0, 1.0, 1.5, 1.2},
    {256, 64, 1, true, 5.0, 0.78, 0.78, 1.5, 1.2},    {256, 128, 1, true, 6.0, 1.05, 1.05, 2.5, 2.5},
    {64, 32, 3, false, 3.4, 0.40, 0.65, 1.4, 0.5},    {64, 64, 3, false, 3.5, 0.52, 0.95, 1.6, 0.8},
    {128, 128, 1, false, 4.8, 1.15, 1.15, 1.8, 1.4},
};
constexpr const F8Shape& f8_shape(F8Way way) { return kF8Shapes[(int)way]; }  // (all but the last two)
constexpr double kF8BytesPerUs = 4.8e6;  // of weights that come from memory
constexpr int kF8WideTokens = 64;        // up to so many, gated products are of widened codes

struct F8Cut {
  F8Way way;
  int64_t tiles, splits;
  double cost;
};

inline int64_t f8_tiles(int rows, int cols, bool gated, int64_t tokens, int64_t n) {
  const int outs = gated ? rows / 2 : rows;
  return (tokens + cols - 1) / cols * ((n + outs - 1) / outs);
}

// The number of parts of K that takes the least time: at least four blocks a part, and all parts' workgroups run at once.
inline F8Cut f8_cut_of(F8Way way, int64_t tokens, int64_t n, int64_t k, int cus) {
  const F8Shape& t = f8_shape(way);
  const int64_t kb = (k + 127) / 128, fill = (int64_t)cus * t.per_cu;
  const double memory = (t.gated ? 2.0 : 1.0) * (double)n * (double)k / kF8BytesPerUs;
  F8Cut best = {way, f8_tiles(t.rows, t.tokens, t.gated, tokens, n), 1, 0};
  for (int64_t s = 1; s == 1 || (s <= kb / 4 && best.tiles * s <= fill); ++s) {
    const int64_t wgs = best.tiles * s, per_cu = wgs >= fill ? t.per_cu : (wgs + cus - 1) / cus, rounds = (wgs + fill - 1) / fill;
    const double step = t.per_cu == 1 ? t.step_full : t.step_alone + (t.step_full - t.step_alone) * (per_cu - 1) / (t.per_cu - 1);
    const double work = (double)(rounds * ((kb + s - 1) / s)) * step;
    const double cost = t.begin + (work > memory ? work : memory) + (s > 1 ? t.join + s * t.join_each : 0);
    if (s == 1 || cost < best.cost) {
      best.cost = cost;
      best.splits = s;
    }
  }
  return best;
}

// The same of the kernel for many tokens (f8_pp.hip): a step takes longer where all CUs work at once.
inline F8Cut f8_cut_large(bool gated, int64_t tokens, int64_t n, int64_t k, int cus) {
  const int64_t tiles = f8_tiles(256, 256, gated, tokens, n), kb = (k + 127) / 128;
  const double busy = tiles >= cus ? 1.0 : (double)tiles / cus;
  return {gated ? F8Way::G256x256 : F8Way::T256x256, tiles, 1,
          8 + (double)((tiles + cus - 1) / cus * kb) * (1.15 + (busy > 0.5 ? (busy - 0.5) * 1.1 : 0.0))};
}

// The way of a call of more than 16 tokens.  exact: by products of widened codes, however many tokens.
inline F8Cut f8_cut(bool gated, bool exact, int64_t tokens, int64_t n, int64_t k, int cus) {
  auto of = [&](F8Way way) { return f8_cut_of(way, tokens, n, k, cus); };
  if (tokens <= 32) return of(gated ? F8Way::G256x32Wide : exact ? F8Way::T64x32Wide : F8Way::T64x32);
  if (gated && (exact || tokens <= kF8WideTokens)) return of(F8Way::G256x64Wide);
  F8Cut best = of(gated ? F8Way::G256x64 : exact ? F8Way::T64x64Wide : F8Way::T64x64);
  auto take = [&](const F8Cut& c, bool even) {  // (a larger tile also where it takes as long)
    if (c.cost < best.cost || (even && c.cost == best.cost)) best = c;
  };
  if (exact) {
    take(of(F8Way::T128x128Wide), true);
    return best;
  }
  if (!gated) take(of(F8Way::T128x64), true);
  take(of(gated ? F8Way::G256x128 : F8Way::T128x128), true);
  take(f8_cut_large(gated, tokens, n, k, cus), false);
  return best;
}

// Tokens that one grid of such tiles can take: whole tiles, of which there are no more than 2^31 threads' worth.
inline int64_t f8_tokens_at_once(F8Way way, int64_t n, int threads) {
  const F8Shape& t = f8_shape(way);
  return ((int64_t)1 << 31) / threads / f8_tiles(t.rows, t.tokens, t.gated, 1, n) * t.tokens;
}

// What calls of up to max_tokens may need for parts of K, in floats, and how many tiles they count.
struct F8Parts {
  int64_t floats, counters;
};
inline F8Parts f8_parts(bool gated, bool exact, int64_t max_tokens, int64_t n, int64_t k, int cus) {
  F8Parts most = {0, 0};
  if (max_tokens <= 16) return most;
  const int64_t pieces = (k + 127) / 128 / 4;
  const F8Way first = gated ? F8Way::G256x32Wide : exact ? F8Way::T64x32Wide : F8Way::T64x32;
  const F8Way last = gated ? exact ? F8Way::G256x64Wide : F8Way::G256x128 : exact ? F8Way::T128x128Wide : F8Way::T128x128;
  for (int way = (int)first; way <= (int)last; ++way) {
    const F8Shape& t = kF8Shapes[way];
    const int64_t limit = way == (int)first ? 32 : way == (int)F8Way::G256x64Wide && !exact ? kF8WideTokens : max_tokens;
    for (int64_t tokens = 1; tokens <= max_tokens && tokens <= limit; tokens += t.tokens) {  // row after row of tiles
      const int64_t tiles = f8_tiles(t.rows, t.tokens, gated, tokens, n), fit = (int64_t)cus * t.per_cu / tiles;
      const int64_t splits = fit < pieces ? fit : pieces;
      if (splits < 2) break;  // (more tiles have no more)
      const int64_t floats = tiles * splits * t.rows * t.tokens;
      if (floats > most.floats) most.floats = floats;
      if (tiles > most.counters) most.counters = tiles;
    }
  }
  return most;
}

}  // namespace bsg
