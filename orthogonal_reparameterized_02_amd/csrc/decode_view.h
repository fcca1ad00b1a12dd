// The rows of a cache that the query of one sequence sees, as up to three runs
// of neighbouring rows: the sinks, the window, and where the cache is a ring
// what of the window lies behind its end.  A run is padded to tiles, so that a
// tile lies in one run; `rows` numbers the padded rows through.
//
// A ring of `rows` rows holds position p in row p for p < sinks and in row
// sinks + (p - sinks) mod (rows - sinks) from there on; the window is at most
// rows - sinks.
#pragma once

#include "attn.h"

namespace poetx {

struct View {
  int last;            // position of the query
  int n0, n1, n2;      // rows of the runs
  int r1, lo, s;       // first row of the window, its position, first row behind the ring's end
  int t0, t1, total;   // padded rows: sinks, window, all

  // TILE rows a tile; ALIGN: tiles begin at multiples of TILE in the cache
  template <int TILE, bool ALIGN> __device__ __forceinline__ void init(const DecodeArgs& a, int len, int start) {
    const int hi = a.ring ? max(len, 0) : min(max(len, 0), a.rows);
    lo = min(max(start, 0), hi);
    if (a.window) lo = max(hi - a.window, 0);
    last = hi - 1;
    n0 = a.window ? min(a.sinks, lo) : 0;
    s = a.sinks;
    r1 = lo, n1 = hi - lo, n2 = 0;
    if (a.ring && lo >= a.sinks) {
      r1 = a.sinks + (lo - a.sinks) % (a.rows - a.sinks);
      n1 = min(hi - lo, a.rows - r1);
      n2 = hi - lo - n1;
    }
    const auto padded = [](int row, int n) {
      if (n == 0) return 0;
      const int first = ALIGN ? row % TILE : 0;
      return (first + n + TILE - 1) / TILE * TILE;
    };
    t0 = padded(0, n0);
    t1 = padded(r1, n1);
    total = t0 + t1 + padded(s, n2);
  }
  // the tile that begins at padded row v: its first row in the cache, the rows
  // [begin, end) of it that are seen, and position less row
  template <int TILE, bool ALIGN> __device__ __forceinline__ void tile(int v, int& row, int& begin, int& end, int& shift) const {
    const int run = v < t0 ? 0 : v < t0 + t1 ? 1 : 2;
    begin = run == 0 ? 0 : run == 1 ? r1 : s;
    end = begin + (run == 0 ? n0 : run == 1 ? n1 : n2);
    shift = run == 0 ? 0 : run == 1 ? lo - r1 : lo + n1 - s;
    row = (ALIGN ? begin / TILE * TILE : begin) + v - (run == 0 ? 0 : run == 1 ? t0 : t0 + t1);
    begin = max(begin, row);
    end = min(end, row + TILE);
  }
};

// rows that a sequence of the cache may see at most, with their padding
inline long view_rows(const DecodeArgs& a, int tile) {
  return a.window ? std::min((long)a.rows, (long)a.window + a.sinks) + 3L * tile : a.rows;
}

}  // namespace poetx
