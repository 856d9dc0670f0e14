// Place of a work item in its group (host and device: constexpr).
#pragma once

namespace moe {

struct Item {
  int g;      // group
  int m0;     // first row of the tile inside the group
  int rows;   // valid rows in the tile
  int n;      // column tile
  int grows;  // rows of the group
};

// A group's row tiles are taken in bands of up to kBand tiles; a
// band's items run column tile outer, row tile inner.  Routed experts at
// large batch have a few row tiles (one band: each weight tile is read from
// HBM once while all of the expert's rows use it); the shared experts'
// many row tiles go band by band, so the workgroups running together on an
// XCD share both activation and weight tiles.
constexpr int kBand = 8;

// Rows of a group's balanced row tiles: 32 * ceil(grows / (32 mt)) for its grows
// rows in mt tiles (grows > 0).  Taken from the blocks of 32 rows: grows + 32 mt
// passes 2^31 from 1.91e9 rows (tiles of 256) or 1.72e9 (of 128) on.
constexpr int balanced_rows(int grows, int mt) { return ((grows - 1) / 32 / mt + 1) * 32; }

// Item `it`, which lies in group g of grows rows.
__attribute__((always_inline)) constexpr Item place_item(long long it, const int* ts, int g,
                                                         int n_tiles, int MT, int grows,
                                                         bool balanced) {
  Item r{};
  r.g = g;
  r.grows = grows;
  const int mt = ts[g + 1] - ts[g];
  const int local = static_cast<int>(it - static_cast<long long>(ts[g]) * n_tiles);
  const int band = mt < kBand ? mt : kBand;
  const int full = mt / band;
  const int in_full = full * band * n_tiles;
  int m = 0;
  if (local < in_full) {
    const int b = local / (band * n_tiles);
    const int rem = local - b * band * n_tiles;
    r.n = rem / band;
    m = b * band + rem % band;
  } else {
    const int last = mt - full * band;
    const int rem = local - in_full;
    r.n = rem / last;
    m = full * band + rem % last;
  }
  const int base = balanced ? balanced_rows(grows, mt) : MT;
  r.m0 = m * base;
  const int left = grows - r.m0;
  r.rows = left < base ? left : base;
  return r;
}

}  // namespace moe
