// What the kernels take out of a workspace, held to this call's own sizes.
//
// The first launch of the grouped product and of the router leaves numbers
// in the workspace that the second turns into addresses.  They are its own
// unless calls share a workspace at the same time, which callers must not
// do; where they do (graphs captured on one stream and replayed on two, say)
// the results have no meaning, but nothing outside the buffers may be
// touched.  Plain arithmetic, so that it is checked on the host.
#pragma once

namespace mxfp4 {

constexpr int within(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// A run of rows of one expert.
struct Unit {
  int expert;  // -1: none
  int row;     // first output row
  int rows;    // output rows from `row` to the end of the group
  int tile;    // its first 16-row tile in the workspace
  int index;   // its number among the expert's units
};

// An entry's first word holds the expert and, above it, the unit's number
// among the expert's (at most 2^20 rows of 16 a unit: 17 bits).
constexpr int kExpertBits = 12, kMaxExperts = 1 << kExpertBits;

// The unit that an entry of four words describes, brought within R rows, E
// experts and `tiles` tiles in the workspace (at least as many as R rows take).
// Minima only: a test of each word, and no unit if one failed, made the short
// products 3 % slower.
constexpr Unit unit_of(int first, int row, int rows, int tile, int R, int E, int tiles, int unit_rows) {
  const unsigned expert = first & (kMaxExperts - 1), last = E - 1;
  const int at = (unsigned)row < (unsigned)R ? row : R;
  const int n = within(rows, 0, R - at);
  const int used = ((n < unit_rows ? n : unit_rows) + 15) >> 4;
  const int most = tiles - (used > 1 ? used : 1);
  return Unit{first < 0 ? -1 : (int)(expert < last ? expert : last), at, n,
              (unsigned)tile < (unsigned)most ? tile : most, first >> kExpertBits};
}

// A unit in the list and one of its column tiles.
struct TilePlace {
  int unit, column;
};

// Item `item` of units x n_tiles, u = item / n_tiles its unit in plain order:
// the units of an expert are taken in blocks of up to `block_units`, the unit
// fastest within a block.  `index` and `rows` are those of unit u.
constexpr TilePlace tile_place(int item, int n_tiles, int units, int u, int index, int rows, int unit_rows,
                               int block_units) {
  const int first = within(u - index, 0, units - 1);  // the expert's first unit
  const int all = index + (rows + unit_rows - 1) / unit_rows;
  const int listed = within(all, 1, units - first);
  const int in_expert = item - first * n_tiles;
  const int block = in_expert / (block_units * n_tiles);
  const int in_block = in_expert - block * block_units * n_tiles;
  const int width = within(listed - block_units * block, 1, block_units);
  const int column = in_block / width;
  return TilePlace{within(first + block_units * block + in_block - column * width, 0, units - 1), column};
}

}  // namespace mxfp4
