// Host-only check of csrc/experts_bounds.hpp (built by
// tests/test_experts_bounds.py with g++): lists of units as the first launch
// writes them come out as they went in, every (unit, column tile) once, and no
// four words whatever give a unit outside this call's rows, experts and tiles.
#include <stdint.h>
#include <stdio.h>

#include <random>
#include <set>
#include <utility>
#include <vector>

#include "../block_scaled_mxfp4_bf16_amd/csrc/experts_bounds.hpp"

using namespace mxfp4;

#define CHECK(c)                                                   \
  do {                                                             \
    if (!(c)) {                                                    \
      fprintf(stderr, "check failed line %d: %s\n", __LINE__, #c); \
      return 1;                                                    \
    }                                                              \
  } while (0)

static std::mt19937 rng(7);
static int below(int n) { return (int)(rng() % (unsigned)n); }

static int wild() {
  switch (rng() % 4) {
    case 0: return (int)rng();
    case 1: return below(5000);
    case 2: return -below(5000);
    default: return (int)(rng() & 1 ? INT32_MAX - (int)(rng() % 3) : INT32_MIN + (int)(rng() % 3));
  }
}

static int own_lists() {
  for (int round = 0; round < 300; ++round) {
    const int E = 1 + below(40), unit_rows = rng() & 1 ? 128 : 16, n_tiles = 1 + below(9), block = 8;
    std::vector<int> words, rows_of;
    int R = 0, tile = 0;
    std::vector<int> size(E);
    for (int &n : size) R += n = below(3) ? below(300) : below(4000);
    if (R == 0) continue;
    int tiles = 0;
    for (int n : size) tiles += (n + 63) / 64 * 4;
    int row = 0;
    for (int e = 0; e < E; ++e) {
      for (int at = 0, i = 0; at < size[e]; at += unit_rows, ++i)
        words.insert(words.end(), {e + i * kMaxExperts, row + at, size[e] - at, tile + at / 16});
      row += size[e];
      tile += (size[e] + 63) / 64 * 4;
    }
    const int units = (int)words.size() / 4;
    std::vector<Unit> list;
    for (int u = 0; u < units; ++u) {
      const int *w = &words[4 * u];
      const Unit unit = unit_of(w[0], w[1], w[2], w[3], R, E, tiles, unit_rows);
      CHECK(unit.expert == (w[0] & 4095) && unit.row == w[1] && unit.rows == w[2] && unit.tile == w[3]);
      CHECK(unit.index == w[0] >> 12);
      list.push_back(unit);
    }
    std::set<std::pair<int, int>> seen;
    for (int item = 0; item < units * n_tiles; ++item) {
      const int u = item / n_tiles;
      const TilePlace p = tile_place(item, n_tiles, units, u, list[u].index, list[u].rows, unit_rows, block);
      CHECK(p.unit >= 0 && p.unit < units && p.column >= 0 && p.column < n_tiles);
      CHECK(list[p.unit].expert == list[u].expert);
      CHECK(seen.insert({p.unit, p.column}).second);
    }
  }
  return 0;
}

static int any_words() {
  int some = 0;
  for (int round = 0; round < 2000000; ++round) {
    const int R = 1 + below(5000), E = 1 + below(64), unit_rows = rng() & 1 ? 128 : 16;
    const int tiles = 4 * ((R + 63) / 64 + below(40));
    const auto near = [](int n) { return rng() % 8 ? below(n + n / 4 + 2) - 1 : wild(); };
    const int word = rng() % 8 ? below(E + 3) + (below(1 << 19) << 12) : wild();
    const Unit u = unit_of(word, near(R), near(R), near(tiles), R, E, tiles, unit_rows);
    some += u.expert >= 0 && u.rows > 0;
    const int64_t used = ((u.rows < unit_rows ? u.rows : unit_rows) + 15) / 16;
    CHECK(u.expert >= -1 && u.expert < E && (u.expert < 0) == (word < 0));
    CHECK(u.row >= 0 && u.rows >= 0 && (int64_t)u.row + u.rows <= R);
    CHECK(u.tile >= 0 && u.tile < tiles && (int64_t)u.tile + used <= tiles && (u.expert < 0 || u.index >= 0));
    const int units = 1 + below(900), n_tiles = 1 + below(200), item = below(units * n_tiles);
    // index and rows as an entry of another list may have them
    const TilePlace p = tile_place(item, n_tiles, units, item / n_tiles, below(1 << 19), below(1 << 20), unit_rows, 8);
    CHECK(p.unit >= 0 && p.unit < units && p.column >= 0 && p.column <= 8 * n_tiles);
  }
  CHECK(some > 1000);
  CHECK(within(-5, 0, 9) == 0 && within(11, 0, 9) == 9 && within(3, 0, 9) == 3);
  return 0;
}

int main() {
  if (own_lists() || any_words()) return 1;
  printf("bounds ok\n");
  return 0;
}
