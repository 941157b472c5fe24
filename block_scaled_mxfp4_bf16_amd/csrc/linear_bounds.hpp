// Where the dense layer's kernels read the prepared matrix, and how full their
// large tiles are.
//
// Buffers and the offsets into them are 32 bits, and bit 31 of an offset says
// that it is out of range, so every offset that an address is made of has to
// stay below 2^31: those of 16-row groups that a tile has past the matrix' last
// one, and of K steps past its end, as well.  A matrix holds up to 2^31 - 1
// bytes of codes, so a group further would be beyond.  Plain arithmetic, so that
// it is checked on the host.
#pragma once

#include <stdint.h>

namespace mxfp4 {

// The 16-row group that stands for group g of a tile: itself, or past the end
// the last one, whose sums are not stored.
constexpr int group_within(int g, int groups) { return g < groups ? g : groups - 1; }

// K steps of 128 that a large tile takes, in rounds of four.
constexpr int tile_steps(int64_t K) { return (int)(((K + 127) / 128 + 3) / 4 * 4); }

// Whether all of a large tile's offsets stay below 2^31: the last lane's 16
// bytes of the last group's codes in the last step.
constexpr bool tile_offsets_fit(int64_t N, int64_t K) {
  return (N / 16 - 1) * K * 8 + (int64_t)tile_steps(K) * 1024 <= INT32_MAX;
}

// Whether 256 x 256 tiles hold enough rows for the round or rounds that 256 CUs
// take them in.  A round lasts as long for one row as for 256, while the small tiles
// take longer with every 32 rows: as much as a round from 512 pieces of 32 x 256 on.
// us a call with large and small tiles, rows of N x 4096: N 32768, 17 rows 40 and
// 21, 64 rows (256 pieces) 40 and 28, 128 rows (512) 40 and 48; N 65536, 32 rows (256)
// 46 and 33, 64 rows (512) 47 and 54; N 131072 of 2048, two rounds, 32 rows (512)
// 56 and 34, 64 rows (1024) 57 and 54, 128 rows 60 and 94; gated the same within 10 %.
constexpr bool tiles_filled(int64_t M, int64_t N) {
  const int64_t n_tiles = (N + 255) / 256, tiles = (M + 255) / 256 * n_tiles;
  return (M + 31) / 32 * n_tiles >= 512 * ((tiles + 255) / 256);
}

}  // namespace mxfp4
