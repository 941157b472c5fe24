// Where the dense layer's kernels read the prepared matrix.
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

}  // namespace mxfp4
