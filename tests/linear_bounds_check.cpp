// Host-only check of csrc/linear_bounds.hpp (built by tests/test_linear_bounds.py
// with g++): over all sizes of the dense layer whose prepared matrix lies near
// its limit, the offsets that a large tile reads codes at stay below 2^31, and
// they are those of the group itself wherever there is one.
#include <stdint.h>
#include <stdio.h>

#include "../block_scaled_mxfp4_bf16_amd/csrc/linear_bounds.hpp"

using namespace mxfp4;

#define CHECK(c)                                                                                       \
  do {                                                                                                 \
    if (!(c)) {                                                                                        \
      fprintf(stderr, "check failed line %d: %s (N %lld, K %lld)\n", __LINE__, #c, (long long)N, (long long)K); \
      return 1;                                                                                        \
    }                                                                                                  \
  } while (0)

int main() {
  const int64_t kMaxBytes = (int64_t)1 << 31, kMaxN = (int64_t)1 << 20, kMaxK = (int64_t)1 << 17;
  int64_t beyond = 0, refused = 0, taken = 0;
  for (int64_t K = 32; K <= kMaxK; K += 32) {
    int64_t most = (kMaxBytes - 1) / (K / 2) / 16 * 16;
    if (most > kMaxN) most = kMaxN;
    for (int64_t N = most; N > most - 512 && N >= 16; N -= 16) {
      const int groups = (int)(N / 16), k = (int)K;
      const int steps = tile_steps(K);
      CHECK(steps % 4 == 0 && steps * 128 >= K && (steps - 4) * 128 < K);
      if (!tile_offsets_fit(N, K)) {
        CHECK(groups * K * 8 + 4096 > kMaxBytes);  // none but the very largest
        ++refused;
        continue;
      }
      ++taken;
      // the last tile's groups: a gated one's up rows begin at half of the groups
      const int plain_end = (int)((N + 255) / 256 * 16), gated_end = groups / 2 + (int)((N / 2 + 127) / 128 * 8);
      for (int g = groups - 20 < 0 ? 0 : groups - 20; g < (plain_end > gated_end ? plain_end : gated_end); ++g) {
        beyond += (int64_t)g * K * 8 >= kMaxBytes;
        const int at = group_within(g, groups) * k * 8;  // as the kernel has it, in 32 bits
        CHECK(at >= 0 && (g < groups ? at == (int64_t)g * K * 8 : at == (int64_t)(groups - 1) * K * 8));
        const int last = at + (steps - 1) * 1024;
        CHECK((int64_t)last + 63 * 16 + 15 < kMaxBytes && last >= at);
      }
    }
  }
  const int64_t N = 0, K = 0;
  CHECK(beyond > 1000 && refused > 0 && taken > 10000);  // groups whose own offset would be beyond are among them
  printf("bounds ok\n");
  return 0;
}
