// Argument checks that the entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/mxfp4.h"
#include "mxfp4_internal.hpp"

namespace mxfp4 {

constexpr int64_t kMaxBytes = (int64_t)1 << 31;  // 32-bit offsets inside the kernels
constexpr int64_t kMaxRows = (int64_t)1 << 20;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int64_t pad_to(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline bool known_type(int t) { return t == MXFP4_TYPE_BF16 || t == MXFP4_TYPE_F16 || t == MXFP4_TYPE_F32; }

inline int64_t size_of(int t) { return t == MXFP4_TYPE_F32 ? 4 : 2; }

// Whether 32-bit offsets reach all of one prepared matrix; sizes are
// compared by division, so that no product overflows.
inline bool matrix_fits(int64_t N, int64_t K) {
  if (N >= kMaxBytes || K >= kMaxBytes) return false;
  return N <= (kMaxBytes - 1) / ((K + 1) / 2) && pad_to(N, 256) <= (kMaxBytes - 1) / pad_to(K / 32 + 1, 8);
}

// The caller's workspace if it gave one, else the library's, behind the
// ticket words that the split-K products keep at zero; `held` keeps that one
// for this call while it lives.
inline mxfp4_status_t take_workspace(void *given, size_t given_bytes, size_t need, hipStream_t stream,
                                     HeldWorkspace *held, void **out) {
  *out = given;
  if (given) return given_bytes >= need && aligned(given, 256) ? MXFP4_OK : MXFP4_ERR_WORKSPACE;
  if (need == 0) return MXFP4_OK;
  const mxfp4_status_t st = hold_workspace(kTicketBytes + need, stream, held);
  if (st == MXFP4_OK) *out = (char *)held->ptr + kTicketBytes;
  return st;
}

}  // namespace mxfp4
