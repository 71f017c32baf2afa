// Checks of a C entry's arguments that the operators' entries share (host only).
#pragma once

#include <stdint.h>

#include "../../include/gdn.h"
#include "gdn_internal.h"

namespace gdn {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

// A bf16 operand of `tokens` rows of `width` elements: GDN_OK, or what is wrong with it.
inline int check_rows(const void* p, long long stride, long long tokens, long long width) {
  if (p == nullptr) return GDN_ERR_ARG;
  if (tokens > 1 && stride < width) return GDN_ERR_ARG;
  if (!aligned(p, 16) || (tokens > 1 && stride % 8 != 0)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

inline int done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : set_cuda_error(e, GDN_ERR_LAUNCH); }

}  // namespace gdn
