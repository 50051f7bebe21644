// mhc_checks.h -- the host-side argument checks that every entry point shares.
#pragma once
#include <cstddef>
#include <cstdint>

#include "mhc.h"

namespace mhc {

constexpr long kMaxElems = 1L << 31;  // T*S*H must stay below this (int indexing)
constexpr int kMaxTokens = 1 << 23;   // bounds the flattened launch grids

inline int check_ptr(const void* p) {
  if (!p) return MHC_EINVAL;
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return MHC_EALIGN;
  return MHC_OK;
}

struct Span {
  uintptr_t lo, hi;
};
inline Span span(const void* p, size_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}
inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline int check_shape(int T, int S, int H) {
  if (T < 0 || S < 1 || H < 1) return MHC_EINVAL;
  if (S > 8) return MHC_EUNSUPPORTED;
  if (H % 4 != 0) return MHC_EALIGN;
  if ((long)T * S * H >= kMaxElems || T >= kMaxTokens) return MHC_EUNSUPPORTED;
  return MHC_OK;
}

}  // namespace mhc
