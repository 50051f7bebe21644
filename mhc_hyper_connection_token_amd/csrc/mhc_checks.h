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

// ---- checks of the 8-bit blocks' kind: types, codes with scales, several outputs ----
inline size_t blocks_of(size_t n) { return (n + 127) / 128; }

// The spans of a codes / scales pair; empty ones for a null pointer.
struct Pair {
  Span codes, scales;
};
inline Pair pair_span(const void* codes, const void* scales, size_t rows, size_t cols,
                      bool square) {
  if (!codes) return Pair{span(nullptr, 0), span(nullptr, 0)};
  const size_t kb = blocks_of(cols);
  return Pair{span(codes, rows * kb * 128),
              span(scales, (square ? blocks_of(rows) : rows) * kb)};
}

// Each of out[] apart from every in[] and from the other outputs.
inline int check_apart(const Span* out, int no, const Span* in, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int k = 0; k < ni; ++k)
      if (overlaps(out[i], in[k])) return MHC_EOVERLAP;
    for (int k = i + 1; k < no; ++k)
      if (overlaps(out[i], out[k])) return MHC_EOVERLAP;
  }
  return MHC_OK;
}

inline int check_ptrs(const void* const* ptrs, int n) {
  for (int i = 0; i < n; ++i)
    if (!ptrs[i]) return MHC_EINVAL;
  for (int i = 0; i < n; ++i)
    if (int rc = check_ptr(ptrs[i])) return rc;
  return MHC_OK;
}

// Span of [rows][H] kept in fp32, or as codes where scales are given.
inline Pair kept_span(const void* p, const unsigned char* scales, size_t rows, size_t H) {
  if (scales) return pair_span(p, scales, rows, H, false);
  return Pair{span(p, rows * H * 4), span(nullptr, 0)};
}

}  // namespace mhc
