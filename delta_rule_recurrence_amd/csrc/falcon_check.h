// Host-side argument checks shared by the C ABI's sources.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "falcon.h"

namespace falcon {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// Largest element count of one tensor; every index then fits an int64_t with
// room to spare, and every grid its 32 bits.
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Most tokens of one call: token indices and what is added to them fit an int.
constexpr int64_t kMaxTokens = int64_t(1) << 30;

// a b c (each >= 0), or -1 beyond kMaxElems.
inline int64_t elems(int64_t a, int64_t b, int64_t c = 1) {
  const __int128 n = static_cast<__int128>(a) * b * c;
  return n > kMaxElems ? -1 : static_cast<int64_t>(n);
}

inline bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return false;
  return true;
}

// True when any of `outs` overlaps another of them or one of `ins`.
inline bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* a = outs.begin(); a != outs.end(); ++a) {
    for (const Range* b = a + 1; b != outs.end(); ++b)
      if (overlap(*a, *b)) return true;
    for (const Range& r : ins)
      if (overlap(*a, r)) return true;
  }
  return false;
}

// Bytes from the first to the last element of `rows` rows.
inline int64_t rows_bytes(int64_t rows, int64_t row, int64_t width, int64_t es) {
  return rows > 0 && width > 0 ? ((rows - 1) * row + width) * es : 0;
}

// Whether `rows` rows of `width` elements, `row` apart, are valid.
inline bool rows_ok(int64_t rows, int64_t row, int64_t width) {
  return row >= width && row <= (int64_t(1) << 31) && elems(rows, row) >= 0;
}

inline bool dtype_ok(int32_t t) { return t == FALCON_F32 || t == FALCON_BF16; }
inline int64_t dtype_bytes(int32_t t) { return t == FALCON_BF16 ? 2 : 4; }

inline falcon_status finish(hipError_t e) { return e == hipSuccess ? FALCON_OK : FALCON_ERR_HIP; }

}  // namespace falcon
