// Host-side argument checks shared by the C ABI's translation units.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

constexpr int kChunk = 64;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool supported_d(int d) { return d == 64 || d == 128; }
inline bool valid_dtype(int dt) { return dt == KDA_F32 || dt == KDA_BF16; }
inline size_t elem_size(int dt) { return dt == KDA_BF16 ? 2 : 4; }

// Largest element count of any [B, T, H, d] tensor accepted (64-bit offsets
// are used throughout; this only rejects sizes whose byte count overflows).
inline bool size_ok(long long a, long long b, long long c, long long d) {
  const long long lim = (1LL << 62);
  long long x = a;
  for (long long y : {b, c, d}) {
    if (y <= 0 || x > lim / y) return false;
    x *= y;
  }
  return true;
}

// Whether [a, a + na) and [b, b + nb) share a byte (NULL: no).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace kda
