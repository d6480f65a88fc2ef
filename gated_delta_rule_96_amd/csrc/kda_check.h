// Host-side argument checks shared by the C ABI's translation units.
#pragma once
#include <hip/hip_runtime.h>
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

// Tokens of a sequence at most.
constexpr int kMaxT = 1 << 30;

// A span of memory an argument covers.
struct Span {
  const void* p;
  size_t n;
};
// Whether an output overlaps an input or another output; an output that
// starts where inputs[same] starts and covers the same bytes is that input
// replaced in place (same < 0: never).
template <int NI, int NO>
bool spans_apart(const Span (&in)[NI], const Span (&out)[NO], const int (&same)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i) {
      if (i == same[o] && in[i].p == out[o].p && in[i].n == out[o].n) continue;
      if (overlap(in[i].p, in[i].n, out[o].p, out[o].n)) return false;
    }
    for (int k = 0; k < o; ++k)
      if (overlap(out[k].p, out[k].n, out[o].p, out[o].n)) return false;
  }
  return true;
}
// Bytes from the first to the last element of `rows` rows of n elements, ld
// apart.
inline size_t rows_bytes(size_t rows, long long ld, size_t n, size_t esz) { return ((rows - 1) * (size_t)ld + n) * esz; }

inline int check_cu(const int* cu, int N, int B, int T) {
  if (!cu) return KDA_OK;
  if (B != 1 || N <= 0 || cu[0] != 0 || cu[N] != T) return KDA_ERR_SHAPE;
  for (int i = 0; i < N; ++i)
    if (cu[i + 1] < cu[i]) return KDA_ERR_SHAPE;
  return KDA_OK;
}

// (hipErrorInvalidConfiguration: sizes beyond a launch's, see max_groups)
inline int hip_status(hipError_t e) {
  return e == hipSuccess ? KDA_OK : e == hipErrorInvalidConfiguration ? KDA_ERR_SHAPE : KDA_ERR_HIP;
}

}  // namespace kda
