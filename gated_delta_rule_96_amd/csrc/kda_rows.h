// Rows of channels as fp32 vectors, and the sequences of a launch: shared by
// the kernels that walk tokens (short convolution, head norms, state space
// scan).
#pragma once
#include "kda_device.h"
#include "kda_launch.h"

namespace kda {

// N consecutive elements of type T as fp32, and back (RNE).  N = 8 or 4: one
// or two 16-byte (or one 8-byte) accesses, the pointer aligned accordingly;
// N = 1: one element.  (Eight are read as fp32 only.)
template <typename T, int N> struct Rows;
template <typename T> struct Rows<T, 1> {
  static __device__ __forceinline__ void load(const T* p, float (&x)[1]) { x[0] = to_f32(*p); }
  static __device__ __forceinline__ void store(T* p, const float (&x)[1]) { *p = from_f32<T>(x[0]); }
};
template <typename T> struct Rows<T, 4> {
  static __device__ __forceinline__ void load(const T* p, float (&x)[4]) {
    const f32x4 v = widen4(load4(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
  }
  static __device__ __forceinline__ void store(T* p, const float (&x)[4]) {
    __builtin_nontemporal_store(narrow4<T>(f32x4{x[0], x[1], x[2], x[3]}), reinterpret_cast<V4<T>*>(p));
  }
};
template <> struct Rows<bf16, 8> {
  static __device__ __forceinline__ void store(bf16* p, const float (&x)[8]) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (bf16)x[i];
    __builtin_nontemporal_store(v, reinterpret_cast<bf16x8*>(p));
  }
};
template <> struct Rows<float, 8> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[8]) {
    const f32x4 a = load4(p), b = load4(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p));
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4*>(p + 4));
  }
};

// The sequence and the part of it that item `item` of a launch is: every
// sequence is cut into parts of `part` tokens (at least one part, also when
// it is empty), numbered through.  Tokens t0 .. t1-1 of sequence n, which
// starts at row `start` and has `len` tokens; `first` / `last`: its first and
// last part.
struct SeqPart {
  int n, li, t0, t1, len;   // li: n counted from the launch's first sequence
  size_t start;
  bool first, last;
};
__device__ __forceinline__ SeqPart seq_part(const SeqTab& s, int item) {
  SeqPart p;
  int k;   // part within the sequence
  if (s.n == 0) {
    p.n = p.li = item / s.parts;
    k = item - p.n * s.parts;
    p.start = (size_t)p.n * s.T;
    p.len = s.T;
  } else {
    int lo = 0, hi = s.n;   // cc[lo] <= item < cc[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.cc[mid] <= item) lo = mid;
      else hi = mid;
    }
    p.n = s.n0 + lo;
    p.li = lo;
    k = item - s.cc[lo];
    p.start = (size_t)s.cu[lo];
    p.len = s.cu[lo + 1] - s.cu[lo];
  }
  p.t0 = k * s.part;
  p.t1 = min(p.t0 + s.part, p.len);
  p.first = k == 0;
  p.last = p.t0 + s.part >= p.len;
  return p;
}

}  // namespace kda
