// Gated linear recurrence with one state a channel: its gates, and the tiles
// of tokens and channels that the forward (kda_lru.hip) and the gradients
// (kda_lru_bwd.hip) share.
//
//   g_t = -c Sigmoid(r_t), or r_t itself;   a_t = e^{g_t}
//   m_t = sqrt(1 - a_t^2), or 1;            u_t = m_t Sigmoid(i_t) x_t
//   h_t = a_t h_{t-1} + u_t,                y_t = h_t
// Over a run of tokens the state moves by h -> P h + H with P the product of
// the run's a and H its own state from zero; runs join by
// (P, H) then (P', H') = (P P', P' H + H').
#pragma once
#include "kda_rows.h"

namespace kda {

// NC channels of a token as they lie in memory.  kWord: two bf16 as one word.
// Where paths meet between load and use, as in the gradients, halves are taken
// apart there (32K x 2048 348 us, as words 336); the forward, which uses them in
// place, is slower with words (64K x 4096 427 us, as halves 419).
template <typename T, int NC, bool kWord = false> struct alignas(sizeof(T) * NC) LruPack {
  T v[NC];
  __device__ __forceinline__ float at(int j) const { return to_f32(v[j]); }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = from_f32<T>(x);
  }
  __device__ __forceinline__ void set(const float (&x)[NC]) {
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = from_f32<T>(x[j]);
  }
};
template <> struct alignas(4) LruPack<bf16, 2, true> {
  unsigned w;
  __device__ __forceinline__ float at(int j) const { return __uint_as_float(j ? w & 0xffff0000u : w << 16); }
  __device__ __forceinline__ void fill(float x) { set({x, x}); }
  __device__ __forceinline__ void set(const float (&x)[2]) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    w = __builtin_bit_cast(unsigned, bf16x2{(bf16)x[0], (bf16)x[1]});
  }
};

// a = e^g by way of d = 1 - a from the series of 1 - e^g where g is near 0, on
// either side: a is then within half a unit of its last place to either side (the
// exponential instruction's error has a bias, which a state that remembers
// thousands of tokens adds up), and 1 - a^2 = d (1 + a) loses nothing near
// a = 1.  Four terms for |g| below 2^-4 (bf16 inputs: what is left out is 2^-23
// of d), eight below 2^-1 (2^-26).
template <typename T> constexpr float lru_near() { return sizeof(T) == 2 ? 0.0625f : 0.5f; }
template <typename T> __device__ __forceinline__ float one_minus_decay_near(float g) {
  constexpr bool kShort = sizeof(T) == 2;
  float s = kShort ? 1.f / 24 : 1.f / 40320;
  if (!kShort) {
    s = fmaf(g, s, 1.f / 5040);
    s = fmaf(g, s, 1.f / 720);
    s = fmaf(g, s, 1.f / 120);
    s = fmaf(g, s, 1.f / 24);
  }
  s = fmaf(g, s, 1.f / 6);
  s = fmaf(g, s, 0.5f);
  return -g * fmaf(g, s, 1.f);
}
// The exponential is taken only where some lane of the wave needs it.
template <typename T> __device__ __forceinline__ float one_minus_decay(float g, float& a) {
  float d = one_minus_decay_near<T>(g);
  a = 1.f - d;
  const bool far = !(__builtin_fabsf(g) < lru_near<T>());   // (NaN too)
  if (__any(far)) {
    const float e = exp2_fast(g * kLog2e);
    a = far ? e : a;
    d = far ? 1.f - e : d;
  }
  return d;
}

// What a call is made of.  kFull: both gates and the unit factor, known when
// the kernel is compiled.
struct LruMode {
  bool gate, igate, unit;
};
template <bool kFull> __device__ __forceinline__ LruMode lru_mode(const LruArgs& a) {
  return kFull ? LruMode{true, true, true} : LruMode{a.c != nullptr, a.i != nullptr, a.unit != 0};
}
inline bool lru_full(const LruArgs& a) { return a.c && a.i && a.unit; }

// a and u of one channel of a token (c: the channel's coefficient).
template <typename T>
__device__ __forceinline__ void lru_gate(const LruMode md, float c, float x, float r, float i, float& a, float& u) {
  const float g = md.gate ? -c * sigmoid_fast(r) : r;
  const float d = one_minus_decay<T>(g, a);
  u = md.igate ? x * sigmoid_fast(i) : x;
  if (md.unit) u *= __builtin_amdgcn_sqrtf(d * (1.f + a));
}

// Channels of a wave's lane: NC neighbours from c on; lanes past D do the last
// ones' loads and store nothing.
struct LruLane {
  int c, cl;   // channel, channel to load from
  bool live;
};
template <int NC> __device__ __forceinline__ LruLane lru_lane(int slice, int D) {
  LruLane l;
  l.c = (slice * 64 + (int)(threadIdx.x & 63)) * NC;
  l.live = l.c < D;
  l.cl = l.live ? l.c : 0;
  return l;
}
// A lane's channels of a row that starts at `row` for all lanes: a scalar
// address and 32 bits of bytes a lane.
template <typename Pk, typename T> __device__ __forceinline__ Pk lru_load(const T* row, int c) {
  return *reinterpret_cast<const Pk*>(reinterpret_cast<const char*>(row) + (unsigned)c * (unsigned)sizeof(T));
}
template <typename Pk, typename T> __device__ __forceinline__ void lru_store(T* row, int c, const Pk& v) {
  *reinterpret_cast<Pk*>(reinterpret_cast<char*>(row) + (unsigned)c * (unsigned)sizeof(T)) = v;
}

template <int NC> __device__ __forceinline__ void lru_coef(const LruArgs& a, const LruLane& l, float (&c)[NC]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) c[k] = a.c ? a.c[l.cl + k] : 0.f;
}

}  // namespace kda
