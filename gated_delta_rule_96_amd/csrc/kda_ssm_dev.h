// Device building blocks of the state space scan (kda_ssm.hip): the chunk's
// step sizes and decay sums, transposed operand slabs from LDS, and the
// staging of token rows.
#pragma once
#include "kda_rows.h"

namespace kda {

constexpr int kSsmThreads = 256;
constexpr int kSsmWaves = 4;
constexpr int kQ = kSeqChunk;   // tokens per chunk

// log(1 + e^x) without overflow; log1p keeps its relative accuracy for very
// negative x.
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// x from the lane that DPP control `ctrl` selects, 0 where there is none.
template <int ctrl, int row_mask = 0xf>
__device__ __forceinline__ double dpp_zero(double x) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, ctrl, row_mask, 0xf, false);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), ctrl, row_mask, 0xf, false);
  return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
// Inclusive sum over the wave's lanes up to each (rows of 16 by shifts of 1,
// 2, 4, 8; then lane 15 of rows 0 and 2, then lane 31, into the rows behind).
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_zero<0x111>(x);
  x += dpp_zero<0x112>(x);
  x += dpp_zero<0x114>(x);
  x += dpp_zero<0x118>(x);
  x += dpp_zero<0x142, 0xA>(x);
  x += dpp_zero<0x143, 0xC>(x);
  return x;
}
__device__ __forceinline__ double lane63(double x) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)b, 63);
  const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(b >> 32), 63);
  return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
__device__ __forceinline__ float exp2_of(double x) { return exp2_fast((float)x); }

// A token's step size and its decay exponent dt A in log2 units (64 bits: sums
// of many tokens keep the small differences between neighbours).
struct StepSize {
  float dt;
  double a;
};
__device__ __forceinline__ StepSize step_size(float raw, float bias, int softplus, double a2) {
  StepSize s;
  const float v = raw + bias;
  s.dt = softplus ? softplus_f(v) : v;
  s.a = (double)s.dt * a2;
  return s;
}

// Rows of LDS tiles are padded so that 16 rows' equal columns fall on
// different banks.
template <typename T> struct LdsPad;
template <> struct LdsPad<bf16> { static constexpr int v = 8; };
template <> struct LdsPad<float> { static constexpr int v = 4; };

// Slab whose reduction index is the LDS row: rows r0 + {4g.., 16+4g..} of one
// column per lane (l16 = lane % 16).  The column of l16 is c0 + step (l16 / 4)
// + l16 % 4.  16-bit types: the transposed LDS read, whose lane 4q + s of a
// group of 16 points at row 4g + q, columns 4s..4s+3 and gets column 4q + s.
template <typename T>
__device__ __forceinline__ Slab<T> slab_tr(const T* p, int pitch, int c0, int step) {
  const int l = lane_id(), g = l >> 4, l16 = l & 15;
  Slab<T> s;
  if constexpr (sizeof(T) == 2) {
    typedef __attribute__((address_space(3))) bf16x4* LdsP;
    const T* a = p + (4 * g + (l16 >> 2)) * pitch + c0 + step * (l16 & 3);
    s = slab_of<T>(__builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a)), __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a + 16 * pitch)));
  } else {
    const T* a = p + (4 * g) * pitch + c0 + step * (l16 >> 2) + (l16 & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.lo[i] = a[i * pitch];
      s.hi[i] = a[(16 + i) * pitch];
    }
  }
  return s;
}

// fp32 values as an operand of products that stay fp32 results: one slab
// (fp32), or three bf16 slabs, each the rounding of what the ones before left
// (8 significant bits each: 24 together).
template <typename T> struct Split;
template <> struct Split<float> { Slab<float> h; };
template <> struct Split<bf16> { Slab<bf16> h, m, l; };
__device__ __forceinline__ void split_of(f32x4 lo, f32x4 hi, Split<float>& s) { s.h = Slab<float>{lo, hi}; }
__device__ __forceinline__ void split_of(f32x4 lo, f32x4 hi, Split<bf16>& s) {
  const V4<bf16> a = narrow4<bf16>(lo), b = narrow4<bf16>(hi);
  const f32x4 ra = lo - widen4(a), rb = hi - widen4(b);
  s.h = slab_of<bf16>(a, b);
  make_slab_split<bf16>(ra, rb, s.m, s.l);
}
// x w elementwise along the reduction index.
template <typename T>
__device__ __forceinline__ Split<T> scaled(const Slab<T>& x, f32x4 w0, f32x4 w1) {
  f32x4 a, b;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = (float)x.v[i] * w0[i];
      b[i] = (float)x.v[4 + i] * w1[i];
    }
  } else {
    a = x.lo * w0;
    b = x.hi * w1;
  }
  Split<T> s;
  split_of(a, b, s);
  return s;
}
// acc += A B with one operand in parts
template <typename T>
__device__ __forceinline__ f32x4 mma_split(const Slab<T>& a, const Split<T>& b, f32x4 acc) {
  acc = mma(a, b.h, acc);
  if constexpr (sizeof(T) == 2) {
    acc = mma(a, b.m, acc);
    acc = mma(a, b.l, acc);
  }
  return acc;
}

template <typename T>
__device__ __forceinline__ f32x4 mma_split(const Split<T>& a, const Slab<T>& b, f32x4 acc) {
  acc = mma(a.h, b, acc);
  if constexpr (sizeof(T) == 2) {
    acc = mma(a.m, b, acc);
    acc = mma(a.l, b, acc);
  }
  return acc;
}

// A state in the accumulator layout: the wave's dv/4 value columns as NT
// tiles, KT tiles of state channels.  kPerm: output row m of tile t is column
// wave CPW + 4 NT (m/4) + 4t + m%4 (a lane of a transposed product then holds
// neighbouring columns); otherwise wave CPW + 16 t + m.
template <int DK, int DV, bool kPerm>
struct State {
  static constexpr int CPW = DV / kSsmWaves, NT = CPW / 16, KT = DK / 16;
  f32x4 s[KT][NT];
  static __device__ __forceinline__ int col(int t) {
    const int l16 = lane_id() & 15, wave = threadIdx.x >> 6;
    return wave * CPW + (kPerm ? 4 * NT * (l16 >> 2) + 4 * t + (l16 & 3) : 16 * t + l16);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t) s[k][t] = zero4();
  }
  __device__ __forceinline__ void load(const float* p) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[k][t][r] = p[(size_t)(16 * k + 4 * g + r) * DV + col(t)];
  }
  __device__ __forceinline__ void store(float* p) const {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) p[(size_t)(16 * k + 4 * g + r) * DV + col(t)] = s[k][t][r];
  }
  // s = s el + rows^T (cols w) over a chunk: rows [kQ][DK] and cols [kQ][DV] in
  // LDS (xs: the wave's operand slabs of cols), one weight per token.
  template <typename T>
  __device__ __forceinline__ void update(float el, const T* rows, int pitch, const Slab<T> (&xs)[2][NT], const float* w) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int q = 0; q < NT; ++q) s[k][q] *= el;
#pragma unroll
    for (int js = 0; js < 2; ++js) {
      const f32x4 w0 = load4(w + 32 * js + 4 * g), w1 = load4(w + 32 * js + 16 + 4 * g);
      Split<T> xw[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) xw[q] = scaled<T>(xs[js][q], w0, w1);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const Slab<T> bs = slab_tr<T>(rows + 32 * js * pitch, pitch, 16 * k, 4);
#pragma unroll
        for (int q = 0; q < NT; ++q) s[k][q] = mma_split(bs, xw[q], s[k][q]);
      }
    }
  }
  template <typename T>
  static __device__ __forceinline__ void slabs(const T* cols, int pitch, Slab<T> (&xs)[2][NT]) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int js = 0; js < 2; ++js)
#pragma unroll
      for (int q = 0; q < NT; ++q)
        xs[js][q] = slab_tr<T>(cols + 32 * js * pitch, pitch, wave * CPW + (kPerm ? 4 : 16) * q, kPerm ? 4 * NT : 4);
  }
};

// kQ rows of D elements from global memory (row stride ld) to LDS (padded),
// through registers: load() issues the loads of rows < n (rows behind are
// zeros), store() writes them.
template <typename T, int D>
struct RowTile {
  static constexpr int VE = 16 / sizeof(T);
  static constexpr int kPer = kQ * D / VE / kSsmThreads;
  static constexpr int kPitch = D + LdsPad<T>::v;
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  u32x4 v[kPer];
  __device__ __forceinline__ void load(const T* p, long long ld, int n) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = (k * kSsmThreads + (int)threadIdx.x) * VE, r = e / D, c = e % D;
      v[k] = u32x4{0, 0, 0, 0};
      if (r < n) v[k] = *reinterpret_cast<const u32x4*>(p + (size_t)r * (size_t)ld + c);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = (k * kSsmThreads + (int)threadIdx.x) * VE, r = e / D, c = e % D;
      *reinterpret_cast<u32x4*>(lds + r * kPitch + c) = v[k];
    }
  }
};

// The work-group's (item, head): consecutive (item, head) pairs go to one XCD
// (work-groups are handed to the 8 XCDs in turn), so that the heads of a part
// find their shared B and C rows in that XCD's L2.
struct ItemHead {
  int item, h;
};
__device__ __forceinline__ bool item_head(int items, int H, ItemHead& w) {
  const unsigned per = gridDim.x >> 3;
  const unsigned id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (id >= (unsigned)items * (unsigned)H) return false;
  w.item = (int)(id / (unsigned)H);
  w.h = (int)(id - (unsigned)w.item * (unsigned)H);
  return true;
}
inline bool item_head_grid(int items, int H, dim3& grid) {
  const long long n = ((long long)items * H + 7) / 8 * 8;
  if (n > 0x7fffffffLL) return false;
  grid = dim3((unsigned)n);
  return true;
}

}  // namespace kda
