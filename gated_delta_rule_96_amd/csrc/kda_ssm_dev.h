// Device building blocks of the state space scan (kda_ssm.hip): the chunk's
// step sizes and decay sums, transposed operand slabs from LDS, and the
// staging of token rows.
#pragma once
#include "kda_rows.h"

namespace kda {

constexpr int kSsmThreads = 256;
constexpr int kSsmWaves = 4;
constexpr int kQ = kSeqChunk;   // tokens per chunk

// Softplus(x) = log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x| in (0, 1], with
// log1p(u) = 2 artanh(z), z = u / (2 + u) <= 1/3, by its series (the first
// term left out is below 2e-9 of the sum): relative accuracy also for
// negative x, where the result is e^x, down to x = -87.3; below it e^x is not a
// normal fp32 number and the result 0 (v_exp_f32 gives no smaller ones).
// e^-|x| as 2^(n + r) with the rounding r of the product by log2(e) put back, so
// that large |x| costs no accuracy; |x| counts as 200 at most, so that
// infinities need no case of their own (NaN stays NaN).
__device__ __forceinline__ float softplus_f(float x) {
  const float ax = fabsf(x), m = ax > 200.f ? -200.f : -ax;
  const float n = m * kLog2e;
  const float r = fmaf(m, 1.925963033500e-8f, fmaf(m, kLog2e, -n));   // log2(e) - fl(log2(e))
  const float e = exp2_fast(n);
  const float u = fmaf(e, r * 0.69314718f, e);
  const float z = u * __builtin_amdgcn_rcpf(2.0f + u), q = z * z;
  float t = 1.f / 15.f;
  t = fmaf(t, q, 1.f / 13.f);
  t = fmaf(t, q, 1.f / 11.f);
  t = fmaf(t, q, 1.f / 9.f);
  t = fmaf(t, q, 1.f / 7.f);
  t = fmaf(t, q, 1.f / 5.f);
  t = fmaf(t, q, 1.f / 3.f);
  const float l = 2.f * z;
  return fmaxf(x, 0.f) + fmaf(l * q, t, l);
}

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
// of many tokens keep the small differences between neighbours).  Exponents
// below kNothing count as it: every factor across such a token is 0 in fp32
// either way (a product of others that outweighs it is out of range itself),
// and the sums of a chunk keep their places behind the point down to 2^-26.
struct StepSize {
  float dt;
  double a;
};
constexpr double kNothing = -1048576.0;
__device__ __forceinline__ StepSize step_size(float raw, float bias, int softplus, double a2) {
  StepSize s;
  const float v = raw + bias;
  s.dt = softplus ? softplus_f(v) : v;
  s.a = (double)s.dt * a2;
  if (s.a < kNothing) s.a = kNothing;
  return s;
}

// Rows of LDS tiles.  16-bit types: a row's start is 8 (row % 8) + 4 (row / 8
// % 2) banks on (row pitch D + 16 elements, rows 8..15 of every 16 another 8
// elements on), so that both the slab reads (16 rows, 16 bytes each from half
// a wave) and the transposed ones (8 rows, 32 bytes each) touch every bank
// once.  fp32: 4 banks a row.
template <typename T> struct LdsRow;
template <> struct LdsRow<bf16> {
  static constexpr int pad = 16;
  static __device__ __forceinline__ int shift(int row) { return row & 8; }
};
template <> struct LdsRow<float> {
  static constexpr int pad = 4;
  static __device__ __forceinline__ int shift(int) { return 0; }
};
template <typename T> __device__ __forceinline__ const T* lds_at(const T* p, int pitch, int row, int col) {
  return p + row * pitch + LdsRow<T>::shift(row) + col;
}

// The readers below take the lane (a kernel may hand it over hidden from the
// compiler, so that a loop does not keep all their addresses in registers).
// Slab whose reduction index is the LDS row: rows r0 + {4g.., 16+4g..} (r0 a
// multiple of 32) of one column per lane (l16 = lane % 16).  The column of l16 is c0 + step (l16 / 4)
// + l16 % 4.  16-bit types: the transposed LDS read, whose lane 4q + s of a
// group of 16 points at row 4g + q, columns 4s..4s+3 and gets column 4q + s.
template <typename T>
__device__ __forceinline__ Slab<T> slab_tr(const T* p, int pitch, int r0, int c0, int step, int l = lane_id()) {
  const int g = l >> 4, l16 = l & 15;
  Slab<T> s;
  if constexpr (sizeof(T) == 2) {
    typedef __attribute__((address_space(3))) bf16x4* LdsP;
    const T* a = lds_at(p, pitch, 4 * g + (l16 >> 2), step * (l16 & 3)) + r0 * pitch + c0;
    s = slab_of<T>(__builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a)), __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a + 16 * pitch)));
  } else {
    const T* a = p + (r0 + 4 * g) * pitch + c0 + step * (l16 >> 2) + (l16 & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.lo[i] = a[i * pitch];
      s.hi[i] = a[(16 + i) * pitch];
    }
  }
  return s;
}
// Slab along a row: columns c0 + {4g.., 16+4g..} of row r0 + l16 (r0 a multiple
// of 16).  RowLanes: where the lane's two halves are in a tile of this pitch;
// the second is hidden from the compiler (once per kernel): joined into one
// two-address read the halves would meet in the same banks.
struct RowLanes {
  int near, far;
};
template <typename T>
__device__ __forceinline__ RowLanes row_lanes(int pitch, int l = lane_id()) {
  const int l16 = l & 15, g = l >> 4;
  RowLanes r;
  r.near = l16 * pitch + LdsRow<T>::shift(l16) + 4 * g;
  r.far = r.near + 16;
  asm("" : "+v"(r.far));
  return r;
}
template <typename T>
__device__ __forceinline__ Slab<T> slab_row(const T* p, const RowLanes& rl, int at) {   // at = r0 pitch + c0
  return slab_of<T>(load4(p + at + rl.near), load4(p + at + rl.far));
}
// Slab of a product of two rows: columns c0 + 8g .. 8g+7, one 16-byte read
// (bf16); any order of the reduction index serves if both operands have it.
template <typename T>
__device__ __forceinline__ Slab<T> slab_any(const T* p, int pitch, int r0, int c0, int l = lane_id()) {
  const T* a = lds_at(p, pitch, l & 15, 8 * (l >> 4)) + r0 * pitch + c0;
  Slab<T> s;
  if constexpr (sizeof(T) == 2) s.v = *reinterpret_cast<const bf16x8*>(a);
  else s = slab_of<T>(load4(a), load4(a + 4));
  return s;
}
// Four columns from c0 of row r0 + l16.
template <typename T>
__device__ __forceinline__ f32x4 four_of_row(const T* p, int pitch, int r0, int c0, int l = lane_id()) {
  return widen4(load4(lds_at(p, pitch, l & 15, 0) + r0 * pitch + c0));
}

// fp32 values as an operand of products that stay fp32 results: one slab
// (fp32), or three bf16 slabs that together are the values exactly: the upper
// eight of the 24 significant bits, the next eight, the rest (truncations).
template <typename T> struct Split;
template <> struct Split<float> { Slab<float> h; };
template <> struct Split<bf16> { Slab<bf16> h, m, l; };
__device__ __forceinline__ void split_of(f32x4 lo, f32x4 hi, Split<float>& s) { s.h = Slab<float>{lo, hi}; }
__device__ __forceinline__ float upper16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// The upper halves of a and b as two bf16.
__device__ __forceinline__ unsigned pack_upper(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ void split_of(f32x4 lo, f32x4 hi, Split<bf16>& s) {
#pragma clang fp contract(off)   // the parts of the rounded value: exact
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  u32x4 h, m, l;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = k < 2 ? lo[2 * k] : hi[2 * k - 4], b = k < 2 ? lo[2 * k + 1] : hi[2 * k - 3];
    const float ra = a - upper16(a), rb = b - upper16(b);
    h[k] = pack_upper(a, b);
    m[k] = pack_upper(ra, rb);
    l[k] = pack_upper(ra - upper16(ra), rb - upper16(rb));
  }
  s.h.v = __builtin_bit_cast(bf16x8, h);
  s.m.v = __builtin_bit_cast(bf16x8, m);
  s.l.v = __builtin_bit_cast(bf16x8, l);
}
// x w elementwise along the reduction index.
template <typename T>
__device__ __forceinline__ Split<T> scaled(const Slab<T>& x, f32x4 w0, f32x4 w1) {
#pragma clang fp contract(off)
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
// lo += A B's lower parts, and acc + A B with one operand in parts.  The lower
// parts have a sum of their own: a product of much larger terms cuts a small
// accumulator off below its own last place (downwards: measured mean error
// 1.2e-8 of the result, which sums over many tokens show), a sum of terms of
// its own size is rounded to nearest (mean error below 1e-9).
template <typename T> __device__ __forceinline__ f32x4 mma_low(const Slab<T>& a, const Split<T>& b, f32x4 lo) {
  if constexpr (sizeof(T) == 2) lo = mma(a, b.m, mma(a, b.l, lo));
  return lo;
}
template <typename T> __device__ __forceinline__ f32x4 mma_low(const Split<T>& a, const Slab<T>& b, f32x4 lo) {
  if constexpr (sizeof(T) == 2) lo = mma(a.m, b, mma(a.l, b, lo));
  return lo;
}
template <typename T> __device__ __forceinline__ f32x4 mma_split(const Split<T>& a, const Slab<T>& b, f32x4 acc) {
  acc = mma(a.h, b, acc);
  if constexpr (sizeof(T) == 2) acc += mma_low(a, b, zero4());
  return acc;
}

// bf16 rows in LDS without padding, filled by direct global-to-LDS loads (16
// bytes a lane to 64 consecutive places of 16 bytes): row r's 16-byte pieces
// are stored at piece ^ swz(r).  swz is chosen so that the reads below touch
// every bank once: slabs along rows (16 rows, one piece each), and transposed
// slabs (8 rows, two neighbouring pieces each).
template <int D>
struct SwzTile {
  static constexpr int kElems = kQ * D;
  static __device__ __forceinline__ int swz(int r) {
    return D == 128 ? ((r & 7) << 1) | ((r >> 3) & 1) : (((r >> 1) & 3) << 1) | ((r >> 3) & 1);
  }
  static __device__ __forceinline__ int at(int row, int col) { return row * D + ((((col >> 3) ^ swz(row)) << 3) | (col & 7)); }
  // Rows 0..63 of p (row stride ld) by the four waves of a set (tid 0..255);
  // rows >= n repeat row n - 1.  Completes with the wave's vector loads.
  static __device__ __forceinline__ void load(bf16* lds, const bf16* p, long long ld, int n, int tid) {
    typedef __attribute__((address_space(3))) void* LdsP;
    typedef const __attribute__((address_space(1))) void* GlbP;
    constexpr int kPieces = D / 8, kRows = 64 / kPieces;   // pieces of a row, rows a wave's load fills
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = kRows * wave + lane / kPieces, c = ((lane % kPieces) ^ swz(r)) * 8;
#pragma unroll
    for (int i = 0; i < 16 / kRows; ++i) {
      constexpr int kStep = 4 * kRows;   // rows between a wave's loads (a multiple of 16)
      bf16* to = lds + (kStep * i + kRows * wave) * D;
      const int row = n >= kQ ? kStep * i + r : min(kStep * i + r, n - 1);
      const unsigned off = ((unsigned)row * (unsigned)ld + (unsigned)c) * 2u;
      __builtin_amdgcn_global_load_lds((GlbP)(reinterpret_cast<const char*>(p) + off), (LdsP)to, 16, 0, 0);
    }
  }
  // Columns 32 z + 8g .. +7 of row r0 + l16: any order of the reduction index.
  static __device__ __forceinline__ Slab<bf16> any(const bf16* t, int r0, int z) {
    const int l16 = lane_id() & 15, g = lane_id() >> 4;
    Slab<bf16> s;
    s.v = *reinterpret_cast<const bf16x8*>(t + r0 * D + ((l16 * D + ((g ^ swz(l16)) << 3)) ^ (32 * z)));
    return s;
  }
  // Columns 32 z + {4g.., 16+4g..} of row 16 it + l16.  RowBase holds the
  // lane's place in each row tile, hidden from the compiler once: two such
  // 8-byte reads joined into one two-address read would meet in the same
  // banks.
  struct RowBase {
    int at[4];
  };
  static __device__ __forceinline__ RowBase row_base() {
    const int l16 = lane_id() & 15, g = lane_id() >> 4;
    RowBase b;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      b.at[it] = (16 * it + l16) * D + ((((g >> 1) ^ swz(l16)) << 3) | ((g & 1) << 2));
      asm("" : "+v"(b.at[it]));
    }
    return b;
  }
  static __device__ __forceinline__ Slab<bf16> row(const bf16* t, const RowBase& b, int it, int z) {
    return slab_of<bf16>(load4(t + (b.at[it] ^ (32 * z))), load4(t + (b.at[it] ^ (32 * z + 16))));
  }
  // Rows r0 + {4g.., 16+4g..} of column c0 + step (l16 / 4) + l16 % 4 (r0 a
  // multiple of 32, c0 of 16 for step 4, of 4 within 32 for step 8).
  static __device__ __forceinline__ Slab<bf16> tr(const bf16* t, int r0, int c0, int step) {
    typedef __attribute__((address_space(3))) bf16x4* LdsP;
    const int l16 = lane_id() & 15, g = lane_id() >> 4, r = 4 * g + (l16 >> 2), q = l16 & 3;
    const bf16* a;
    if (step == 4) a = t + r0 * D + ((r * D + ((((q >> 1) ^ swz(r)) << 3) | ((q & 1) << 2))) ^ c0);
    else a = t + r0 * D + ((r * D + ((q ^ swz(r)) << 3)) ^ (c0 & ~7)) + (c0 & 7);
    return slab_of<bf16>(__builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a)), __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LdsP)(a + 16 * D)));
  }
  // Four columns from c (a multiple of 4) of row r0 + l16.
  static __device__ __forceinline__ f32x4 four(const bf16* t, int r0, int c) {
    const int l16 = lane_id() & 15;
    return widen4(load4(t + r0 * D + l16 * D + ((((c >> 3) ^ swz(l16)) << 3) | (c & 7))));
  }
};
// The same reads of a padded tile.
template <typename T, int D>
struct PadTile {
  static constexpr int kPitch = D + LdsRow<T>::pad;
  static __device__ __forceinline__ Slab<T> tr(const T* t, int r0, int c0, int step) { return slab_tr<T>(t, kPitch, r0, c0, step); }
};

// A state in the accumulator layout: the wave's dv/4 value columns as NT
// tiles, KT tiles of state channels.  Output row m of tile t is column wave CPW
// + 4 NT (m/4) + 4t + m%4: a lane of a transposed product then holds
// neighbouring columns.
template <int DK, int DV>
struct State {
  static constexpr int CPW = DV / kSsmWaves, NT = CPW / 16, KT = DK / 16;
  f32x4 s[KT][NT];
  static __device__ __forceinline__ int col(int t) {
    const int l16 = lane_id() & 15, wave = (threadIdx.x >> 6) & (kSsmWaves - 1);
    return wave * CPW + 4 * NT * (l16 >> 2) + 4 * t + (l16 & 3);
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
  // s = s el + rows^T (cols w) over a chunk, in two steps: the weighted operand
  // xw from the wave's slabs of cols [kQ][DV] and one weight per token, and the
  // products with rows [kQ][DK] in LDS (Tile: how those are laid out).  The
  // chunk's sum is formed apart from the state: small parts are not rounded
  // to the state's last place one by one.  The lower parts start the sum (one
  // addition less per element than a sum of their own, and a mean error of
  // 1e-8, see mma_low).
  template <typename T>
  static __device__ __forceinline__ void weigh(const Slab<T> (&xs)[2][NT], const float* w, Split<T> (&xw)[2][NT]) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int js = 0; js < 2; ++js) {
      const f32x4 w0 = load4(w + 32 * js + 4 * g), w1 = load4(w + 32 * js + 16 + 4 * g);
#pragma unroll
      for (int q = 0; q < NT; ++q) xw[js][q] = scaled<T>(xs[js][q], w0, w1);
    }
  }
  template <typename Tile, typename T>
  __device__ __forceinline__ void update(float el, const T* rows, const Split<T> (&xw)[2][NT]) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const Slab<T> b0 = Tile::tr(rows, 0, 16 * k, 4), b1 = Tile::tr(rows, 32, 16 * k, 4);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const f32x4 low = mma_low(b1, xw[1][q], mma_low(b0, xw[0][q], zero4()));
        const f32x4 sum = mma(b1, xw[1][q].h, mma(b0, xw[0][q].h, low));
#pragma unroll
        for (int r = 0; r < 4; ++r) s[k][q][r] = fmaf(s[k][q][r], el, sum[r]);
      }
    }
  }
  template <typename Tile, typename T>
  static __device__ __forceinline__ void slabs(const T* cols, Slab<T> (&xs)[2][NT]) {
    const int wave = (threadIdx.x >> 6) & (kSsmWaves - 1);
#pragma unroll
    for (int js = 0; js < 2; ++js)
#pragma unroll
      for (int q = 0; q < NT; ++q)
        xs[js][q] = Tile::tr(cols, 32 * js, wave * CPW + 4 * q, 4 * NT);
  }
};

// A state kept transposed (nothing multiplies it): tile (k, q) of the wave holds
// value columns wave CPW + 16 q + 4g .. +3 of state channel 16 k + l16, so that
// it is read and written 16 bytes a lane.
template <int DK, int DV>
struct SweepState {
  static constexpr int CPW = DV / kSsmWaves, NT = CPW / 16, KT = DK / 16;
  f32x4 s[KT][NT];
  static __device__ __forceinline__ int at(int k, int q) {
    const int l16 = lane_id() & 15, g = lane_id() >> 4, wave = (threadIdx.x >> 6) & (kSsmWaves - 1);
    return (16 * k + l16) * DV + wave * CPW + 16 * q + 4 * g;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int q = 0; q < NT; ++q) s[k][q] = zero4();
  }
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int q = 0; q < NT; ++q) s[k][q] = load4(p + at(k, q));
  }
  __device__ __forceinline__ void store(float* p) const {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int q = 0; q < NT; ++q) *reinterpret_cast<f32x4*>(p + at(k, q)) = s[k][q];
  }
  // As State::weigh and update, with the products the other way round.  kLow:
  // the lower parts' sum stays apart to the end.
  template <bool kLow, typename TileK, typename TileV, typename T>
  __device__ __forceinline__ void update(float el, const T* rows, const T* cols, const float* w) {
    const int g = lane_id() >> 4, wave = (threadIdx.x >> 6) & (kSsmWaves - 1);
    Split<T> xw[2][NT];
#pragma unroll
    for (int js = 0; js < 2; ++js) {
      const f32x4 w0 = load4(w + 32 * js + 4 * g), w1 = load4(w + 32 * js + 16 + 4 * g);
#pragma unroll
      for (int q = 0; q < NT; ++q) xw[js][q] = scaled<T>(TileV::tr(cols, 32 * js, wave * CPW + 16 * q, 4), w0, w1);
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const Slab<T> b0 = TileK::tr(rows, 0, 16 * k, 4), b1 = TileK::tr(rows, 32, 16 * k, 4);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const f32x4 low = mma_low(xw[1][q], b1, mma_low(xw[0][q], b0, zero4()));
        const f32x4 sum = mma(xw[1][q].h, b1, mma(xw[0][q].h, b0, kLow ? zero4() : low));
#pragma unroll
        for (int r = 0; r < 4; ++r) s[k][q][r] = fmaf(s[k][q][r], el, sum[r]);
        if constexpr (kLow && sizeof(T) == 2) s[k][q] += low;
      }
    }
  }
};

// kQ rows of D elements from global memory (row stride ld) to LDS (padded),
// through the registers of kThreads threads: load() issues the loads of rows
// < n (rows behind are zeros), store() writes them.
template <typename T, int D, int kThreads = kSsmThreads>
struct RowTile {
  static constexpr int VE = 16 / sizeof(T);
  static constexpr int kPer = kQ * D / VE / kThreads;
  static constexpr int kRows = kThreads * VE / D;   // rows between a thread's pieces (a multiple of 8)
  static constexpr int kPitch = D + LdsRow<T>::pad;
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  u32x4 v[kPer];
  // p and ld are the same for all threads: a scalar base per piece, and one
  // 32-bit offset per thread (ld is at most 2^24 elements)
  __device__ __forceinline__ void load(const T* p, long long ld, int n, int tid) {
    const int r = tid * VE / D, c = tid * VE % D;
    const unsigned off = ((unsigned)r * (unsigned)ld + (unsigned)c) * (unsigned)sizeof(T);
    const char* base = reinterpret_cast<const char*>(p);
    const size_t step = (size_t)kRows * (size_t)ld * sizeof(T);
    if (n >= kQ) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[k] = *reinterpret_cast<const u32x4*>(base + k * step + off);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        v[k] = u32x4{0, 0, 0, 0};
        if (k * kRows + r < n) v[k] = *reinterpret_cast<const u32x4*>(base + k * step + off);
      }
    }
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
    const int r = tid * VE / D, c = tid * VE % D;
    T* q = lds + r * kPitch + LdsRow<T>::shift(r) + c;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      static_assert(kRows % 16 == 0 || kRows == 8 || sizeof(T) != 2, "rows keep their shift");
      *reinterpret_cast<u32x4*>(q + k * kRows * kPitch) = v[k];
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
inline dim3 item_head_grid(int items, int H) { return dim3(((unsigned)items * (unsigned)H + 7) / 8 * 8); }
// Items of a launch at most: 512 threads for each (item, head) (scan and
// gradients, or two sweep work-groups of 256).
inline long long most_items(int H) { return (max_groups(512) - 7) / H; }

}  // namespace kda
