// Product of 8-bit rows with 8-bit weights, both e4m3 with fp32 scales: every
// 128 channels of a row share a scale, every 128 x 128 tile of the weights.
//
//   c[m, n] = sum_kb sa[m, kb] sw[n / 128, kb] sum_{k in kb} a[m, k] w[n, k]
// The inner sum is one MFMA step of 128 reduction indices started from zero;
// its result joins the fp32 accumulator with one fma by sa sw.
//
// The weights are the MFMA's left operand, so that a lane holds four
// neighbouring outputs of one row (an 8- or 16-byte store) and needs one scale
// per 16 rows instead of four.
#include "kda_rows.h"

namespace kda {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) const void* GlbP;
typedef __attribute__((address_space(3))) void* LdsP;
typedef unsigned char u8;

typedef unsigned char u8;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// 32 reduction indices of a row (or column) as an operand of the product, and
// D = A (16 x 128) B (128 x 16): lane l holds the same indices on both sides,
// of row (column) l % 16; D's rows 4 (l / 16) .. + 3 of column l % 16.
// bf16 outputs take the 8-bit matrix instruction: twice the rate, but its sum
// of 128 products is off by 1.4e-5 of the sum's rms (measured; a 120th of the
// output's rounding).  fp32 outputs take fp16 operands, which hold e4m3 and its
// products exactly: 5e-8 to 8e-8 over 4096 indices.
template <typename T> struct Frag;
template <> struct Frag<bf16> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) { v = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}; }
};
template <> struct Frag<float> {
  f16x8 v[4];
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = q < 2 ? lo[2 * q + h] : hi[2 * q - 4 + h];
        const f16x2 x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d, 1.f, false), y = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d, 1.f, true);
        v[q][4 * h] = x[0];
        v[q][4 * h + 1] = x[1];
        v[q][4 * h + 2] = y[0];
        v[q][4 * h + 3] = y[1];
      }
  }
};
__device__ __forceinline__ f32x4 mma128(const Frag<bf16>& a, const Frag<bf16>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero4(), 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma128(const Frag<float>& a, const Frag<float>& b) {
  f32x4 d = zero4();
#pragma unroll
  for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[q], b.v[q], d, 0, 0, 0);
  return d;
}

template <typename T> __device__ __forceinline__ void store_out(const Gemm8Args& g, long long m, int n, f32x4 v) {
  T* p = (T*)g.c + m * g.N + n;
  if ((g.N & 3) == 0) {   // n is a multiple of 4: all four inside, and aligned
    if (n < g.N) *reinterpret_cast<V4<T>*>(p) = narrow4<T>(v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < g.N) p[i] = from_f32<T>(v[i]);
}

// ---------------------------------------------------------------- tiles
// Rows of 128 bytes in LDS, the eight 16-byte pieces of row r stored in the
// order p ^ (r / 2 % 8): the 16 rows an operand read touches then lie in
// different banks.
__device__ __forceinline__ int lds_piece(int r, int p) { return r * 128 + ((p ^ ((r >> 1) & 7)) << 4); }


// Work-group tile BM x BN, WM x WN waves; `left` reduction indices of a step
// are inside K (128 but for the last).
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm8_tile_kernel(const Gemm8Args g, unsigned tm, unsigned tn) {
  constexpr int kThreads = 64 * WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int LA = BM * 8 / kThreads, LB = BN * 8 / kThreads;   // 16-byte pieces a thread stages
  static_assert(kThreads % 128 == 0 && BN / WN <= 128 && BM <= 256 && BN <= 256 && BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "tile");
  extern __shared__ u8 smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave % WM, wn = wave / WM, r = lane & 15, grp = lane >> 4;
  // tiles of one XCD (work-groups b, b + 8, ..) are neighbours: runs of eight
  // tile rows share a column of weights in its L2
  const unsigned tiles = tm * tn, per = (tiles + 7) / 8;
  const unsigned t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (t >= tiles || (blockIdx.x >> 3) >= per) return;
  const unsigned run = 8 * tn, first = t / run * 8, h = min(8u, tm - first), in = t % run;
  const long long m0 = (long long)(first + in % h) * BM;
  const int n0 = (int)(in / h) * BN;
  const int KB = (g.K + 127) / 128, rows = (int)min((long long)BM, g.M - m0), cols = min(BN, g.N - n0);

  // A tile's rows are at most 255 strides of 2^24 bytes apart: 32-bit offsets.
  // Rows past the last re-read that one and are not stored.
  const u8 *ga = g.a + m0 * g.lda, *gw = g.w + (size_t)n0 * g.K;
  unsigned oa[LA], ob[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int s = i * kThreads + tid, row = s >> 3;
    oa[i] = (unsigned)min(row, rows - 1) * (unsigned)g.lda + ((s & 7) ^ ((row >> 1) & 7)) * 16;
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int s = i * kThreads + tid, row = s >> 3;
    ob[i] = (unsigned)min(row, cols - 1) * (unsigned)g.K + ((s & 7) ^ ((row >> 1) & 7)) * 16;
  }
  // Pieces past K re-read the row's first block; the products left out are made
  // zero on a's side (what is read of w there is w's own row: no new NaN).
  auto stage = [&](int kb) {
    u8* base = smem + (kb & 1) * (BM + BN) * 128 + wave * 1024;
    const size_t k = (size_t)kb * 128;
    if (kb * 128 + 128 <= g.K) {
#pragma unroll
      for (int i = 0; i < LA; ++i) __builtin_amdgcn_global_load_lds((GlbP)(ga + k + oa[i]), (LdsP)(base + i * kThreads * 16), 16, 0, 0);
#pragma unroll
      for (int i = 0; i < LB; ++i) __builtin_amdgcn_global_load_lds((GlbP)(gw + k + ob[i]), (LdsP)(base + BM * 128 + i * kThreads * 16), 16, 0, 0);
    } else {
      const int c = ((tid & 7) ^ ((tid >> 4) & 7)) * 16;   // (the same piece of every row this thread stages)
      const size_t kc = (int)k + c < g.K ? k : (size_t)0 - c;
#pragma unroll
      for (int i = 0; i < LA; ++i) __builtin_amdgcn_global_load_lds((GlbP)(ga + kc + oa[i]), (LdsP)(base + i * kThreads * 16), 16, 0, 0);
#pragma unroll
      for (int i = 0; i < LB; ++i) __builtin_amdgcn_global_load_lds((GlbP)(gw + kc + ob[i]), (LdsP)(base + BM * 128 + i * kThreads * 16), 16, 0, 0);
    }
  };
  const float* gsa = g.sa + m0 * g.lsa;
  unsigned os[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) os[i] = (unsigned)min(wm * (BM / WM) + i * 16 + r, rows - 1) * (unsigned)g.lsa;
  const float* sw = g.sw + (size_t)min((n0 + wn * (BN / WN)) / 128, (g.N - 1) / 128) * KB;

  // where this lane's pieces grp and grp + 4 of row r of a 16-row tile are
  // (tiles are 2048 bytes apart and start at the same place in the order)
  const int lo = lds_piece(r, grp), hi = lds_piece(r, grp + 4);
  auto frag = [&](const u8* tile) {
    Frag<T> f;
    f.set(*reinterpret_cast<const i32x4*>(tile + lo), *reinterpret_cast<const i32x4*>(tile + hi));
    return f;
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = zero4();
  // scales of the coming step as loaded: multiplied behind the next wait, as a
  // use before would wait for the step's tiles as well
  float an[MT], wnx = sw[0];
#pragma unroll
  for (int i = 0; i < MT; ++i) an[i] = gsa[os[i]];
  stage(0);
  for (int kb = 0; kb < KB; ++kb) {
    // this wave's pieces of step kb are in LDS (a barrier alone does not wait
    // for loads to LDS), and every wave has read what it needs of step kb - 1
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float f[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) f[i] = an[i] * wnx;
    if (kb + 1 < KB) {
      wnx = sw[kb + 1];
#pragma unroll
      for (int i = 0; i < MT; ++i) an[i] = (gsa + kb + 1)[os[i]];
      stage(kb + 1);
    }
    const u8* ta = smem + (kb & 1) * (BM + BN) * 128 + wm * (BM / WM) * 128;
    const u8* tb = smem + (kb & 1) * (BM + BN) * 128 + (BM + wn * (BN / WN)) * 128;
    Frag<T> xa[MT];
    if (kb * 128 + 128 <= g.K) {
#pragma unroll
      for (int i = 0; i < MT; ++i) xa[i] = frag(ta + i * 2048);
    } else {
      const int left = g.K - kb * 128;
      const i32x4 z{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MT; ++i)
        xa[i].set(grp * 16 < left ? *reinterpret_cast<const i32x4*>(ta + i * 2048 + lo) : z,
                  grp * 16 + 64 < left ? *reinterpret_cast<const i32x4*>(ta + i * 2048 + hi) : z);
    }
    // Product q's result joins its sum two products later: its latency passes
    // behind them.
    Frag<T> wb[2];
    wb[0] = frag(tb);
    f32x4 p[3];
#pragma unroll
    for (int q = 0; q < NT * MT + 2; ++q) {
      if (q < NT * MT) {
        const int j = q / MT, i = q % MT;
        if (i == 0 && j + 1 < NT) wb[(j + 1) & 1] = frag(tb + (j + 1) * 2048);
        p[q % 3] = mma128(wb[j & 1], xa[i]);
      }
      __builtin_amdgcn_sched_barrier(0);   // (the compiler would put the fmas in front)
      if (q >= 2) {
        const int j = (q - 2) / MT, i = (q - 2) % MT;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][i][e] = fmaf(p[(q - 2) % 3][e], f[i], acc[j][i][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = wm * (BM / WM) + i * 16 + r;
    if (row >= rows) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) store_out<T>(g, m0 + row, n0 + wn * (BN / WN) + j * 16 + 4 * grp, acc[j][i]);
  }
}

// ---------------------------------------------------------------- few rows
// Up to 16 MT rows: bound by the weights' bytes.  A work-group takes 16
// outputs of every row; its waves take every WK-th block of K straight from
// memory and are joined through LDS.
template <typename T, int MT, int WK>
__global__ __launch_bounds__(64 * WK) void gemm8_rows_kernel(const Gemm8Args g) {
  __shared__ f32x4 part[WK][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, grp = lane >> 4;
  const int n0 = blockIdx.x * 16, KB = (g.K + 127) / 128;
  const u8* pw = g.w + (size_t)min(n0 + r, g.N - 1) * g.K;
  const float* sw = g.sw + (size_t)(n0 / 128) * KB;
  const u8* pa[MT];
  const float* sa[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long long m = min((long long)(i * 16 + r), g.M - 1);
    pa[i] = g.a + m * g.lda;
    sa[i] = g.sa + m * g.lsa;
    acc[i] = zero4();
  }
  for (int kb = wave; kb < KB; kb += WK) {
    const int k0 = kb * 128 + grp * 16, k1 = k0 + 64;
    const i32x4 z{0, 0, 0, 0};
    const i32x4 w0 = k0 < g.K ? *reinterpret_cast<const i32x4*>(pw + k0) : z, w1 = k1 < g.K ? *reinterpret_cast<const i32x4*>(pw + k1) : z;
    Frag<T> wb, xa;
    wb.set(w0, w1);
    const float s = sw[kb];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const i32x4 a0 = k0 < g.K ? *reinterpret_cast<const i32x4*>(pa[i] + k0) : z, a1 = k1 < g.K ? *reinterpret_cast<const i32x4*>(pa[i] + k1) : z;
      xa.set(a0, a1);
      const f32x4 p = mma128(wb, xa);
      const float f = sa[i][kb] * s;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], f, acc[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += WK) {
    const long long m = i * 16 + r;
    f32x4 v = part[0][i][lane];
#pragma unroll
    for (int q = 1; q < WK; ++q) v += part[q][i][lane];
    if (m < g.M) store_out<T>(g, m, n0 + 4 * grp, v);
  }
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t tile_go(const Gemm8Args& g, hipStream_t st) {
  constexpr int kThreads = 64 * WM * WN, kLds = 2 * (BM + BN) * 128;
  const long long tm = (g.M + BM - 1) / BM, tn = (g.N + BN - 1) / BN, n = (tm * tn + 7) / 8 * 8;
  if (n > max_groups(kThreads)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_tile_kernel<T, BM, BN, WM, WN>), dim3((unsigned)n), dim3(kThreads), kLds, st, g, (unsigned)tm, (unsigned)tn);
  return hipGetLastError();
}

template <typename T, int MT, int WK>
hipError_t rows_go(const Gemm8Args& g, hipStream_t st) {
  if ((g.N + 15) / 16 > max_groups(64 * WK)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_rows_kernel<T, MT, WK>), dim3((unsigned)((g.N + 15) / 16)), dim3(64 * WK), 0, st, g);
  return hipGetLastError();
}

template <typename T>
hipError_t gemm8_go(const Gemm8Args& g, hipStream_t st) {
  if (g.M <= 16) return rows_go<T, 1, 4>(g, st);
  if (g.M <= 32) return rows_go<T, 2, 4>(g, st);
  if (g.M <= 64) return rows_go<T, 4, 4>(g, st);
  if ((g.M + 255) / 256 * ((g.N + 255) / 256) >= 192) return tile_go<T, 256, 256, 4, 2>(g, st);
  return tile_go<T, 128, 128, 2, 2>(g, st);
}

}  // namespace

hipError_t launch_gemm8(int out_bf16, const Gemm8Args& g, hipStream_t st) {
  return out_bf16 ? gemm8_go<bf16>(g, st) : gemm8_go<float>(g, st);
}

}  // namespace kda
