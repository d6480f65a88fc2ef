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
// Measured: 8192 x 12288 x 4096 389 to 400 us (2.1 PFLOP/s; a library's product of
// such operands with one scale each 338), 8191 x 8480 x 4096 281, 256 rows of the
// first 22.5, one row 11.  Of the large tile's time the matrix instructions take
// 49%, and no single part binds it: without the loads to LDS it ran at 2.31
// PFLOP/s, without its reads of the weights from LDS 2.31, without three in four of
// the fmas that join blocks 2.15, with every load from the cache 2.18 (2.04 then).
// The next step's first operands read behind the last products of a step: the
// same.
#include "kda_rows.h"

namespace kda {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) const void* GlbP;
typedef __attribute__((address_space(3))) void* LdsP;
typedef unsigned char u8;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// 32 reduction indices of a row (or column) as an operand of the product, and
// D = A (16 x 128) B (128 x 16): lane l holds the same indices on both sides,
// of row (column) l % 16; D's rows 4 (l / 16) .. + 3 of column l % 16.
// bf16 outputs take the 8-bit matrix instruction, twice the rate, whose products
// are not summed in 32 bits: of every 8 neighbouring k each is cut towards zero at
// 2^-13 of their largest power of two (measured for every place in a block; factors
// below 2^-6 count as 2^-6), so a block is off by at most 7 x 2^-13 of the sum of
// those, 2^-10 of sum |a w|; the output rounds by 2^-9 to 2^-8.  Only where large
// products cancel does it show.  Random rows: 1.4e-5 of the sum's rms.  fp32 outputs
// take fp16 operands, which hold e4m3 and its products exactly: 5e-8 to 8e-8 over 4096
// indices.
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
  T* p = (T*)g.c + m * g.ldc + n;
  if ((g.ldc & 3) == 0) {   // (and with it N) n is a multiple of 4: all four inside, and aligned
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

// Work-group tile BM x BN.  A step is one block of 128 reduction indices; R of
// them are in LDS, in sets of U that the waves meet for: a step's loads are
// issued R - U steps before it.  KG groups of WM x WN waves take a set's steps by
// turns, with sums of their own that are joined through LDS at the end: fewer
// waves read a step's operands, and larger pieces each (64 x 64 tiles, 8 waves for
// every step against two groups of 4: 12.7 and 10.9 us for 64 x 4096 x 4096, 19.4
// and 15.9 in fp32; 64 x 128: 16.6 and 15.0 for 512 x 4096 x 4096; with 128 x 128 two
// groups leave no room for loads further ahead: 24.6 and 25.0).
template <typename T, int BM, int BN, int WM, int WN, int KG, int R, int U>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void gemm8_tile_kernel(const Gemm8Args g, unsigned tm, unsigned tn) {
  constexpr int kThreads = 64 * WM * WN * KG, MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int LA = BM * 8 / kThreads, LB = BN * 8 / kThreads;   // 16-byte pieces a thread stages
  static_assert(kThreads % 128 == 0 && BN / WN <= 128 && BM <= 256 && BN <= 256 && BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "tile");
  extern __shared__ u8 smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, grp = lane >> 4;
  const int wm = wave % WM, wn = wave / WM % WN, kg = wave / (WM * WN);
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
  // Pieces past K re-read the row's first block; the products left out are
  // made zero on a's side (what is read of w there is w's own row: no new NaN).
  // (A thread stages the same piece of every row it stages.)
  const int ck = ((tid & 7) ^ ((tid >> 4) & 7)) * 16;
  auto step_offset = [&](int kb) { return (unsigned)(kb * 128 + ck < g.K ? kb * 128 : -ck); };
  auto stage = [&](int n, int kb, unsigned k) {   // the n-th of a thread's LA + LB pieces of step kb
    u8* base = smem + kb % R * ((BM + BN) * 128) + wave * 1024;
    if (n < LA) __builtin_amdgcn_global_load_lds((GlbP)(ga + (oa[n < LA ? n : 0] + k)), (LdsP)(base + n * kThreads * 16), 16, 0, 0);
    else __builtin_amdgcn_global_load_lds((GlbP)(gw + (ob[n < LA ? 0 : n - LA] + k)), (LdsP)(base + BM * 128 + (n - LA) * kThreads * 16), 16, 0, 0);
  };
  // The rows' scales go through LDS four steps at a time, one row a thread: a
  // scale a lane straight from memory touched a cache line a row in every step
  // (8192 x 12288 x 4096: 524 us).
  constexpr int kSc = R * (BM + BN) * 128;   // their place in LDS: two sets of [BM][4]
  static_assert(kThreads >= BM, "a thread a row");
  const bool sc4 = (KB & 3) == 0 && (g.lsa & 3) == 0 && (reinterpret_cast<uintptr_t>(g.sa) & 15) == 0;
  const float* gsa = g.sa + m0 * g.lsa;
  const unsigned os = (unsigned)min(tid, rows - 1) * (unsigned)g.lsa;
  auto stage_scales = [&](int kq) {   // of steps 4 kq .. 4 kq + 3
    if (wave * 64 >= BM) return;
    u8* base = smem + kSc + (kq & 1) * (BM * 16);
    if (sc4) {
      __builtin_amdgcn_global_load_lds((GlbP)(gsa + 4 * kq + os), (LdsP)(base + wave * 1024), 16, 0, 0);
    } else {   // set kq as [4][BM]
#pragma unroll
      for (int e = 0; e < 4; ++e)
        __builtin_amdgcn_global_load_lds((GlbP)(gsa + min(4 * kq + e, KB - 1) + os), (LdsP)(base + e * (BM * 4) + wave * 256), 4, 0, 0);
    }
  };
  const int row_at = sc4 ? 16 : 4, step_at = sc4 ? 4 : BM * 4;   // bytes between rows, between steps
  const u8* sc = smem + kSc + (wm * (BM / WM) + r) * row_at;
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
  stage_scales(0);
#pragma unroll
  for (int kb = 0; kb < R - U; ++kb) {
    const unsigned k = step_offset(min(kb, KB - 1));
#pragma unroll
    for (int n = 0; n < LA + LB; ++n) stage(n, kb, k);
  }
  float ws64 = 0.f;
  for (int k0 = 0; k0 < KB; k0 += U) {
    // This wave's pieces of these steps are in LDS (a barrier alone does not
    // wait for loads to LDS): behind them are at least those of R - 2 U steps.
    // Every wave has read what it needs of the set before.
    // (A fence in front of the barrier would wait for all loads in flight.)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((R - 2 * U) * (LA + LB)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if ((k0 & 63) == 0) {
      ws64 = sw[min(k0 + lane, KB - 1)];   // a lane a step
      asm volatile("" : "+v"(ws64));       // (waited for here, not in every step)
    }
    if ((k0 & 3) == 0 && k0 + 4 < KB) stage_scales((k0 >> 2) + 1);
#pragma unroll
    for (int u = 0; u < U; u += KG) {
      const int kb = k0 + u + kg;
      if (U > 1 && kb >= KB) break;
      const float ws = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws64), kb & 63));
      float f[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        f[i] = ws * *reinterpret_cast<const float*>(sc + ((kb >> 2) & 1) * (BM * 16) + (kb & 3) * step_at + i * 16 * row_at);
      unsigned kn[KG];   // (behind the last step its blocks again, unused)
#pragma unroll
      for (int e = 0; e < KG; ++e) kn[e] = step_offset(min(k0 + u + e + R - U, KB - 1));
      const u8* ta = smem + kb % R * ((BM + BN) * 128) + wm * (BM / WM) * 128;
      const u8* tb = ta + (BM - wm * (BM / WM) + wn * (BN / WN)) * 128;
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
          // the coming loads one by one between the first products: issued at once
          // they hold the wave until the cache has taken them (480 us), spread over
          // all products the last ones come late (490; 451 like this)
          constexpr int kAll = KG * (LA + LB), kEach = (kAll + NT * MT - 1) / (NT * MT);
#pragma unroll
          for (int n = q * kEach; n < (q + 1) * kEach && n < kAll; ++n)
            stage(n % (LA + LB), k0 + u + n / (LA + LB) + R - U, kn[n / (LA + LB)]);
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
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load to LDS outlives the work-group
  if constexpr (KG > 1) {
    static_assert((KG - 1) * BM * BN * 4 <= R * (BM + BN) * 128, "room for the sums");
    f32x4* part = reinterpret_cast<f32x4*>(smem) + (wave % (WM * WN)) * (NT * MT * 64) + lane;
    __syncthreads();
    if (kg)
#pragma unroll
      for (int q = 0; q < NT * MT; ++q) part[(kg - 1) * (BM * BN / 4) + q * 64] = acc[q / MT][q % MT];
    __syncthreads();
    if (kg) return;
#pragma unroll
    for (int e = 0; e < KG - 1; ++e)
#pragma unroll
      for (int q = 0; q < NT * MT; ++q) acc[q / MT][q % MT] += part[e * (BM * BN / 4) + q * 64];
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = wm * (BM / WM) + i * 16 + r;
    if (row >= rows) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) store_out<T>(g, m0 + row, n0 + wn * (BN / WN) + j * 16 + 4 * grp, acc[j][i]);
  }
}

// ---------------------------------------------------------------- few outputs
// 16 rows and 16 NT outputs a work-group; its WK waves take every WK-th block of
// K straight from memory and are joined through LDS.
template <typename T, int NT, int WK>
__global__ __launch_bounds__(64 * WK) void gemm8_rows_kernel(const Gemm8Args g, unsigned tn) {
  __shared__ f32x4 part[WK][NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, grp = lane >> 4;
  const unsigned rb = blockIdx.x / tn;
  const long long m0 = 16LL * rb;
  const int n0 = (int)(blockIdx.x - rb * tn) * (16 * NT), KB = (g.K + 127) / 128, cols = min(16 * NT, g.N - n0);
  const int rows = (int)min(16LL, g.M - m0), m = min(r, rows - 1);
  const u8* ga = g.a + m0 * g.lda;
  const float* gsa = g.sa + m0 * g.lsa;
  const u8* gw = g.w + (size_t)n0 * g.K;
  const float* sw = g.sw + (size_t)(n0 / 128) * KB;
  unsigned ow[NT];   // (rows past the last re-read that one)
#pragma unroll
  for (int j = 0; j < NT; ++j) ow[j] = (unsigned)min(j * 16 + r, cols - 1) * (unsigned)g.K + grp * 16;
  const unsigned oa = (unsigned)m * (unsigned)g.lda + grp * 16, os = (unsigned)m * (unsigned)g.lsa;
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = zero4();
  for (int kb = wave; kb < KB; kb += WK) {
    const unsigned k = (unsigned)kb * 128;
    const bool in0 = (int)k + grp * 16 < g.K, in1 = (int)k + grp * 16 + 64 < g.K;
    const i32x4 z{0, 0, 0, 0};
    Frag<T> wb[NT], xa;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      wb[j].set(in0 ? *reinterpret_cast<const i32x4*>(gw + (ow[j] + k)) : z, in1 ? *reinterpret_cast<const i32x4*>(gw + (ow[j] + k + 64)) : z);
    xa.set(in0 ? *reinterpret_cast<const i32x4*>(ga + (oa + k)) : z, in1 ? *reinterpret_cast<const i32x4*>(ga + (oa + k + 64)) : z);
    const float f = gsa[os + (unsigned)kb] * sw[kb];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const f32x4 p = mma128(wb[j], xa);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(p[e], f, acc[j][e]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  for (int j = wave; j < NT; j += WK) {
    f32x4 v = part[0][j][lane];
#pragma unroll
    for (int k = 1; k < WK; ++k) v += part[k][j][lane];
    if (r < rows) store_out<T>(g, m0 + r, n0 + j * 16 + 4 * grp, v);
  }
}

constexpr int kTileThreads = 512;
template <typename T, int BM, int BN, int WM, int WN, int KG, int R, int U>
hipError_t tile_go(const Gemm8Args& g, hipStream_t st) {
  constexpr int kThreads = 64 * WM * WN * KG, kLds = R * (BM + BN) * 128 + 2 * BM * 16;
  static_assert(kThreads == kTileThreads && kLds <= 160 * 1024 && (U == 1 || U == 2 || U == 4) && U % KG == 0 && R >= 2 * U && R - 2 * U <= 4, "LDS, sets of scales");
  const long long tm = (g.M + BM - 1) / BM, tn = (g.N + BN - 1) / BN, n = (tm * tn + 7) / 8 * 8;
  if (n > max_groups(kThreads)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_tile_kernel<T, BM, BN, WM, WN, KG, R, U>), dim3((unsigned)n), dim3(kThreads), kLds, st, g, (unsigned)tm, (unsigned)tn);
  return hipGetLastError();
}

template <typename T, int NT, int WK>
hipError_t rows_go(const Gemm8Args& g, hipStream_t st) {
  const long long tn = (g.N + 16 * NT - 1) / (16 * NT), n = tn * ((g.M + 15) / 16);
  if (n > max_groups(64 * WK)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm8_rows_kernel<T, NT, WK>), dim3((unsigned)n), dim3(64 * WK), 0, st, g, (unsigned)tn);
  return hipGetLastError();
}

// Tiles by the time of a round of 256 work-groups, one a CU, us for K = 4096:
// what a shape takes is its rounds times that.  Measured, 4096 outputs, bf16:
// 256 rows 64 x 64 11.2, 64 x 128 14.0; 512 rows 64 x 128 15.0, 64 x 64 20.5; 1024
// rows 128 x 128 24.5, 64 x 128 28.5; 1536 rows 192 x 128 34.7, 128 x 256 39.2; 2048
// rows 128 x 256 40, 128 x 128 47; 1536 x 8192 192 x 256 55.8, 256 x 256 61.0; 8192 rows
// 256 x 256 131, 128 x 256 148.  fp32: 17 and 23, 24 and 30, 41 and 46, 56 and 65, 64
// and 78; the two largest do not fit the registers there.  Two smaller
// work-groups a CU, each with fewer steps in LDS, took 41 for 2048 rows in 128 x
// 128.
struct TileTime {
  int bm, bn;
  float bf16_us, f32_us;
};
constexpr TileTime kTiles[7] = {{64, 64, 11.f, 16.5f}, {64, 128, 15.f, 24.f}, {128, 128, 24.3f, 41.f}, {192, 128, 34.5f, 56.f}, {128, 256, 39.5f, 62.f},
                                {192, 256, 54.f, 0.f}, {256, 256, 66.f, 0.f}};
template <typename T> constexpr int tile_kinds() { return sizeof(T) == 2 ? 7 : 5; }

template <typename T> float round_us(int i) { return sizeof(T) == 2 ? kTiles[i].bf16_us : kTiles[i].f32_us; }
long long tiles_of(const TileTime& t, long long M, long long N) { return (M + t.bm - 1) / t.bm * ((N + t.bn - 1) / t.bn); }

// The tile that takes least for M x N, and its time.  (Of more work-groups than
// a launch may have: the largest only, which the launch refuses in its turn.)
template <typename T> int best_tile(long long M, long long N, float& least) {
  int best = tile_kinds<T>() - 1;
  least = (float)((tiles_of(kTiles[best], M, N) + 255) / 256) * round_us<T>(best);
  for (int i = 0; i < tile_kinds<T>() - 1; ++i) {
    const long long n = tiles_of(kTiles[i], M, N);
    const float us = (float)((n + 255) / 256) * round_us<T>(i);
    if (us < least && n <= max_groups(kTileThreads) - 8) {
      best = i;
      least = us;
    }
  }
  return best;
}

template <typename T> hipError_t tile_by(int i, const Gemm8Args& g, hipStream_t st) {
  switch (i) {
    case 0: return tile_go<T, 64, 64, 2, 2, 2, 6, 2>(g, st);
    case 1: return tile_go<T, 64, 128, 2, 2, 2, 6, 2>(g, st);
    case 2: return tile_go<T, 128, 128, 4, 2, 1, 4, 1>(g, st);
    case 3: return tile_go<T, 192, 128, 4, 2, 1, 3, 1>(g, st);
    case 4: return tile_go<T, 128, 256, 2, 4, 1, 3, 1>(g, st);
    default: break;
  }
  if constexpr (sizeof(T) == 2) return i == 5 ? tile_go<T, 192, 256, 4, 2, 1, 2, 1>(g, st) : tile_go<T, 256, 256, 4, 2, 1, 2, 1>(g, st);
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t gemm8_go(const Gemm8Args& g, hipStream_t st) {
  // Few outputs: 16 rows and 16 or 32 columns a work-group where those are no
  // more than the CUs (us, beside 64 x 64 tiles: 64 x 1024 x 4096 7.7 and 13.4, in fp32
  // 7.7 and 16.2; 64 x 2048: 8.8 and 13.6, 9.0 and 16.2; 16 x 8192: 9.9 and 12.4, 10.0
  // and 16.1).  Few rows of more outputs: 64 columns, so that the weights come in
  // longer runs (8 x 12288 x 4096: 13.1; 32 columns 15.5, 16 columns 15.2, tiles 13.4; in
  // fp32 13.5; 15.6, 15.6, 16.6).  The rule goes by the work-groups alone and is not
  // the best everywhere: 16 x 12288 in bf16 14.1, tiles 13.6; 1 x 8192 x 8192 by 32
  // columns 19.5, by 16 15.0.
  const long long rb = (g.M + 15) / 16;
  if (rb * ((g.N + 15) / 16) <= 256) return rows_go<T, 1, 8>(g, st);
  if (rb * ((g.N + 31) / 32) <= 256) return rows_go<T, 2, 8>(g, st);
  if (g.M <= 16 && g.N <= 1 << 27) return rows_go<T, 4, 16>(g, st);   // (beyond, more work-groups than a launch has)
  float one = 0.f;
  int main_tile = best_tile<T>(g.M, g.N, one), rest_tile = 0;
  // Where a last round would be mostly empty: whole rounds of one tile, and the
  // columns that are left in a second launch (kGap us) with theirs
  // (8191 x 8480 x 4096: 281 us; one launch 305).
  constexpr float kGap = 4.f;
  const float k = (float)g.K / 4096.f;
  int cut = 0;
  for (int i = 0; i < tile_kinds<T>(); ++i) {
    const TileTime& t = kTiles[i];
    const long long rows = (g.M + t.bm - 1) / t.bm, rounds = tiles_of(t, g.M, g.N) / 256, cols = rounds * 256 / rows * t.bn;
    if (rounds == 0 || cols == 0 || cols >= g.N || cols % 128) continue;   // (scales are of 128 columns)
    float rest;
    const int r = best_tile<T>(g.M, g.N - cols, rest);
    const float us = (float)rounds * round_us<T>(i) + rest + kGap / k;
    if (us < one) {
      one = us;
      main_tile = i;
      rest_tile = r;
      cut = (int)cols;
    }
  }
  if (!cut) return tile_by<T>(main_tile, g, st);
  Gemm8Args a = g, b = g;
  a.N = cut;
  b.N = g.N - cut;
  b.w += (size_t)cut * g.K;
  b.sw += (size_t)(cut / 128) * ((g.K + 127) / 128);
  b.c = static_cast<T*>(g.c) + cut;
  const hipError_t e = tile_by<T>(main_tile, a, st);
  return e != hipSuccess ? e : tile_by<T>(rest_tile, b, st);
}

}  // namespace

hipError_t launch_gemm8(int out_bf16, const Gemm8Args& g, hipStream_t st) {
  return out_bf16 ? gemm8_go<bf16>(g, st) : gemm8_go<float>(g, st);
}

}  // namespace kda
