// Root-mean-square norm of the residual stream with the residual's addition,
// its output in the input's type or in 8 bits with scales, and its gradients.
//
// A row is one token, D channels:
//   h = x + res, rounded to the stream's type (h = x without a residual)
//   n = w h r,  r = 1 / sqrt(mean(h^2) + eps)
//   y = n, or q = e4m3(n / s) with one s = max |n| / 448 for every 128 channels
// The norm is that of the rounded h, so that the backward, which has h in
// hand, differentiates what the forward computed.
// Backward, u = h r:  dx = r (w dy - u mean(w dy u)) + dh;  dw = sum dy u.
//
// Bound by HBM: one pass, every row read and written once.  A row is held in
// registers by part of a wave (up to 256 channels), a wave (2048), four or
// sixteen, eight neighbouring channels a lane, so 16 lanes hold the 128 channels
// of a scale and its maximum stays inside a DPP row.  All arithmetic is fp32 up to the
// one rounding of each output.  65536 x 4096 bf16 with the residual to 8 bits 322
// us (7 bytes a channel, 5.9 TB/s), 8191 x 2056 with an fp32 stream 39 us (5.2),
// gradients of 32768 x 4096 bf16 with dw 192 us (5.6); 256 rows are bound by the
// launch.
#include "kda_rows.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;
// A block whose largest |n| is below this has scale 1 and zeros (448 / max
// would overflow below 2^-119).
constexpr float kBlockMin = 0x1p-100f;

template <typename T> struct Raw8;   // eight channels as loaded
template <> struct Raw8<bf16> {
  bf16x8 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const bf16x8*>(p); }
  __device__ __forceinline__ float at(int i) const { return (float)v[i]; }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = load4(p);
    b = load4(p + 4);
  }
  __device__ __forceinline__ float at(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};

// L: the lanes that hold a row, 8 to 64 of a wave or those of several waves.
// Sum over a row's lanes of this wave, in all of them.
template <int L> __device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int off = 1; off < (L < 64 ? L : 64); off <<= 1) x += __shfl_xor(x, off);
  return x;
}

// Largest x >= 0 of each 16 lanes (of 8 with L = 8), in all of them.
template <int L> __device__ __forceinline__ float max16(float x) {
  x = fmaxf(x, dpp_f<0xB1>(x));    // quad_perm [1,0,3,2]
  x = fmaxf(x, dpp_f<0x4E>(x));    // quad_perm [2,3,0,1]
  x = fmaxf(x, dpp_f<0x141>(x));   // row_half_mirror
  return L == 8 ? x : fmaxf(x, dpp_f<0x140>(x));   // row_mirror
}

// Sums over the W waves that share a row.  `red` has two sets of slots, used
// by turns, so one barrier a row is enough: a wave overwrites a set only
// behind the next row's barrier, which every wave passes after its reads.
constexpr int waves_of(int L) { return L > 64 ? L / 64 : 1; }
template <int L, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float (*red)[N][waves_of(L)], int turn, int wave) {
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = lane_sum<L>(s[k]);
  if (L <= 64) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[turn][k][wave] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    s[k] = 0.f;
#pragma unroll
    for (int q = 0; q < waves_of(L); ++q) s[k] += red[turn][k][q];
  }
}

// Vector j of a row's lane: channels 8 (j L + lane) .. + 7.
template <int L> __device__ __forceinline__ int channel(int j, int lane) { return 8 * (j * L + lane); }

template <int NV, int L> __device__ __forceinline__ void load_weights(const float* w, int D, int lane, float (&wv)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = channel<L>(j, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) wv[j][i] = 1.f;
    if (w && c < D) Rows<float, 8>::load(w + c, wv[j]);
  }
}

// Threads of a work-group, and the rows it holds at once.
constexpr int group_threads(int L) { return L > kThreads ? L : kThreads; }
constexpr int group_rows(int L) { return group_threads(L) / L; }
// A thread's lane in its row, and its row of the work-group's.
template <int L> __device__ __forceinline__ int row_lane() { return L > 64 ? threadIdx.x : threadIdx.x % L; }
template <int L> __device__ __forceinline__ int row_of() { return L > 64 ? 0 : threadIdx.x / L; }

// T: type of x and of y; TH: type of the stream (res and h).
template <typename T, typename TH, bool kRes, bool kFp8, int NV, int L>
__global__ __launch_bounds__(group_threads(L)) void norm_fwd_kernel(const NormArgs a, long long groups) {
  __shared__ float red[2][1][waves_of(L)];
  constexpr int kPer = group_rows(L);
  const int lane = row_lane<L>(), wave = threadIdx.x >> 6, D = a.D;
  const float inv = 1.f / (float)D;
  float w[NV][8];
  load_weights<NV, L>(a.w, D, lane, w);
  int turn = 0;
  for (long long m = (long long)blockIdx.x * kPer + row_of<L>(); m < a.rows; m += groups * kPer, turn ^= 1) {
    Raw8<T> x[NV];
    Raw8<TH> r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel<L>(j, lane);
      if (c < D) {
        x[j].load((const T*)a.x + m * a.ldx + c);
        if (kRes) r[j].load((const TH*)a.res + m * a.ldr + c);
      }
    }
    float h[NV][8], sq[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel<L>(j, lane);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
      if (c < D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = kRes ? to_f32(from_f32<TH>(x[j].at(i) + r[j].at(i))) : x[j].at(i);
        if (kRes) Rows<TH, 8>::store((TH*)a.sum + m * D + c, h[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sq[0] = fmaf(h[j][i] * inv, h[j][i], sq[0]);
    }
    row_sum<L, 1>(sq, red, turn, wave);
    const float rn = 1.f / sqrtf(sq[0] + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel<L>(j, lane);
      float n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = h[j][i] * rn * w[j][i];
      if (kFp8) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(n[i]));
        top = max16<L>(top);   // (lanes past D hold zeros)
        const bool live = top >= kBlockMin;
        const float q = live ? kE4m3Max / top : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = live || n[i] != n[i] ? n[i] * q : 0.f;
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(n[0], n[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(n[2], n[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(n[4], n[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(n[6], n[7], hi, true);
        if (c < D) {
          *reinterpret_cast<int2*>((unsigned char*)a.y + m * D + c) = make_int2(lo, hi);
          if ((lane & 15) == 0) a.scale[m * ((D + 127) / 128) + (c >> 7)] = live ? top / kE4m3Max : 1.f;
        }
      } else if (c < D) {
        Rows<T, 8>::store((T*)a.y + m * D + c, n);
      }
    }
  }
}

// Gradients.  T: type of h, dh and dx; TG: type of dy.  The lanes that hold a
// row walk their rows and keep the sums of dw of their channels; they are
// partial rows of the workspace.  (fp32, as the eight to 32 sums of a lane would
// take twice the registers in 64 bits: up to rows / 512 terms one after the other,
// off by that many units of the terms' absolute sum at worst; the partial rows are
// summed in 64 bits.)
template <typename T, typename TG, int NV, int L>
__global__ __launch_bounds__(group_threads(L)) void norm_bwd_kernel(const NormArgs a, long long groups) {
  __shared__ float red[2][2][waves_of(L)];
  constexpr int kPer = group_rows(L);
  const int lane = row_lane<L>(), wave = threadIdx.x >> 6, D = a.D;
  const float inv = 1.f / (float)D;
  float w[NV][8], dw[NV][8];
  load_weights<NV, L>(a.w, D, lane, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  int turn = 0;
  for (long long m = (long long)blockIdx.x * kPer + row_of<L>(); m < a.rows; m += groups * kPer, turn ^= 1) {
    Raw8<T> h[NV], s[NV];
    Raw8<TG> g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel<L>(j, lane);
      if (c < D) {
        h[j].load((const T*)a.x + m * a.ldx + c);
        g[j].load((const TG*)a.dy + m * D + c);
        if (a.res) s[j].load((const T*)a.res + m * D + c);
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (channel<L>(j, lane) < D)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = h[j].at(i) * inv;
          sum[0] = fmaf(v, h[j].at(i), sum[0]);
          sum[1] = fmaf(g[j].at(i) * w[j][i], v, sum[1]);
        }
    row_sum<L, 2>(sum, red, turn, wave);
    // dx = r (w dy - u mean(w dy h) r): no power of r alone
    const float rn = 1.f / sqrtf(sum[0] + a.eps), k = sum[1] * rn;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = channel<L>(j, lane);
      if (c >= D) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = h[j].at(i) * rn, gy = g[j].at(i);
        dw[j][i] = fmaf(gy, u, dw[j][i]);
        o[i] = rn * (gy * w[j][i] - u * k);
        if (a.res) o[i] += s[j].at(i);
      }
      Rows<T, 8>::store((T*)a.y + m * D + c, o);
    }
  }
  if (!a.part) return;
  // one partial row a wave (a work-group where several waves hold a row)
  const long long holder = L > 64 ? blockIdx.x : (long long)blockIdx.x * (kThreads / 64) + wave;
#pragma unroll
  for (int off = L; off < 64; off <<= 1)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[j][i] += __shfl_xor(dw[j][i], off);
  if ((threadIdx.x & 63) >= L) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = channel<L>(j, lane);
    if (c < D) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<f32x4*>(a.part + holder * D + c + 4 * q) = f32x4{dw[j][4 * q], dw[j][4 * q + 1], dw[j][4 * q + 2], dw[j][4 * q + 3]};
    }
  }
}

// Work-groups at most.  Forward: a row (of up to 2048 channels four and more)
// each, as the next row's loads then come from another work-group while this one
// sums (64K rows of 4096 to 8 bits: 328 us; 8192 work-groups 356, 2048 386); rows of
// sixteen waves leave no room for another and walk on (8192 rows of 16384: 169;
// a row each 176).  Backward, where each keeps a partial row of dw (64K rows of
// 4096: 380 us; 1024 448, 256 460).
constexpr int kBwdGroups = 512;
int fwd_groups(int D) { return D <= 8192 ? 1 << 20 : 2048; }

// Lanes that hold a row of D channels, and their vectors of eight.  Short rows
// share a wave (2^20 rows of 64 to 8 bits: 55 us, a wave each 354).
int row_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : D <= 2048 ? 64 : D <= 8192 ? 256 : 1024; }
unsigned norm_groups(long long rows, int D, int most) {
  const int per = group_rows(row_lanes(D));
  const long long g = (rows + per - 1) / per;
  return (unsigned)(g < most ? g : most);
}
long long part_rows(long long rows, int D) {
  return (long long)norm_groups(rows, D, kBwdGroups) * (row_lanes(D) > 64 ? 1 : kThreads / 64);
}

// The instance for rows of D channels.
#define KDA_NORM_LAUNCH(kernel, ...) hipLaunchKernelGGL((kernel<__VA_ARGS__>), grid, th, 0, st, a, (long long)groups)
#define KDA_NORM_BY_WIDTH(kernel, ...)                                    \
  do {                                                                    \
    const dim3 grid(groups), th(group_threads(row_lanes(a.D)));           \
    if (a.D <= 64) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 1, 8);            \
    else if (a.D <= 128) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 1, 16);     \
    else if (a.D <= 256) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 1, 32);     \
    else if (a.D <= 512) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 1, 64);     \
    else if (a.D <= 1024) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 2, 64);    \
    else if (a.D <= 2048) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 4, 64);    \
    else if (a.D <= 4096) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 2, 256);   \
    else if (a.D <= 8192) KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 4, 256);   \
    else KDA_NORM_LAUNCH(kernel, __VA_ARGS__, 2, 1024);                   \
    return hipGetLastError();                                             \
  } while (0)

template <typename T, typename TH, bool kRes, bool kFp8>
hipError_t fwd_go(const NormArgs& a, hipStream_t st) {
  const unsigned groups = norm_groups(a.rows, a.D, fwd_groups(a.D));
  KDA_NORM_BY_WIDTH(norm_fwd_kernel, T, TH, kRes, kFp8);
}
template <typename T, typename TH, bool kRes>
hipError_t fwd_out(const NormArgs& a, hipStream_t st) {
  return a.scale ? fwd_go<T, TH, kRes, true>(a, st) : fwd_go<T, TH, kRes, false>(a, st);
}
template <typename T, typename TG>
hipError_t bwd_go(const NormArgs& a, hipStream_t st) {
  const unsigned groups = norm_groups(a.rows, a.D, kBwdGroups);
  KDA_NORM_BY_WIDTH(norm_bwd_kernel, T, TG);
}

}  // namespace

hipError_t launch_norm_fwd(int is_bf16, int sum_bf16, const NormArgs& a, hipStream_t st) {
  if (!a.res) return is_bf16 ? fwd_out<bf16, bf16, false>(a, st) : fwd_out<float, float, false>(a, st);
  if (!is_bf16) return fwd_out<float, float, true>(a, st);
  return sum_bf16 ? fwd_out<bf16, bf16, true>(a, st) : fwd_out<bf16, float, true>(a, st);
}

size_t norm_bwd_workspace_bytes(long long rows, int D) {
  return ((size_t)part_rows(rows, D) * D * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_norm_bwd(int is_bf16, int dy_bf16, const NormArgs& a, float* dw, hipStream_t st) {
  hipError_t e;
  if (is_bf16) e = dy_bf16 ? bwd_go<bf16, bf16>(a, st) : bwd_go<bf16, float>(a, st);
  else e = dy_bf16 ? bwd_go<float, bf16>(a, st) : bwd_go<float, float>(a, st);
  if (e != hipSuccess || !a.part) return e;
  return launch_sum_rows(a.part, (size_t)part_rows(a.rows, a.D), (unsigned)a.D, 0, 0, dw, nullptr, nullptr, st);
}

}  // namespace kda
