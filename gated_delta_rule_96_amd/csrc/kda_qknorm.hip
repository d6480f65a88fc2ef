// Norms of query and key heads with the position rotation in the same pass,
// and their gradients.
//
// A row is one head of one token, d channels:
//   n = w * x r,  r = 1 / sqrt(mean(x^2) + eps) or 1 / sqrt(sum(x^2) + eps)
//   y = R(p) n: channel pairs (a, b) of the first `rot` channels turn by the
//   angle of the token's position, (a cos - b sin, b cos + a sin), with cos and
//   sin read from a table [n_pos][rot / 2]; the pairs are (i, i + rot/2), or
//   the neighbours (2i, 2i + 1).
// Backward: dn = R(-p) dy;  dw = sum dn x r;
//   dx = r w dn - x r^3 (sum w dn x) / d   (without the 1/d for the sum norm).
//
// Bound by HBM: one pass, every row read and written once.  A group of L
// lanes holds a row, eight channels a lane chosen so that a pair's two halves
// are in the same lane (two four-channel accesses): the rotation needs no
// lane traffic, the norm a sum over L lanes.  A wave takes 64/L x R heads of
// one token, so a token's table row is read once for all of them.  Rows are
// in fp32 between the loads and the one rounding at the end.
// Measured (bf16): 65536 tokens x 64 heads of 128 382 us (5.7 TB/s); gradients
// of 32768 tokens x 32 heads 205 us (5.2 TB/s); a token for 256 sequences x 40
// heads 4.5 us (14 through the Python binding): two memory trips one behind the
// other, position and table, in a launch of a tenth of the card.
#include "kda_rows.h"

namespace kda {

namespace {

constexpr int kQkThreads = 256;
// Heads a lane group holds at once: forward (64K tokens x 64 heads of 128: 370
// us; two 382, eight 408; fewer heads would like fewer: 8 query heads and 1 key
// head 92, two 70) and backward (32K tokens x 32 heads: 206 us; one 217, four
// 244; 64K x 8 + 1 heads: 150; 145, 284).
constexpr int kQkRows = 4, kBwdRows = 2;
// Work-groups of the backward at most, each with a partial row of dw (same
// cases: 206 and 150 us; 768 210 and 177, 1536 227 and 189, 2048 212 and 156:
// more do not all run at once and end unevenly).
constexpr int kBwdGroups = 1024;

// Where a lane's eight channels are.
struct LanePlace {
  int off0, off1, ti;   // channels off0..+3, off1..+3; first of its four table columns
  bool live, turn;
};
template <bool kInter> __device__ __forceinline__ LanePlace lane_place(const QkArgs& a, int c) {
  LanePlace p;
  p.live = 8 * c < a.d;
  p.turn = 8 * c < a.rot;
  p.ti = 4 * c;
  p.off0 = 8 * c;
  p.off1 = 8 * c + 4;
  if (!kInter && p.turn) {
    p.off0 = 4 * c;
    p.off1 = a.rot / 2 + 4 * c;
  }
  return p;
}

struct Turn {
  float c[4], s[4];
};
// A token's table columns of this lane; NaN for a position outside the table.
__device__ __forceinline__ Turn load_turn(const QkArgs& a, const LanePlace& p, long long m) {
  Turn t;
  if (!(p.live && p.turn)) return t;
  const int pos = a.pos ? a.pos[m] : a.pos0 + (int)(m % a.T);
  if (pos < 0 || pos >= a.n_pos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t.c[i] = t.s[i] = __builtin_nanf("");
    return t;
  }
  const size_t at = (size_t)pos * (a.rot / 2) + p.ti;
  const f32x4 c = load4(a.cos + at), s = load4(a.sin + at);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.c[i] = c[i];
    t.s[i] = s[i];
  }
  return t;
}
__device__ __forceinline__ void turn2(float c, float s, float& u, float& v) {
  const float a = u * c - v * s;
  v = v * c + u * s;
  u = a;
}
// x (channels off0..+3 in x[0..3], off1..+3 in x[4..7]) turned by the angle
// (sg = 1) or back (sg = -1).
template <bool kInter>
__device__ __forceinline__ void turn8(const Turn& t, float sg, float (&x)[8]) {
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn2(t.c[i], sg * t.s[i], x[2 * i], x[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn2(t.c[i], sg * t.s[i], x[i], x[4 + i]);
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* row, const LanePlace& p, float (&x)[8]) {
  const f32x4 u = widen4(load4(row + p.off0)), v = widen4(load4(row + p.off1));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = u[i];
    x[4 + i] = v[i];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* row, const LanePlace& p, const float (&x)[8]) {
  __builtin_nontemporal_store(narrow4<T>(f32x4{x[0], x[1], x[2], x[3]}), reinterpret_cast<V4<T>*>(row + p.off0));
  __builtin_nontemporal_store(narrow4<T>(f32x4{x[4], x[5], x[6], x[7]}), reinterpret_cast<V4<T>*>(row + p.off1));
}
__device__ __forceinline__ void load_w(const float* w, const LanePlace& p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 1.f;
  if (w && p.live) load8<float>(w, p, x);
}

template <int L>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) x += __shfl_xor(x, off);
  return x;
}

// Task `task` of a token's: which of q and k, and its first head.
struct Heads {
  long long m;
  int kind, h0;
};
__device__ __forceinline__ Heads task_heads(long long task, unsigned per, unsigned tq, int nh) {
  Heads h;
  h.m = task / per;
  const unsigned r = (unsigned)(task - h.m * per);
  h.kind = r >= tq;
  h.h0 = (int)(h.kind ? r - tq : r) * nh;
  return h;
}

template <typename T, int L, bool kInter>
__global__ __launch_bounds__(kQkThreads) void qk_fwd_kernel(const QkArgs a, unsigned per, unsigned tq, long long first, long long tasks) {
  constexpr int G = 64 / L, NH = G * kQkRows;
  const int lane = threadIdx.x & 63, c = lane & (L - 1), grp = lane / L;
  const long long task = first + (long long)blockIdx.x * (kQkThreads / 64) + (threadIdx.x >> 6);
  if (task >= tasks) return;
  const Heads hs = task_heads(task, per, tq, NH);
  const LanePlace p = lane_place<kInter>(a, c);
  const int H = hs.kind ? a.H[1] : a.H[0];
  const T* x = (const T*)(hs.kind ? a.x[1] : a.x[0]) + hs.m * (hs.kind ? a.ld[1] : a.ld[0]);
  T* y = (T*)(hs.kind ? a.y[1] : a.y[0]) + hs.m * ((long long)H * a.d);
  float v[kQkRows][8];
#pragma unroll
  for (int r = 0; r < kQkRows; ++r) {
    const int h = hs.h0 + r * G + grp;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
    if (p.live && h < H) load8(x + (long long)h * a.d, p, v[r]);
  }
  const Turn t = load_turn(a, p, hs.m);
  float w[8];
  load_w(hs.kind ? a.w[1] : a.w[0], p, w);
  const float inv = a.rms ? 1.f / (float)a.d : 1.f;
#pragma unroll
  for (int r = 0; r < kQkRows; ++r) {
    const int h = hs.h0 + r * G + grp;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(v[r][i] * inv, v[r][i], sq);
    const float rn = 1.0f / sqrtf(lane_sum<L>(sq) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] *= rn * w[i];
    if (p.turn) turn8<kInter>(t, 1.f, v[r]);
    if (p.live && h < H) store8(y + (long long)h * a.d, p, v[r]);
  }
}

// A wave walks its tasks (task, task + number of waves, ...) and keeps the
// sums of dwq and dwk of its lanes' channels; a work-group joins its lane
// groups and waves in a fixed order into one partial row [dwq, dwk].
template <typename T, typename TG, int L, bool kInter>
__global__ __launch_bounds__(kQkThreads) void qk_bwd_kernel(const QkArgs a, unsigned per, unsigned tq, long long tasks) {
  constexpr int G = 64 / L, NH = G * kBwdRows, kWaves = kQkThreads / 64;
  __shared__ float red[kWaves][2][L * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & (L - 1), grp = lane / L;
  const LanePlace p = lane_place<kInter>(a, c);
  const float inv = a.rms ? 1.f / (float)a.d : 1.f;
  float w[2][8], dw[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    load_w(a.w[k], p, w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
  }
  for (long long task = (long long)blockIdx.x * kWaves + wave; task < tasks; task += (long long)gridDim.x * kWaves) {
    const Heads hs = task_heads(task, per, tq, NH);
    const int H = hs.kind ? a.H[1] : a.H[0];
    const T* x = (const T*)(hs.kind ? a.x[1] : a.x[0]) + hs.m * (hs.kind ? a.ld[1] : a.ld[0]);
    const TG* dy = (const TG*)(hs.kind ? a.dy[1] : a.dy[0]) + hs.m * ((long long)H * a.d);
    T* dx = (T*)(hs.kind ? a.y[1] : a.y[0]) + hs.m * ((long long)H * a.d);
    float v[kBwdRows][8], g[kBwdRows][8];
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      const int h = hs.h0 + r * G + grp;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = g[r][i] = 0.f;
      if (p.live && h < H) {
        load8(x + (long long)h * a.d, p, v[r]);
        load8(dy + (long long)h * a.d, p, g[r]);
      }
    }
    const Turn t = load_turn(a, p, hs.m);
    float wk[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wk[i] = hs.kind ? w[1][i] : w[0][i];
      s[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      const int h = hs.h0 + r * G + grp;
      if (p.turn && h < H) turn8<kInter>(t, -1.f, g[r]);
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fmaf(v[r][i] * inv, v[r][i], sq);
        dot = fmaf(g[r][i] * wk[i], v[r][i], dot);
      }
      sq = lane_sum<L>(sq);
      dot = lane_sum<L>(dot);
      // dx = r (w dn - (x r) (sum w dn x) r / d): no power of r alone.  A lane
      // group without a head adds nothing to s (with eps = 0 its r is infinite)
      const float rn = h < H ? 1.0f / sqrtf(sq + a.eps) : 0.f;
      const float k = dot * rn * inv;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = v[r][i] * rn;
        s[i] = fmaf(g[r][i], u, s[i]);
        o[i] = rn * (g[r][i] * wk[i] - u * k);
      }
      if (p.live && h < H) store8(dx + (long long)h * a.d, p, o);
    }
    if (hs.kind) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[1][i] += s[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[0][i] += s[i];
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[k][i];
#pragma unroll
      for (int off = L; off < 64; off <<= 1) v += __shfl_xor(v, off);
      if (grp == 0 && p.live) red[wave][k][(i < 4 ? p.off0 : p.off1 - 4) + i] = v;
    }
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * a.d; j += kQkThreads) {
    const int k = j >= a.d, ch = j - k * a.d;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) v += red[q][k][ch];
    a.part[(size_t)blockIdx.x * (2 * a.d) + j] = v;
  }
}

int row_lanes(int d) {
  int l = 8;
  while (l * 8 < d) l <<= 1;
  return l;
}
struct Tasks {
  unsigned per, tq;
  long long n;
};
Tasks qk_tasks(long long tokens, int Hq, int Hk, int d, int rows) {
  const int nh = 64 / row_lanes(d) * rows;
  Tasks t;
  t.tq = (unsigned)((Hq + nh - 1) / nh);
  t.per = t.tq + (unsigned)((Hk + nh - 1) / nh);
  t.n = tokens * t.per;
  return t;
}
unsigned bwd_groups(long long tasks) {
  const long long g = (tasks + kQkThreads / 64 - 1) / (kQkThreads / 64);
  return (unsigned)(g < kBwdGroups ? g : kBwdGroups);
}

template <typename T, bool kInter>
hipError_t fwd_go(const QkArgs& a, hipStream_t st) {
  const Tasks t = qk_tasks(a.tokens, a.H[0], a.H[1], a.d, kQkRows);
  constexpr int kWaves = kQkThreads / 64;
  for (long long first = 0; first < t.n; first += max_groups(kQkThreads) * kWaves) {   // (launches of one call)
    const long long left = (t.n - first + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(left < max_groups(kQkThreads) ? left : max_groups(kQkThreads))), th(kQkThreads);
    switch (row_lanes(a.d)) {
      case 8: hipLaunchKernelGGL((qk_fwd_kernel<T, 8, kInter>), grid, th, 0, st, a, t.per, t.tq, first, t.n); break;
      case 16: hipLaunchKernelGGL((qk_fwd_kernel<T, 16, kInter>), grid, th, 0, st, a, t.per, t.tq, first, t.n); break;
      case 32: hipLaunchKernelGGL((qk_fwd_kernel<T, 32, kInter>), grid, th, 0, st, a, t.per, t.tq, first, t.n); break;
      default: hipLaunchKernelGGL((qk_fwd_kernel<T, 64, kInter>), grid, th, 0, st, a, t.per, t.tq, first, t.n); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename T, typename TG, bool kInter>
hipError_t bwd_go(const QkArgs& a, unsigned groups, hipStream_t st) {
  const Tasks t = qk_tasks(a.tokens, a.H[0], a.H[1], a.d, kBwdRows);
  const dim3 grid(groups), th(kQkThreads);
  switch (row_lanes(a.d)) {
    case 8: hipLaunchKernelGGL((qk_bwd_kernel<T, TG, 8, kInter>), grid, th, 0, st, a, t.per, t.tq, t.n); break;
    case 16: hipLaunchKernelGGL((qk_bwd_kernel<T, TG, 16, kInter>), grid, th, 0, st, a, t.per, t.tq, t.n); break;
    case 32: hipLaunchKernelGGL((qk_bwd_kernel<T, TG, 32, kInter>), grid, th, 0, st, a, t.per, t.tq, t.n); break;
    default: hipLaunchKernelGGL((qk_bwd_kernel<T, TG, 64, kInter>), grid, th, 0, st, a, t.per, t.tq, t.n); break;
  }
  return hipGetLastError();
}
template <bool kInter>
hipError_t bwd_types(int is_bf16, int dy_bf16, const QkArgs& a, unsigned groups, hipStream_t st) {
  if (!is_bf16) return bwd_go<float, float, kInter>(a, groups, st);
  return dy_bf16 ? bwd_go<bf16, bf16, kInter>(a, groups, st) : bwd_go<bf16, float, kInter>(a, groups, st);
}

}  // namespace

hipError_t launch_qk_fwd(int is_bf16, const QkArgs& a, hipStream_t st) {
  if (a.inter) return is_bf16 ? fwd_go<bf16, true>(a, st) : fwd_go<float, true>(a, st);
  return is_bf16 ? fwd_go<bf16, false>(a, st) : fwd_go<float, false>(a, st);
}

size_t qk_bwd_workspace_bytes(long long tokens, int Hq, int Hk, int d) {
  const size_t n = (size_t)bwd_groups(qk_tasks(tokens, Hq, Hk, d, kBwdRows).n) * 2 * d * sizeof(float);
  return (n + 255) & ~(size_t)255;
}

hipError_t launch_qk_bwd(int is_bf16, int dy_bf16, const QkArgs& a0, float* dwq, float* dwk, hipStream_t st) {
  QkArgs a = a0;
  if (!dwq && !dwk) a.part = nullptr;   // no weight gradient wanted: no partial rows
  const unsigned groups = bwd_groups(qk_tasks(a.tokens, a.H[0], a.H[1], a.d, kBwdRows).n);
  const hipError_t e = a.inter ? bwd_types<true>(is_bf16, dy_bf16, a, groups, st) : bwd_types<false>(is_bf16, dy_bf16, a, groups, st);
  if (e != hipSuccess || !a.part) return e;
  return launch_sum_rows(a.part, groups, (unsigned)a.d, (unsigned)a.d, 0, dwq, dwk, nullptr, st);
}

}  // namespace kda
