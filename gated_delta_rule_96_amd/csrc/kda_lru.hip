// Gated linear recurrence with one state a channel (kda_lru_dev.h has the
// formulas): prompts, packed prompts, single tokens.
//
// A wave holds R tokens of 64 NC channels in registers, a work-group kWaves
// runs of them, one behind the other: a part of a sequence.  Its (P, H) are
// joined over the waves in LDS.  Sequences of several parts run in three
// launches: every part's (P, H), the states that enter the parts, and the
// outputs.
#include "kda_lru_dev.h"

namespace kda {

namespace {

constexpr int kWaves = 8, kR = 16, kPart = kWaves * kR;

// a and u of a wave's run of R tokens from token t on; tokens past the part's
// end leave the state as it is.
template <typename T, int NC, int R>
__device__ __forceinline__ void load_run(const LruArgs& g, const SeqPart& p, const LruLane& l, int t, float (&a)[R][NC], float (&u)[R][NC]) {
  typedef LruPack<T, NC> Pk;
  const LruMode md = lru_mode(g);
  Pk x[R], r[R], i[R];
  if (t < p.t1) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const size_t row = p.start + (size_t)min(t + k, p.t1 - 1);
      x[k] = *reinterpret_cast<const Pk*>((const T*)g.x + row * (size_t)g.ldx + l.cl);
      r[k] = *reinterpret_cast<const Pk*>((const T*)g.r + row * (size_t)g.ldr + l.cl);
      if (md.igate) i[k] = *reinterpret_cast<const Pk*>((const T*)g.i + row * (size_t)g.ldi + l.cl);
    }
  }
  float c[NC];
  lru_coef<NC>(g, l, c);
#pragma unroll
  for (int k = 0; k < R; ++k) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      a[k][j] = 1.f;
      u[k][j] = 0.f;
    }
    if (t + k < p.t1)
#pragma unroll
      for (int j = 0; j < NC; ++j) lru_gates<T>(md, c[j], to_f32(x[k].v[j]), to_f32(r[k].v[j]), md.igate ? to_f32(i[k].v[j]) : 0.f, a[k][j], u[k][j]);
  }
}

// P and H of a run.
template <int NC, int R>
__device__ __forceinline__ void run_sum(const float (&a)[R][NC], const float (&u)[R][NC], float (&P)[NC], float (&H)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    P[j] = a[0][j];
    H[j] = u[0][j];
  }
#pragma unroll
  for (int k = 1; k < R; ++k)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      H[j] = fmaf(a[k][j], H[j], u[k][j]);
      P[j] *= a[k][j];
    }
}

// (P, H) of every part: to seg [items][2][D].
template <typename T, int NC>
__global__ __launch_bounds__(64 * kWaves) void lru_part_kernel(const LruArgs g, const SeqTab s, unsigned slices, float* seg) {
  __shared__ float red[2][kWaves][64 * NC];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned item = blockIdx.x / slices;
  const LruLane l = lru_lane<NC>((int)(blockIdx.x - item * slices), g.D);
  const SeqPart p = seq_part(s, (int)item);
  float a[kR][NC], u[kR][NC], P[NC], H[NC];
  load_run<T, NC, kR>(g, p, l, p.t0 + wave * kR, a, u);
  run_sum<NC, kR>(a, u, P, H);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    red[0][wave][lane * NC + j] = P[j];
    red[1][wave][lane * NC + j] = H[j];
  }
  __syncthreads();
  if (wave || !l.live) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float q = red[0][w][lane * NC + j];
      H[j] = fmaf(q, H[j], red[1][w][lane * NC + j]);
      P[j] *= q;
    }
  float* to = seg + (size_t)item * 2 * g.D + l.c;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    to[j] = P[j];
    to[g.D + j] = H[j];
  }
}

// The states that enter a sequence's parts, over their H; and its final state.
__global__ __launch_bounds__(64) void lru_chain_kernel(const LruArgs g, const SeqTab s, float* seg) {
  const int blocks = (g.D + 63) / 64, li = blockIdx.x / blocks, c = (blockIdx.x - li * blocks) * 64 + threadIdx.x;
  if (c >= g.D) return;
  const int n = s.n0 + li;
  const int i0 = s.n ? s.cc[li] : li * s.parts, i1 = s.n ? s.cc[li + 1] : i0 + s.parts;
  float h = g.h0 ? g.h0[(size_t)n * g.D + c] : 0.f;
#pragma unroll 8
  for (int i = i0; i < i1; ++i) {
    float* at = seg + (size_t)i * 2 * g.D + c;
    const float P = at[0], H = at[g.D];
    at[g.D] = h;
    h = fmaf(P, h, H);
  }
  if (g.ht) g.ht[(size_t)n * g.D + c] = h;
}

// Outputs.  seg null: every sequence is one part.
template <typename T, int NC>
__global__ __launch_bounds__(64 * kWaves) void lru_out_kernel(const LruArgs g, const SeqTab s, unsigned slices, const float* seg) {
  __shared__ float red[2][kWaves][64 * NC];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned item = blockIdx.x / slices;
  const LruLane l = lru_lane<NC>((int)(blockIdx.x - item * slices), g.D);
  const SeqPart p = seq_part(s, (int)item);
  float a[kR][NC], u[kR][NC], P[NC], H[NC], h[NC];
  const float* from = seg ? seg + (size_t)item * 2 * g.D + g.D : g.h0 ? g.h0 + (size_t)p.n * g.D : nullptr;
#pragma unroll
  for (int j = 0; j < NC; ++j) h[j] = from ? from[l.cl + j] : 0.f;
  load_run<T, NC, kR>(g, p, l, p.t0 + wave * kR, a, u);
  run_sum<NC, kR>(a, u, P, H);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    red[0][wave][lane * NC + j] = P[j];
    red[1][wave][lane * NC + j] = H[j];
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int j = 0; j < NC; ++j) h[j] = fmaf(red[0][w][lane * NC + j], h[j], red[1][w][lane * NC + j]);
  if (!l.live) return;
  const int t = p.t0 + wave * kR;
#pragma unroll
  for (int k = 0; k < kR; ++k) {
    LruPack<T, NC> o;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      h[j] = fmaf(a[k][j], h[j], u[k][j]);
      o.v[j] = from_f32<T>(h[j]);
    }
    if (t + k < p.t1) *reinterpret_cast<LruPack<T, NC>*>((T*)g.y + (p.start + (size_t)(t + k)) * g.D + l.c) = o;
  }
  if (!seg && g.ht && wave == kWaves - 1)
#pragma unroll
    for (int j = 0; j < NC; ++j) g.ht[(size_t)p.n * g.D + l.c + j] = h[j];
}

// One token per sequence.
template <typename T, int NC>
__global__ __launch_bounds__(256) void lru_step_kernel(const LruArgs g, unsigned B, unsigned CG) {
  const unsigned id = blockIdx.x * 256 + threadIdx.x, n = id / CG;
  if (n >= B) return;
  const int ch = (int)(id - n * CG) * NC;
  typedef LruPack<T, NC> Pk;
  const LruMode md = lru_mode(g);
  const Pk x = *reinterpret_cast<const Pk*>((const T*)g.x + n * (size_t)g.ldx + ch), r = *reinterpret_cast<const Pk*>((const T*)g.r + n * (size_t)g.ldr + ch);
  Pk i = x, o;
  if (md.igate) i = *reinterpret_cast<const Pk*>((const T*)g.i + n * (size_t)g.ldi + ch);
  const size_t at = (size_t)n * g.D + ch;
  const LruPack<float, NC> h0 = *reinterpret_cast<const LruPack<float, NC>*>(g.h0 + at);
  LruPack<float, NC> ht;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float a, u;
    lru_gates<T>(md, g.c ? g.c[ch + j] : 0.f, to_f32(x.v[j]), to_f32(r.v[j]), to_f32(i.v[j]), a, u);
    ht.v[j] = fmaf(a, h0.v[j], u);
    o.v[j] = from_f32<T>(ht.v[j]);
  }
  *reinterpret_cast<Pk*>((T*)g.y + at) = o;
  *reinterpret_cast<LruPack<float, NC>*>(g.ht + at) = ht;
}

// Whether rows may be read and written two channels at a time.
bool pairs(const LruArgs& a, size_t esz) {
  if (a.D % 2 || a.ldx % 2 || a.ldr % 2 || (a.i && a.ldi % 2)) return false;
  for (const void* p : {a.x, a.r, a.i, (const void*)a.y})
    if (reinterpret_cast<uintptr_t>(p) % (2 * esz)) return false;
  return true;
}

template <typename T, int NC>
hipError_t fwd_go(const LruArgs& a, const int* cu, int N, int B, int T_, float* seg, hipStream_t st) {
  const unsigned slices = (unsigned)((a.D + 64 * NC - 1) / (64 * NC));
  if (!seq_tabs_fit(cu, N, B, T_, kPart, max_groups(64 * kWaves) / slices)) return hipErrorInvalidConfiguration;
  const int end = cu ? N : B;
  for (int n = 0; n < end;) {
    SeqTab s;
    n = make_seq_tab(s, cu, N, n, B, T_, kPart);
    const int seqs = s.n ? s.n : B;
    const bool one = s.items == seqs;   // no sequence has a second part
    const dim3 grid((unsigned)s.items * slices), th(64 * kWaves);
    if (!one) {
      hipLaunchKernelGGL((lru_part_kernel<T, NC>), grid, th, 0, st, a, s, slices, seg);
      hipLaunchKernelGGL(lru_chain_kernel, dim3((unsigned)(a.D + 63) / 64 * seqs), dim3(64), 0, st, a, s, seg);
    }
    hipLaunchKernelGGL((lru_out_kernel<T, NC>), grid, th, 0, st, a, s, slices, one ? nullptr : seg);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int NC>
hipError_t step_go(const LruArgs& a, int B, hipStream_t st) {
  const unsigned CG = (unsigned)(a.D / NC);
  const long long n = ((long long)B * CG + 255) / 256;
  if (n > max_groups(256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((lru_step_kernel<T, NC>), dim3((unsigned)n), dim3(256), 0, st, a, (unsigned)B, CG);
  return hipGetLastError();
}

}  // namespace

size_t lru_workspace_bytes(int is_packed, int N, int B, int T, int D) {
  const size_t items = is_packed ? (size_t)T / kPart + (size_t)N : (size_t)B * (((size_t)T + kPart - 1) / kPart);
  return (items * 2 * D * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_lru_fwd(int is_bf16, const LruArgs& a, const int* cu, int N, int B, int T, void* workspace, hipStream_t st) {
  float* seg = static_cast<float*>(workspace);
  if (is_bf16) return pairs(a, 2) ? fwd_go<bf16, 2>(a, cu, N, B, T, seg, st) : fwd_go<bf16, 1>(a, cu, N, B, T, seg, st);
  return pairs(a, 4) ? fwd_go<float, 2>(a, cu, N, B, T, seg, st) : fwd_go<float, 1>(a, cu, N, B, T, seg, st);
}

hipError_t launch_lru_step(int is_bf16, const LruArgs& a, int B, hipStream_t st) {
  if (is_bf16) return pairs(a, 2) ? step_go<bf16, 2>(a, B, st) : step_go<bf16, 1>(a, B, st);
  return pairs(a, 4) ? step_go<float, 2>(a, B, st) : step_go<float, 1>(a, B, st);
}

}  // namespace kda
