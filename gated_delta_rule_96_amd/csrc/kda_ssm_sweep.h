// State sweeps of the scan: the states alone, along the tokens or (gradients)
// against them, in parts that a small kernel chains.
//
//   along:    S <- exp(cum_Q) S + sum_j exp(cum_Q - cum_j) dt_j B_j x_j^T
//   against: dS <- exp(cum_Q) dS + sum_i exp(cum_i) C_i dy_i^T
// chunk by chunk (cum: the chunk's running sums of dt A).
#pragma once
#include "kda_ssm_dev.h"

namespace kda {
namespace {   // a copy of the kernels per translation unit

struct SweepArgs {
  SsmArgs f;                  // dt, A, bias, softplus, H, G, and the workspace
  const void *rows, *cols;    // [tokens][G][dk] (B, or C) and [tokens][H][dv] (x, or dy)
  long long ldrows, ldcols;
  const float* from;          // [N][H][dk][dv]: state before the first / behind the last token, or null
  float* to;                  // state at the other end, or null
  float* at;                  // [chunks][H][dk][dv]: the state entering every chunk
  int subs;                   // work-groups (and slots) a part's own sum is split over, in token order
};

template <typename T, int DK, int DV>
struct SweepLds {
  static constexpr int PK = RowTile<T, DK>::kPitch, PV = RowTile<T, DV>::kPitch;
  T b[kQ * PK];
  T x[kQ * PV];
  float w[kQ];
};

// kKeep: starts from the part's true state, keeps the state entering every
// chunk (along: before it; against: behind it) and the one at the far end.
// Otherwise the own sum (from zero) and decay of each 1/subs of a part, for
// every part another one follows.  kLow: State::update.
template <typename T, int DK, int DV, bool kRev, bool kKeep, bool kLow>
__global__ __launch_bounds__(kSsmThreads, sizeof(T) == 2 ? 2 : 1) void ssm_sweep_kernel(const SweepArgs a, const SeqTab sq) {
  typedef SweepLds<T, DK, DV> Lds;
  typedef State<DK, DV, false> St;
  __shared__ __align__(16) char smem[sizeof(Lds)];
  Lds& sm = *reinterpret_cast<Lds*>(smem);
  const SsmArgs& f = a.f;
  ItemHead w;
  if (!item_head(sq.items * (kKeep ? 1 : a.subs), f.H, w)) return;
  const int sub = kKeep ? 0 : w.item % a.subs;
  if (!kKeep) w.item /= a.subs;
  SeqPart p = seq_part(sq, w.item);
  const bool final_part = kRev ? p.first : p.last, start_part = kRev ? p.last : p.first;
  if (!kKeep) {
    if (final_part) return;
    // every other part ends where the next begins: along the tokens it has
    // sq.part of them (a whole number of chunks for each share)
    const int len = (p.t1 - p.t0) / a.subs;
    p.t0 += sub * len;
    p.t1 = p.t0 + len;
  }
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int h = w.h, grp = h / (f.H / f.G);
  const double a2 = (double)f.A[h] * 1.4426950408889634074;
  const float bias = f.bias ? f.bias[h] : 0.f;
  const T* x = (const T*)a.cols + p.start * (size_t)a.ldcols + (size_t)h * DV;
  const T* bm = (const T*)a.rows + p.start * (size_t)a.ldrows + (size_t)grp * DK;
  const T* dt = (const T*)f.dt + p.start * (size_t)f.lddt + h;
  constexpr size_t sd = (size_t)DK * DV;
  // slot of this part's own sum, which becomes the next part's start
  const size_t slot = ((size_t)(w.item - p.li - (kRev ? 1 : 0)) * a.subs + sub) * f.H + h;
  St S;
  if (!kKeep) S.zero();
  else if (!start_part) S.load(f.seg + (kRev ? slot + (size_t)a.subs * f.H : slot - (size_t)a.subs * f.H) * sd);
  else if (a.from) S.load(a.from + ((size_t)p.n * f.H + h) * sd);
  else S.zero();
  double total = 0.0;

  RowTile<T, DK> rb;
  RowTile<T, DV> rx;
  float raw = 0.f;
  auto fetch = [&](int t) {
    const int n = p.t1 - t;
    rb.load(bm + (size_t)t * (size_t)a.ldrows, a.ldrows, n, tid);
    rx.load(x + (size_t)t * (size_t)a.ldcols, a.ldcols, n, tid);
    raw = lane < n ? to_f32(dt[(size_t)(t + lane) * (size_t)f.lddt]) : 0.f;
  };
  const int nch = (p.t1 - p.t0 + kQ - 1) / kQ;
  const int chunk0 = (sq.n ? sq.cb[p.li] : p.li * sq.chunks) + p.t0 / kQ;
  auto start = [&](int k) { return p.t0 + kQ * (kRev ? nch - 1 - k : k); };
  if (nch > 0) fetch(start(0));
  for (int k = 0; k < nch; ++k) {
    const int t = start(k), n = min(p.t1 - t, kQ);
    StepSize s = step_size(raw, bias, f.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const double cum = wave_scan(s.a), last = lane63(cum);
    __syncthreads();   // the chunk before is done with LDS
    rb.store(sm.b, tid);
    rx.store(sm.x, tid);
    if (wave == 0) sm.w[lane] = kRev ? exp2_of(cum) : exp2_of(last - cum) * s.dt;
    if (k + 1 < nch) fetch(start(k + 1));
    if (kKeep) S.store(a.at + ((size_t)(chunk0 + (t - p.t0) / kQ) * f.H + h) * sd);
    __syncthreads();
    Slab<T> xs[2][St::NT];
    St::template slabs<PadTile<T, DV>>(sm.x, xs);
    Split<T> xw[2][St::NT];
    St::weigh(xs, sm.w, xw);
    S.template update<kLow, PadTile<T, DK>>(exp2_of(last), sm.b, xw);
    total += last;
  }
  if (!kKeep) {
    S.store(f.seg + slot * sd);
    if (tid == 0) f.sum[slot] = total;
  } else if (final_part && a.to) {
    S.store(a.to + ((size_t)p.n * f.H + h) * sd);
  }
}

// Chains a sequence's parts: a part's own sum becomes the state the next part
// (along or against the tokens) starts from.  One thread a four-column piece
// of one (sequence, head).
template <bool kRev>
__global__ __launch_bounds__(256) void ssm_chain_kernel(const SweepArgs a, const SeqTab sq, int sd4) {
  const unsigned per = (unsigned)(sd4 / 256);
  const unsigned nh = blockIdx.x / per;
  const int H = a.f.H, li = (int)(nh / (unsigned)H), h = (int)(nh - (unsigned)li * H);
  const int e = (int)((blockIdx.x - nh * per) * 256 + threadIdx.x);
  const int first = sq.n ? sq.cc[li] : li * sq.parts, parts = sq.n ? sq.cc[li + 1] - first : sq.parts;
  if (parts < 2) return;
  const size_t n = (size_t)(sq.n ? sq.n0 + li : li);
  f32x4 s = a.from ? load4(a.from + ((n * H + h) * sd4 + e) * 4) : zero4();
  f32x4* seg = reinterpret_cast<f32x4*>(a.f.seg);
  // where the final state replaces the first one, the first part may start
  // after the last one has written: it reads this copy
  if (!kRev && a.f.start) reinterpret_cast<f32x4*>(a.f.start)[((size_t)(first - li) * a.subs * H + h) * sd4 + e] = s;
  for (int k = 0; k + 1 < parts; ++k) {
    const size_t slot = (size_t)(first - li + (kRev ? parts - 2 - k : k)) * a.subs * H + h;
    for (int q = 0; q < a.subs; ++q) s = s * exp2_of(a.f.sum[slot + (size_t)q * H]) + seg[(slot + (size_t)q * H) * sd4 + e];
    seg[slot * sd4 + e] = s;
  }
}

template <typename T, int DK, int DV, bool kRev, bool kKeep, bool kLow>
hipError_t launch_sweep(const SweepArgs& a, const SeqTab& s, hipStream_t st) {
  dim3 grid;
  if (s.items > 0x7fffffff / 2 || !item_head_grid(s.items * (kKeep ? 1 : a.subs), a.f.H, grid)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((ssm_sweep_kernel<T, DK, DV, kRev, kKeep, kLow>), grid, dim3(kSsmThreads), 0, st, a, s);
  return hipGetLastError();
}
inline hipError_t launch_chain(const SweepArgs& a, const SeqTab& s, int seqs, int sd, bool rev, hipStream_t st) {
  const long long blocks = (long long)seqs * a.f.H * (sd / 4 / 256);
  if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
  if (rev) hipLaunchKernelGGL(ssm_chain_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, st, a, s, sd / 4);
  else hipLaunchKernelGGL(ssm_chain_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, st, a, s, sd / 4);
  return hipGetLastError();
}

}  // namespace
}  // namespace kda
