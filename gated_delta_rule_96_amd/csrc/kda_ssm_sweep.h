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

// The part (or share of one) a work-group sweeps, and its slot.
struct SweepPart {
  SeqPart p;
  int h, chunk0;        // head; the launch's number of chunk p.t0 / kQ
  size_t slot;          // of this part's own sum, which becomes the next part's start
  bool start, final;    // the part the sweep starts with / ends with
};
template <bool kRev, bool kKeep>
__device__ __forceinline__ bool sweep_part(const SweepArgs& a, const SeqTab& sq, SweepPart& s) {
  ItemHead w;
  if (!item_head(sq.items * (kKeep ? 1 : a.subs), a.f.H, w)) return false;
  const int sub = kKeep ? 0 : w.item % a.subs;
  if (!kKeep) w.item /= a.subs;
  s.p = seq_part(sq, w.item);
  s.h = w.h;
  s.final = kRev ? s.p.first : s.p.last;
  s.start = kRev ? s.p.last : s.p.first;
  if (!kKeep) {
    if (s.final) return false;
    // every other part ends where the next begins: along the tokens it has
    // sq.part of them (a whole number of chunks for each share)
    const int len = (s.p.t1 - s.p.t0) / a.subs;
    s.p.t0 += sub * len;
    s.p.t1 = s.p.t0 + len;
  }
  s.slot = ((size_t)(w.item - s.p.li - (kRev ? 1 : 0)) * a.subs + sub) * a.f.H + w.h;
  s.chunk0 = (sq.n ? sq.cb[s.p.li] : s.p.li * sq.chunks) + s.p.t0 / kQ;
  return true;
}
// The state a kept sweep starts from, and where the last one goes.
template <bool kRev, bool kKeep, typename St>
__device__ __forceinline__ void sweep_begin(const SweepArgs& a, const SweepPart& s, size_t sd, St& S) {
  if (!kKeep) S.zero();
  else if (!s.start) S.load(a.f.seg + (kRev ? s.slot + (size_t)a.subs * a.f.H : s.slot - (size_t)a.subs * a.f.H) * sd);
  else if (a.from) S.load(a.from + ((size_t)s.p.n * a.f.H + s.h) * sd);
  else S.zero();
}
template <bool kKeep, typename St>
__device__ __forceinline__ void sweep_end(const SweepArgs& a, const SweepPart& s, size_t sd, const St& S, double total) {
  if (!kKeep) {
    S.store(a.f.seg + s.slot * sd);
    if (threadIdx.x == 0) a.f.sum[s.slot] = total;
  } else if (s.final && a.to) {
    S.store(a.to + ((size_t)s.p.n * a.f.H + s.h) * sd);
  }
}

// kKeep: starts from the part's true state, keeps the state entering every
// chunk (along: before it; against: behind it) and the one at the far end.
// Otherwise the own sum (from zero) and decay of each 1/subs of a part, for
// every part another one follows.  kLow: SweepState::update.  fp32 inputs.
template <int DK, int DV, bool kRev, bool kKeep>
__global__ __launch_bounds__(kSsmThreads) void ssm_sweep_f32_kernel(const SweepArgs a, const SeqTab sq) {
  typedef float T;
  typedef SweepState<DK, DV> St;
  constexpr size_t sd = (size_t)DK * DV;
  __shared__ __align__(16) T sb[kQ * RowTile<T, DK>::kPitch];
  __shared__ __align__(16) T sx[kQ * RowTile<T, DV>::kPitch];
  __shared__ __align__(16) float sw[kQ];
  const SsmArgs& f = a.f;
  SweepPart sp;
  if (!sweep_part<kRev, kKeep>(a, sq, sp)) return;
  const SeqPart& p = sp.p;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int h = sp.h, grp = h / (f.H / f.G);
  const double a2 = (double)f.A[h] * 1.4426950408889634074;
  const float bias = f.bias ? f.bias[h] : 0.f;
  const T* x = (const T*)a.cols + p.start * (size_t)a.ldcols + (size_t)h * DV;
  const T* bm = (const T*)a.rows + p.start * (size_t)a.ldrows + (size_t)grp * DK;
  const T* dt = (const T*)f.dt + p.start * (size_t)f.lddt + h;
  St S;
  sweep_begin<kRev, kKeep>(a, sp, sd, S);
  double total = 0.0;
  RowTile<T, DK> rb;
  RowTile<T, DV> rx;
  float raw = 0.f;
  auto fetch = [&](int t) {
    const int n = p.t1 - t;
    rb.load(bm + (size_t)t * (size_t)a.ldrows, a.ldrows, n, tid);
    rx.load(x + (size_t)t * (size_t)a.ldcols, a.ldcols, n, tid);
    raw = lane < n ? dt[(size_t)(t + lane) * (size_t)f.lddt] : 0.f;
  };
  const int nch = (p.t1 - p.t0 + kQ - 1) / kQ;
  auto start = [&](int k) { return p.t0 + kQ * (kRev ? nch - 1 - k : k); };
  if (nch > 0) fetch(start(0));
  for (int k = 0; k < nch; ++k) {
    const int t = start(k), n = min(p.t1 - t, kQ);
    StepSize s = step_size(raw, bias, f.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const double cum = wave_scan(s.a), last = lane63(cum);
    __syncthreads();   // the chunk before is done with LDS
    rb.store(sb, tid);
    rx.store(sx, tid);
    if (wave == 0) sw[lane] = kRev ? exp2_of(cum) : exp2_of(last - cum) * s.dt;
    if (k + 1 < nch) fetch(start(k + 1));
    if (kKeep) S.store(a.at + ((size_t)(sp.chunk0 + (t - p.t0) / kQ) * f.H + h) * sd);
    __syncthreads();
    S.template update<false, PadTile<T, DK>, PadTile<T, DV>>(exp2_of(last), sb, sx, sw);
    total += last;
  }
  sweep_end<kKeep>(a, sp, sd, S, total);
}

// The same for bf16: the rows of the next chunk go straight into the other
// half of LDS while this one's products run (one barrier a chunk), and the
// four waves take turns at forming the next chunk's weights.  64K tokens x 32
// heads of 128 x 128, own sums: 206 us (as first written 244 against 289 with
// rows through registers and two barriers); the products are 98 us of it at 2
// GHz (96 matrix instructions a wave and chunk, two waves per SIMD), their
// splits and LDS operands the rest.
template <int DK, int DV, bool kRev, bool kKeep, bool kLow>
__global__ __launch_bounds__(kSsmThreads, 2) void ssm_sweep_kernel(const SweepArgs a, const SeqTab sq) {
  typedef bf16 T;
  typedef SweepState<DK, DV> St;
  typedef SwzTile<DK> TK;
  typedef SwzTile<DV> TV;
  constexpr size_t sd = (size_t)DK * DV;
  __shared__ __align__(16) T sb[2][TK::kElems];
  __shared__ __align__(16) T sx[2][TV::kElems];
  __shared__ __align__(16) float sw[2][kQ];
  __shared__ double slast[2];
  const SsmArgs& f = a.f;
  SweepPart sp;
  if (!sweep_part<kRev, kKeep>(a, sq, sp)) return;
  const SeqPart& p = sp.p;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int h = sp.h, grp = h / (f.H / f.G);
  const double a2 = (double)f.A[h] * 1.4426950408889634074;
  const float bias = f.bias ? f.bias[h] : 0.f;
  const T* x = (const T*)a.cols + p.start * (size_t)a.ldcols + (size_t)h * DV;
  const T* bm = (const T*)a.rows + p.start * (size_t)a.ldrows + (size_t)grp * DK;
  const unsigned short* dt = (const unsigned short*)f.dt + p.start * (size_t)f.lddt + h;
  const int nch = (p.t1 - p.t0 + kQ - 1) / kQ;
  auto start = [&](int k) { return p.t0 + kQ * (kRev ? nch - 1 - k : k); };
  auto fetch = [&](int k) {
    if (k >= nch) return;
    const int t = start(k), n = p.t1 - t;
    TK::load(sb[k & 1], bm + (size_t)t * (size_t)a.ldrows, a.ldrows, n, tid);
    TV::load(sx[k & 1], x + (size_t)t * (size_t)a.ldcols, a.ldcols, n, tid);
  };
  // chunk k's step sizes are loaded and its weights formed by wave k % 4
  unsigned raw = 0;
  auto fetch_dt = [&](int k) {
    if (k < nch) raw = dt[(size_t)min(start(k) + lane, p.t1 - 1) * (size_t)f.lddt];
  };
  auto weights = [&](int k) {
    if (k >= nch || wave != (k & 3)) return;
    const int n = p.t1 - start(k);
    StepSize s = step_size(__uint_as_float(raw << 16), bias, f.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const double cum = wave_scan(s.a), last = lane63(cum);
    // rows behind the part's end repeat its last one: they weigh nothing
    sw[k & 1][lane] = lane >= n ? 0.f : kRev ? exp2_of(cum) : exp2_of(last - cum) * s.dt;
    if (lane == 0) slast[k & 1] = last;
    fetch_dt(k + 4);
  };
  auto rows_there = [&] { asm volatile("s_waitcnt vmcnt(0)" : "+v"(raw) : : "memory"); };
  St S;
  sweep_begin<kRev, kKeep>(a, sp, sd, S);
  double total = 0.0;
  fetch_dt(wave);
  fetch(0);
  weights(0);
  rows_there();
  __syncthreads();
  for (int k = 0; k < nch; ++k) {
    fetch(k + 1);
    weights(k + 1);
    const double last = slast[k & 1];
    if (kKeep) S.store(a.at + ((size_t)(sp.chunk0 + (kRev ? nch - 1 - k : k)) * f.H + h) * sd);
    S.template update<kLow, TK, TV>(exp2_of(last), sb[k & 1], sx[k & 1], sw[k & 1]);
    total += last;
    rows_there();
    __syncthreads();
  }
  sweep_end<kKeep>(a, sp, sd, S, total);
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
  const dim3 grid = item_head_grid(s.items * (kKeep ? 1 : a.subs), a.f.H);
  if constexpr (sizeof(T) == 2)
    hipLaunchKernelGGL((ssm_sweep_kernel<DK, DV, kRev, kKeep, kLow>), grid, dim3(kSsmThreads), 0, st, a, s);
  else
    hipLaunchKernelGGL((ssm_sweep_f32_kernel<DK, DV, kRev, kKeep>), grid, dim3(kSsmThreads), 0, st, a, s);
  return hipGetLastError();
}
inline hipError_t launch_chain(const SweepArgs& a, const SeqTab& s, int seqs, int sd, bool rev, hipStream_t st) {
  // (a sequence is cut only where a launch's sequences have fewer than 2^16 heads together)
  const dim3 grid((unsigned)seqs * (unsigned)a.f.H * (unsigned)(sd / 4 / 256));
  if (rev) hipLaunchKernelGGL(ssm_chain_kernel<true>, grid, dim3(256), 0, st, a, s, sd / 4);
  else hipLaunchKernelGGL(ssm_chain_kernel<false>, grid, dim3(256), 0, st, a, s, sd / 4);
  return hipGetLastError();
}

}  // namespace
}  // namespace kda
