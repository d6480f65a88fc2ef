// Gradients of the gated linear recurrence (kda_lru_dev.h has the forward's
// formulas).  With l_t = dL/dh_t and e_t = a_t l_t what a token hands to the one
// before it:
//   l_t = dy_t + e_{t+1}  (e behind the last token: dht),  dh0 = e_1
//   dx = l m s,   di = l m x s (1 - s),   s = Sigmoid(i)
//   dg = a (l h_{t-1} - l s x a / m)      (the second term with unit only)
//   dr = dg g (1 - Sigmoid(r)),  dc = -sum dg Sigmoid(r)   (dr = dg without c)
// (1 - Sigmoid in fp32: off by 3 x 2^-24 of 1, not of itself.)
// A part of a sequence (as in the forward) takes e from the right by
// e -> P e + K with K = sum_t P_t dy_t, P_t the product of its a up to t.
// Where m = 0 (a decay of exactly 1) its derivative counts as 0.
//
// Three launches where a sequence has several parts (one otherwise): every
// part's P, H, K; the states and the e that enter the parts; the gradients.  The
// last walks the parts from the end, so that what the first read last is still
// in the cache.  The inputs are read twice: 22 bytes an element pass (bf16) where
// the formulas need 14.  (One launch that carries both ways would have to hold
// every input between the state that comes from the left and the e from the right.
// With the states known, from a walk over x, r and i alone or from the forward,
// one launch could take the e from part to part as the forward takes the state, in
// 20 bytes or 14; that has not been built.)
//
// Bound by HBM in both passes, in bf16 nearly as much by the exponentials and
// roots (4 sequences of 8192 x 2048 with every gradient: sums 121 us, 4.4 TB/s;
// chain 15; gradients 167, 5.6 TB/s; dc 8; 322 in all.  fp32: 200 and 325 us,
// 5.3 and 5.8 TB/s).  The tile: runs of 8 in parts of 32 tokens 340 us, runs of 4
// 358 to 362, parts of 64 375 (timed together).  One sequence behind the other,
// so that the second pass finds its inputs in the last-level cache, 376 against
// 344: the ends of the launches cost more than it gives.
#include "kda_lru_dev.h"

namespace kda {

namespace {

constexpr int kWaves = 4, kR = 8, kPart = kWaves * kR;   // kR tokens a wave's run

// A run's rows as loaded.
template <typename T, int NC, int R> struct BwdRun {
  LruPack<T, NC, true> x[R], r[R], i[R], dy[R];
};
template <typename T, int NC, int R, bool kFull>
__device__ __forceinline__ void load_rows(const LruBwdArgs& b, const SeqPart& p, const LruLane& l, int t, BwdRun<T, NC, R>& w) {
  typedef LruPack<T, NC, true> Pk;
  const int n = p.t1 - t;
  if (n <= 0) return;
  const size_t row = p.start + (size_t)t;
  const T *px = (const T*)b.f.x + row * (size_t)b.f.ldx, *pr = (const T*)b.f.r + row * (size_t)b.f.ldr;
  const T *pi = (const T*)b.f.i + row * (size_t)b.f.ldi, *pd = (const T*)b.dy + row * (size_t)b.f.D;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int q = min(k, n - 1);
    w.x[k] = lru_load<Pk>(px + q * b.f.ldx, l.cl);
    w.r[k] = lru_load<Pk>(pr + q * b.f.ldr, l.cl);
    w.dy[k] = lru_load<Pk>(pd + (long long)q * b.f.D, l.cl);
  }
  if (kFull || b.f.i)
#pragma unroll
    for (int k = 0; k < R; ++k) w.i[k] = lru_load<Pk>(pi + min(k, n - 1) * b.f.ldi, l.cl);
  if (n < R) {   // tokens past the part's end: a = 1, u = 0, dy = 0
    const float open = b.f.c ? -__builtin_inff() : 0.f;
#pragma unroll
    for (int k = 1; k < R; ++k)
      if (k >= n) {
        w.x[k].fill(0.f);
        w.i[k].fill(0.f);
        w.dy[k].fill(0.f);
        w.r[k].fill(open);
      }
  }
}

// P, H and K of a run of n tokens from its tokens' a, u and dy, which `gate`
// gives.
template <typename T, int NC, int R, typename F>
__device__ __forceinline__ void run_sums(const BwdRun<T, NC, R>& w, int n, float (&P)[NC], float (&H)[NC], float (&K)[NC], F gate) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    P[j] = 1.f;
    H[j] = K[j] = 0.f;
  }
  if (n <= 0) return;
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float a, u;
      const float d = w.dy[k].at(j);
      gate(k, j, a, u);
      P[j] = k ? P[j] * a : a;
      H[j] = k ? fmaf(a, H[j], u) : u;
      K[j] = k ? fmaf(P[j], d, K[j]) : a * d;
    }
}

// seg [items][3][D]: P, H, K of every part.
template <typename T, int NC, bool kFull>
__global__ __launch_bounds__(64 * kWaves, 4) void lru_bwd_part_kernel(const LruBwdArgs b, const SeqTab s, unsigned slices, float* seg) {
  constexpr int R = kR;
  __shared__ float red[3][kWaves][64 * NC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, D = b.f.D;
  const unsigned item = blockIdx.x / slices;
  const LruLane l = lru_lane<NC>((int)(blockIdx.x - item * slices), D);
  const SeqPart p = seq_part(s, (int)item);
  const int t = p.t0 + wave * R;
  BwdRun<T, NC, R> w;
  load_rows<T, NC, R, kFull>(b, p, l, t, w);
  float c[NC], P[NC], H[NC], K[NC];
  lru_coef<NC>(b.f, l, c);
  const LruMode md = lru_mode<kFull>(b.f);
  run_sums<T, NC, R>(w, p.t1 - t, P, H, K, [&](int k, int j, float& a, float& u) {
    lru_gate<T>(md, c[j], w.x[k].at(j), w.r[k].at(j), md.igate ? w.i[k].at(j) : 0.f, a, u);
  });
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    red[0][wave][lane * NC + j] = P[j];
    red[1][wave][lane * NC + j] = H[j];
    red[2][wave][lane * NC + j] = K[j];
  }
  __syncthreads();
  if (wave || !l.live) return;
#pragma unroll
  for (int q = 1; q < kWaves; ++q)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float f = red[0][q][lane * NC + j];
      K[j] = fmaf(P[j], red[2][q][lane * NC + j], K[j]);
      H[j] = fmaf(f, H[j], red[1][q][lane * NC + j]);
      P[j] *= f;
    }
  float* to = seg + (size_t)item * 3 * D + l.c;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    to[j] = P[j];
    to[D + j] = H[j];
    to[2 * D + j] = K[j];
  }
}

// What enters a sequence's parts: states over H, e from the right over K.  A
// work-group takes CH channels: CH of its threads at a time take a run of the
// parts, join their runs in LDS and walk them again.  `first`: work-groups of the
// launches before.
constexpr int kChainThreads = 1024;
template <int CH>
__global__ __launch_bounds__(kChainThreads) void lru_bwd_chain_kernel(const LruBwdArgs b, const SeqTab s, float* seg, unsigned first) {
  constexpr int kRuns = kChainThreads / CH;
  __shared__ float red[3][kRuns][CH];
  const unsigned id = first + blockIdx.x;
  const int D = b.f.D, blocks = (D + CH - 1) / CH, li = id / blocks;
  const int run = CH == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : threadIdx.x / CH, lane = threadIdx.x % CH;
  const int c0 = (id - li * blocks) * CH + lane;
  const bool live = c0 < D;
  const int c = live ? c0 : 0, n = s.n0 + li;
  const int i0 = s.n ? s.cc[li] : li * s.parts, i1 = s.n ? s.cc[li + 1] : i0 + s.parts;
  const int per = (i1 - i0 + kRuns - 1) / kRuns, lo = min(i0 + run * per, i1), hi = min(lo + per, i1);
  float* at = seg + c;
  float P = 1.f, H = 0.f, K = 0.f;
#pragma unroll 4
  for (int i = lo; i < hi; ++i) {
    const float* q = at + (size_t)i * 3 * D;
    const float p = q[0];
    H = fmaf(p, H, q[D]);
    K = fmaf(P, q[2 * D], K);
    P *= p;
  }
  red[0][run][lane] = P;
  red[1][run][lane] = H;
  red[2][run][lane] = K;
  __syncthreads();
  float h = b.f.h0 ? b.f.h0[(size_t)n * D + c] : 0.f, e = b.dht ? b.dht[(size_t)n * D + c] : 0.f;
  for (int q = 0; q < run; ++q) h = fmaf(red[0][q][lane], h, red[1][q][lane]);
  for (int q = kRuns - 1; q > run; --q) e = fmaf(red[0][q][lane], e, red[2][q][lane]);
  if (!live) return;
#pragma unroll 4
  for (int i = lo; i < hi; ++i) {
    float* q = at + (size_t)i * 3 * D;
    const float p = q[0], v = q[D];
    q[D] = h;
    h = fmaf(p, h, v);
  }
#pragma unroll 4
  for (int i = hi - 1; i >= lo; --i) {
    float* q = at + (size_t)i * 3 * D;
    const float p = q[0], v = q[2 * D];
    q[2 * D] = e;
    e = fmaf(p, e, v);
  }
  if (b.dh0 && run == 0) b.dh0[(size_t)n * D + c] = e;
}

// Gradients.  seg null: every sequence is one part.  dcp [items][D]: every
// part's -sum of dg Sigmoid(r), or null (32 tokens in fp32; the parts are summed in
// 64 bits).
template <typename T, int NC, bool kFull>
__global__ __launch_bounds__(64 * kWaves, 3) void lru_bwd_out_kernel(const LruBwdArgs b, const SeqTab s, unsigned slices, const float* seg, float* dcp) {
  constexpr int R = kR;
  typedef LruPack<T, NC, true> Pk;
  __shared__ float red[3][kWaves][64 * NC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, D = b.f.D;
  const unsigned id = gridDim.x - 1 - blockIdx.x, item = id / slices;
  const LruLane l = lru_lane<NC>((int)(id - item * slices), D);
  const SeqPart p = seq_part(s, (int)item);
  const int t = p.t0 + wave * R, n = p.t1 - t;
  BwdRun<T, NC, R> w;
  load_rows<T, NC, R, kFull>(b, p, l, t, w);
  // of every token: a, u (later the state before it), Sigmoid(r), Sigmoid(i), m
  // and 1/m; the second walk has them from the first
  float a[R][NC], u[R][NC], sr[R][NC], si[R][NC], m[R][NC], im[R][NC], c[NC], P[NC], H[NC], K[NC], h[NC], e[NC], sum[NC];
  lru_coef<NC>(b.f, l, c);
  const LruMode md = lru_mode<kFull>(b.f);
  const float *from = b.f.h0 ? b.f.h0 + (size_t)p.n * D : nullptr, *back = b.dht ? b.dht + (size_t)p.n * D : nullptr;
  if (seg) {
    from = seg + ((size_t)item * 3 + 1) * D;
    back = from + D;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    h[j] = from ? from[l.cl + j] : 0.f;
    e[j] = back ? back[l.cl + j] : 0.f;
    sum[j] = 0.f;
  }
  run_sums<T, NC, R>(w, n, P, H, K, [&](int k, int j, float& av, float& uv) {
    const float r = w.r[k].at(j);
    sr[k][j] = md.gate ? sigmoid_fast(r) : 1.f;
    si[k][j] = md.igate ? sigmoid_fast(w.i[k].at(j)) : 1.f;
    const float d = one_minus_decay<T>(md.gate ? -c[j] * sr[k][j] : r, av);
    m[k][j] = im[k][j] = 1.f;
    if (md.unit) {
      const float q = d * (1.f + av);
      im[k][j] = __builtin_fabsf(q) < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q);
      m[k][j] = q * im[k][j];
    }
    uv = w.x[k].at(j) * si[k][j] * m[k][j];
    a[k][j] = av;
    u[k][j] = uv;
  });
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    red[0][wave][lane * NC + j] = P[j];
    red[1][wave][lane * NC + j] = H[j];
    red[2][wave][lane * NC + j] = K[j];
  }
  __syncthreads();
  for (int q = 0; q < wave; ++q)
#pragma unroll
    for (int j = 0; j < NC; ++j) h[j] = fmaf(red[0][q][lane * NC + j], h[j], red[1][q][lane * NC + j]);
  for (int q = kWaves - 1; q > wave; --q)
#pragma unroll
    for (int j = 0; j < NC; ++j) e[j] = fmaf(red[0][q][lane * NC + j], e[j], red[2][q][lane * NC + j]);
  if (n > 0)
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float before = h[j];
        h[j] = fmaf(a[k][j], h[j], u[k][j]);
        u[k][j] = before;
      }
#pragma unroll
  for (int k = R - 1; k >= 0; --k) {
    if (k >= n) continue;
    float dx[NC], dr[NC], di[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float x = w.x[k].at(j), s = si[k][j], lt = w.dy[k].at(j) + e[j];
      e[j] = a[k][j] * lt;
      const float gx = lt * m[k][j] * s;
      const float dg = e[j] * (md.unit ? fmaf(-a[k][j], x * s * im[k][j], u[k][j]) : u[k][j]);
      dx[j] = gx;
      di[j] = gx * x * (1.f - s);
      dr[j] = md.gate ? dg * (-c[j] * sr[k][j]) * (1.f - sr[k][j]) : dg;
      sum[j] = fmaf(dg, sr[k][j], sum[j]);
    }
    if (l.live) {
      const size_t row = (p.start + (size_t)(t + k)) * D;
      Pk o;
      o.set(dx);
      lru_store((T*)b.dx + row, l.c, o);
      o.set(dr);
      lru_store((T*)b.dr + row, l.c, o);
      if (md.igate) {
        o.set(di);
        lru_store((T*)b.di + row, l.c, o);
      }
    }
  }
  if (!seg && b.dh0 && wave == 0 && l.live)
#pragma unroll
    for (int j = 0; j < NC; ++j) b.dh0[(size_t)p.n * D + l.c + j] = e[j];
  if (!dcp) return;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NC; ++j) red[0][wave][lane * NC + j] = sum[j];
  __syncthreads();
  if (wave || !l.live) return;
#pragma unroll
  for (int q = 1; q < kWaves; ++q)
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[j] += red[0][q][lane * NC + j];
#pragma unroll
  for (int j = 0; j < NC; ++j) dcp[(size_t)item * D + l.c + j] = -sum[j];
}

// The chain's work-groups, in several launches where one cannot have them (the
// parts' launch has fewer than 2^24 of 64 or 128 channels of a part, so there are
// fewer than 2^27 here).
template <int CH>
hipError_t chain_go(const LruBwdArgs& b, const SeqTab& s, int seqs, float* seg, hipStream_t st) {
  const long long all = (long long)((b.f.D + CH - 1) / CH) * seqs;
  for (long long first = 0; first < all; first += max_groups(kChainThreads)) {
    const long long n = all - first < max_groups(kChainThreads) ? all - first : max_groups(kChainThreads);
    hipLaunchKernelGGL(lru_bwd_chain_kernel<CH>, dim3((unsigned)n), dim3(kChainThreads), 0, st, b, s, seg, (unsigned)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool pairs(const LruBwdArgs& b, size_t esz) {
  const LruArgs& a = b.f;
  if (a.D % 2 || a.ldx % 2 || a.ldr % 2 || (a.i && a.ldi % 2)) return false;
  for (const void* p : {a.x, a.r, a.i, b.dy, (const void*)b.dx, (const void*)b.dr, (const void*)b.di})
    if (reinterpret_cast<uintptr_t>(p) % (2 * esz)) return false;
  return true;
}

size_t all_items(int is_packed, int N, int B, int T) {
  return is_packed ? (size_t)T / kPart + (size_t)N : (size_t)B * (((size_t)T + kPart - 1) / kPart);
}

template <typename T, int NC, bool kFull>
hipError_t bwd_go(const LruBwdArgs& b, const int* cu, int N, int B, int T_, float* ws, hipStream_t st) {
  const int D = b.f.D;
  const unsigned slices = (unsigned)((D + 64 * NC - 1) / (64 * NC));
  if (!seq_tabs_fit(cu, N, B, T_, kPart, max_groups(64 * kWaves) / slices)) return hipErrorInvalidConfiguration;
  float* dcp = b.dc ? ws : nullptr;
  float* seg = ws + all_items(cu != nullptr, N, B, T_) * D;
  size_t rows = 0;
  const int end = cu ? N : B;
  for (int n = 0; n < end;) {
    SeqTab s;
    n = make_seq_tab(s, cu, N, n, B, T_, kPart);
    const int seqs = s.n ? s.n : B;
    const dim3 grid((unsigned)s.items * slices), th(64 * kWaves);
    const bool one = s.items == seqs;   // no sequence has a second part
    if (!one) {
      hipLaunchKernelGGL((lru_bwd_part_kernel<T, NC, kFull>), grid, th, 0, st, b, s, slices, seg);
      // By 64 channels, or by 16 and more runs where a sequence has many parts
      // (65536 x 64: 61 us in all, by 64 channels 94; 65536 x 512: 184 and 218; 256
      // parts, 4 sequences of 8192 x 2048: 346 and 342; 8, 64 of 256 x 512: 68 and 49).
      int longest = s.n ? 0 : s.parts;
      for (int i = 0; i < s.n; ++i) longest = s.cc[i + 1] - s.cc[i] > longest ? s.cc[i + 1] - s.cc[i] : longest;
      const hipError_t e = longest <= 256 ? chain_go<64>(b, s, seqs, seg, st) : chain_go<16>(b, s, seqs, seg, st);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((lru_bwd_out_kernel<T, NC, kFull>), grid, th, 0, st, b, s, slices, one ? nullptr : seg, dcp ? dcp + rows * D : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    rows += s.items;
  }
  return dcp ? launch_sum_rows(dcp, rows, (unsigned)D, 0, 0, b.dc, nullptr, nullptr, st) : hipSuccess;
}

template <typename T>
hipError_t bwd_type(const LruBwdArgs& b, const int* cu, int N, int B, int T_, float* ws, hipStream_t st) {
  if (pairs(b, sizeof(T))) return lru_full(b.f) ? bwd_go<T, 2, true>(b, cu, N, B, T_, ws, st) : bwd_go<T, 2, false>(b, cu, N, B, T_, ws, st);
  return lru_full(b.f) ? bwd_go<T, 1, true>(b, cu, N, B, T_, ws, st) : bwd_go<T, 1, false>(b, cu, N, B, T_, ws, st);
}

}  // namespace

size_t lru_bwd_workspace_bytes(int is_packed, int N, int B, int T, int D) {
  return (all_items(is_packed, N, B, T) * 4 * D * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_lru_bwd(int is_bf16, const LruBwdArgs& b, const int* cu, int N, int B, int T, void* workspace, hipStream_t st) {
  float* ws = static_cast<float*>(workspace);
  return is_bf16 ? bwd_type<bf16>(b, cu, N, B, T, ws, st) : bwd_type<float>(b, cu, N, B, T, ws, st);
}

}  // namespace kda
