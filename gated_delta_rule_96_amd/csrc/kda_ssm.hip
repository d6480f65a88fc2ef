// Selective state space scan with one decay per head (scalar A), its chunked
// form for prompts and its single-token step.
//
// Per head h, with S in R^{dk x dv} (state channels as rows), B and C of the
// head's group g = h / (H/G), dt = raw + bias or Softplus(raw + bias):
//   S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T
//   y_t = S_t^T C_t + D x_t
//
// Chunks of Q = 64 tokens, cum_i the sum of dt A inside the chunk up to i:
//   y_i = exp(cum_i) S_0^T C_i + sum_{j<=i} M_ij x_j + D x_i,
//         M_ij = (C_i . B_j) exp(cum_i - cum_j) dt_j
//   S_Q = exp(cum_Q) S_0 + sum_j exp(cum_Q - cum_j) dt_j B_j x_j^T
// Every factor is exp of a difference that is <= 0 for A <= 0: nothing is
// rescaled, any decay is in range (sums and differences of exponents in 48 bits
// or more, see step_size and PipeLds).  Later tokens never reach an earlier one's
// y, also not as 0 x inf or 0 x NaN.
//
// A work-group walks the chunks of one part of one sequence for one head with
// the whole state in registers: of four waves, wave w owns dv/4 value columns
// (as MFMA accumulators, so that two stacked tiles are directly the operand
// of the next chunk's S^T C product).  All products are formed transposed
// (value columns as rows of the output tile): a lane then holds neighbouring
// value columns of one token and stores them together.  M goes through LDS
// once (wave w forms rows 16w.. of it), x and B are read with transposed LDS
// reads where the token is the reduction index.  bf16 has four waves more,
// which load and form M one chunk ahead (ssm_pipe_kernel).
//
// Parts: a sequence is cut so that one work-group per CU runs; a first pass
// (kda_ssm_sweep.h) sums each part's own states (no y), a small kernel chains
// them, the second pass starts every part from its state.  That reads x and B
// twice; it keeps the chain of dependent chunks short without waits between
// work-groups.
//
// Measured (65536 tokens, 32 heads of 128 x 128, bf16): 620 us, 1.8 TB/s of
// the inputs and outputs and 220 TFLOP/s of the products (traced kernel by
// kernel: first pass 206, chaining 11, scan 410).
// Neither rate binds: a chunk's 144 matrix instructions per state wave are 147
// us of the scan's time at 2 GHz; the rest are their LDS operands, the exact
// splits, the state's scaling and y's stores of the same four waves, one
// work-group per CU, whose tiles and state fill LDS and registers.
//
// Rounding (bf16): C, B and x are exact operands; M and the state as the
// operand of S^T C are rounded to bf16 (2^-8 of each product's terms, like
// y's own rounding).  The state itself is fp32 and its update splits
// dt x exp(...) into three bf16 parts (24 bits), so that it is an fp32 result:
// two parts (16 bits) leave a relative error of 2.7e-6, far above fp32's.
// fp32 inputs: fp32 MFMA throughout, nothing rounded.
#include "kda_ssm_sweep.h"

namespace kda {

namespace {

// One scan work-group per CU (64K tokens x 32 heads: 610 us, 16K of fp32: 692;
// 128 in all 911 and 1210, 512 633 and 709).
constexpr int kScanWgs = 256;
// A part's own sum is formed in two shares: two sweep work-groups per CU (the
// same tokens: 610 and 692 us; one share 641 and 716, four 619 and 704).
constexpr int kSubs = 2;

template <int DK, int DV>
struct ChunkLds {
  static constexpr int PK = RowTile<float, DK>::kPitch, PV = RowTile<float, DV>::kPitch;
  float c[kQ * PK];
  float b[kQ * PK];
  float x[kQ * PV];
  Slab<float> m[8 * 64];      // M rows of tile it, slab js, at (2 it + js) 64 + lane
  double cum[kQ];
  float ecum[kQ], wdt[kQ], dt[kQ];
};

// The scan of a part, fp32: y and, for a sequence's last part, its final state.
template <int DK, int DV>
__global__ __launch_bounds__(kSsmThreads) void ssm_chunk_kernel(const SsmArgs a, const SeqTab sq) {
  typedef float T;
  typedef ChunkLds<DK, DV> Lds;
  typedef State<DK, DV> St;
  constexpr int NT = St::NT, PK = Lds::PK, PV = Lds::PV;
  __shared__ __align__(16) char smem[sizeof(Lds)];
  Lds& sm = *reinterpret_cast<Lds*>(smem);
  ItemHead w;
  if (!item_head(sq.items, a.H, w)) return;
  const SeqPart p = seq_part(sq, w.item);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int h = w.h, grp = h / (a.H / a.G);
  const double a2 = (double)a.A[h] * 1.4426950408889634074;
  const float bias = a.bias ? a.bias[h] : 0.f, dskip = a.D ? a.D[h] : 0.f;
  const T* x = (const T*)a.x + p.start * (size_t)a.ldx + (size_t)h * DV;
  const T* bm = (const T*)a.B + p.start * (size_t)a.ldb + (size_t)grp * DK;
  const T* cm = (const T*)a.C + p.start * (size_t)a.ldc + (size_t)grp * DK;
  const T* dt = (const T*)a.dt + p.start * (size_t)a.lddt + h;
  T* y = (T*)a.y + (p.start * (size_t)a.H + h) * DV;
  const size_t yld = (size_t)a.H * DV;

  const RowLanes rk = row_lanes<T>(PK);
  St S;
  const size_t sd = (size_t)DK * DV;
  const size_t slot = (size_t)(w.item - p.li) * kSubs * a.H + h;   // of the next part's start
  if (!p.first) S.load(a.seg + (slot - (size_t)kSubs * a.H) * sd);
  else if (a.start && !p.last) S.load(a.start + slot * sd);
  else if (a.h0) S.load(a.h0 + ((size_t)p.n * a.H + h) * sd);
  else S.zero();
  RowTile<T, DK> rc, rb;
  RowTile<T, DV> rx;
  float raw = 0.f;
  auto fetch = [&](int t) {
    const int n = p.t1 - t;
    rc.load(cm + (size_t)t * (size_t)a.ldc, a.ldc, n, tid);
    rb.load(bm + (size_t)t * (size_t)a.ldb, a.ldb, n, tid);
    rx.load(x + (size_t)t * (size_t)a.ldx, a.ldx, n, tid);
    raw = lane < n ? dt[(size_t)(t + lane) * (size_t)a.lddt] : 0.f;
  };
  if (p.t0 < p.t1) fetch(p.t0);
  for (int t = p.t0; t < p.t1; t += kQ) {
    const int n = min(p.t1 - t, kQ);
    // step sizes and decay sums: every wave forms them, one array each is kept
    StepSize s = step_size(raw, bias, a.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const double cum = wave_scan(s.a), last = lane63(cum);
    __syncthreads();   // the chunk before is done with LDS
    rc.store(sm.c, tid);
    rb.store(sm.b, tid);
    rx.store(sm.x, tid);
    if (wave == 0) {
      sm.cum[lane] = cum;
    } else if (wave == 1) {
      sm.ecum[lane] = exp2_of(cum);
    } else if (wave == 2) {
      sm.wdt[lane] = exp2_of(last - cum) * s.dt;
    } else {
      sm.dt[lane] = s.dt;
    }
    if (t + kQ < p.t1) fetch(t + kQ);
    __syncthreads();

    // rows 16 wave .. of M, transposed tiles (rows j, columns i)
    const int it = wave, i = 16 * it + l16;
    Slab<T> cs[DK / 32];
#pragma unroll
    for (int k = 0; k < DK / 32; ++k) cs[k] = slab_any(sm.c, PK, 16 * it, 32 * k);
    const double ci = sm.cum[i];
#pragma unroll
    for (int js = 0; js < 2; ++js) {
      if (2 * js > it) continue;
      f32x4 v[2] = {zero4(), zero4()};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int jt = 2 * js + q;
        if (jt > it) continue;
        f32x4 acc = zero4();
#pragma unroll
        for (int k = 0; k < DK / 32; ++k) acc = mma(slab_any(sm.b, PK, 16 * jt, 32 * k), cs[k], acc);
        const int j = 16 * jt + 4 * g;
        const f32x4 dj = load4(sm.dt + j);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[q][r] = j + r <= i ? acc[r] * exp2_of(ci - sm.cum[j + r]) * dj[r] : 0.f;
      }
      sm.m[(2 * it + js) * 64 + lane] = make_slab<T>(v[0], v[1]);
    }
    __syncthreads();

    Slab<T> xs[2][NT];
    St::template slabs<PadTile<T, DV>>(sm.x, xs);
    // a product with zeros is NaN exactly where x is not finite: the masked
    // entries of M would then spread later tokens' values to earlier ones
    f32x4 probe = zero4();
#pragma unroll
    for (int js = 0; js < 2; ++js)
#pragma unroll
      for (int q = 0; q < NT; ++q) probe = mma(Slab<T>{}, xs[js][q], probe);
    const bool finite = !__any(probe[0] != probe[0]);
    f32x4 acc[4][NT];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[it][q] = zero4();
#pragma unroll
    for (int k = 0; k < DK / 32; ++k) {
      Slab<T> ss[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) ss[q] = make_slab<T>(S.s[2 * k][q], S.s[2 * k + 1][q]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const Slab<T> cs = slab_row(sm.c, rk, 16 * it * PK + 32 * k);
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[it][q] = mma(ss[q], cs, acc[it][q]);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = 16 * it + l16, c = wave * St::CPW + 4 * NT * g;
      const float e = sm.ecum[i];
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[it][q] *= e;
      if (finite) {
#pragma unroll
        for (int js = 0; js <= it / 2; ++js) {
          const Slab<T> m = sm.m[(2 * it + js) * 64 + lane];
#pragma unroll
          for (int q = 0; q < NT; ++q) acc[it][q] = mma(xs[js][q], m, acc[it][q]);
        }
      } else {   // token by token, later ones left out
#pragma unroll 1
        for (int j = 0; j <= i; ++j) {
          const T* mp = reinterpret_cast<const T*>(sm.m + (2 * it + (j >> 5)) * 64 + ((j >> 2) & 3) * 16 + l16);
          const float m = mp[4 * ((j >> 4) & 1) + (j & 3)];
#pragma unroll
          for (int q = 0; q < NT; ++q) acc[it][q] += m * load4(lds_at(sm.x, PV, j, c + 4 * q));
        }
      }
      float o[4 * NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        const f32x4 xi = four_of_row(sm.x, PV, 16 * it, c + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[4 * q + r] = a.D ? fmaf(dskip, xi[r], acc[it][q][r]) : acc[it][q][r];
      }
      if (i < n) Rows<T, 4 * NT>::store(y + (size_t)(t + i) * yld + c, o);
    }

    Split<T> xw[2][NT];
    St::weigh(xs, sm.wdt, xw);
    S.template update<PadTile<T, DK>>(exp2_of(last), sm.b, xw);
  }
  if (p.last && a.ht) S.store(a.ht + ((size_t)p.n * a.H + h) * sd);
}

// The same scan for bf16 with the work of a chunk split over two sets of four
// waves that run one chunk apart: the front waves fetch chunk k + 2 straight
// into LDS, form chunk k + 1's M and chunk k + 2's step sizes, while the back
// waves take chunk k's products with S, its y and the state's update.  One
// barrier a chunk; the matrix instructions of one set cover the loads and
// exponents of the other (64K tokens x 32 heads: 491 us for this kernel as first
// written against 628 with four waves that do one thing after the other; 410
// now).
constexpr int kPipeThreads = 2 * kSsmThreads;

template <int DK, int DV>
struct PipeLds {
  bf16 c[3][kQ * DK];
  bf16 b[3][kQ * DK];
  bf16 x[3][kQ * DV];
  Slab<bf16> m[2][6 * 64];   // M rows of tile it, slab js, at (it + max(it - 2, 0) + js) 64 + lane
  struct Sizes {
    // decay sums as two floats each, 48 bits together: small steps behind a
    // large one differ far below its size.  64K tokens x 32 heads, packed
    // prompts: 643 and 79 us; one float each 641 and 78, but M off by a tenth
    // behind a step of 1e5; as doubles 667 and 98.
    float cum[kQ], low[kQ];
    float ecum[kQ], wdt[kQ], dt[kQ];
  } z[3];
  float el[4];               // exp(cum_Q) of chunk k at k % 3
};
__device__ __forceinline__ int m_slab(int it, int js) { return it + (it > 2 ? it - 2 : 0) + js; }

template <int DK, int DV>
__global__ __launch_bounds__(kPipeThreads, 2) void ssm_pipe_kernel(const SsmArgs a, const SeqTab sq) {
  typedef bf16 T;
  typedef PipeLds<DK, DV> Lds;
  typedef State<DK, DV> St;
  typedef SwzTile<DK> TK;
  typedef SwzTile<DV> TV;
  constexpr int NT = St::NT;
  __shared__ __align__(16) char smem[sizeof(Lds)];
  Lds& sm = *reinterpret_cast<Lds*>(smem);
  ItemHead w;
  if (!item_head(sq.items, a.H, w)) return;
  const SeqPart p = seq_part(sq, w.item);
  const bool front = threadIdx.x >= kSsmThreads;   // waves 4..7
  const int tid = threadIdx.x & (kSsmThreads - 1), wave = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int h = w.h, grp = h / (a.H / a.G);
  const int nch = (p.t1 - p.t0 + kQ - 1) / kQ;
  constexpr size_t sd = (size_t)DK * DV;

  if (front) {
    const double a2 = (double)a.A[h] * 1.4426950408889634074;
    const float bias = a.bias ? a.bias[h] : 0.f;
    const size_t t00 = p.start + p.t0;
    const T* x = (const T*)a.x + t00 * (size_t)a.ldx + (size_t)h * DV;
    const T* bm = (const T*)a.B + t00 * (size_t)a.ldb + (size_t)grp * DK;
    const T* cm = (const T*)a.C + t00 * (size_t)a.ldc + (size_t)grp * DK;
    const T* dt = (const T*)a.dt + t00 * (size_t)a.lddt + h;
    const int len = p.t1 - p.t0;
    // step sizes are loaded one chunk further ahead than the rows
    // (and kept as loaded: converting them would wait for them)
    unsigned raw = 0;
    auto fetch_dt = [&](int k) {
      if (len > 0) raw = reinterpret_cast<const unsigned short*>(dt)[(size_t)min(kQ * k + lane, len - 1) * (size_t)a.lddt];
    };
    auto fetch = [&](int k) {
      if (k >= nch) return;
      const int t = kQ * k, n = len - t, q = k % 3;
      TK::load(sm.c[q], cm + (size_t)t * (size_t)a.ldc, a.ldc, n, tid);
      TK::load(sm.b[q], bm + (size_t)t * (size_t)a.ldb, a.ldb, n, tid);
      TV::load(sm.x[q], x + (size_t)t * (size_t)a.ldx, a.ldx, n, tid);
    };
    // step sizes and decay sums: every wave forms them, one array each is kept
    auto sizes = [&](int k) {
      StepSize s = step_size(__uint_as_float(raw << 16), bias, a.softplus, a2);
      if (lane >= len - kQ * k) s = StepSize{0.f, 0.0};
      const double cum = wave_scan(s.a), last = lane63(cum);
      typename Lds::Sizes& z = sm.z[k % 3];
      if (wave == 0) {
        z.cum[lane] = (float)cum;
        z.low[lane] = (float)(cum - (double)(float)cum);
      } else if (wave == 1) {
        z.ecum[lane] = exp2_of(cum);
        if (lane == 0) sm.el[k % 3] = exp2_of(last);
      } else if (wave == 2) {
        z.wdt[lane] = exp2_of(last - cum) * s.dt;
      } else {
        z.dt[lane] = s.dt;
      }
    };
    // rows 16 wave .. of M, transposed tiles (rows j, columns i)
    auto scores = [&](int k) {
      if (k >= nch) return;
      const T *tc = sm.c[k % 3], *tb = sm.b[k % 3];
      const typename Lds::Sizes& z = sm.z[k % 3];
      const int it = wave, i = 16 * it + l16;
      Slab<T> cs[DK / 32];
#pragma unroll
      for (int q = 0; q < DK / 32; ++q) cs[q] = TK::any(tc, 16 * it, q);
      const float ci = z.cum[i], li = z.low[i];
#pragma unroll
      for (int js = 0; js < 2; ++js) {
        if (2 * js > it) continue;
        f32x4 v[2] = {zero4(), zero4()};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int jt = 2 * js + q;
          if (jt > it) continue;
          f32x4 acc = zero4();
#pragma unroll
          for (int y = 0; y < DK / 32; ++y) acc = mma(TK::any(tb, 16 * jt, y), cs[y], acc);
          const int j = 16 * jt + 4 * g;
          const f32x4 dj = load4(z.dt + j), cj = load4(z.cum + j), lj = load4(z.low + j);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[q][r] = j + r <= i ? acc[r] * exp2_fast((ci - cj[r]) + (li - lj[r])) * dj[r] : 0.f;
        }
        sm.m[k & 1][m_slab(it, js) * 64 + lane] = make_slab<T>(v[0], v[1]);
      }
    };
    // all of the wave's loads (the compiler counts those straight into LDS and
    // waits for the step sizes where they are used: here, once)
    auto rows_there = [&] { asm volatile("s_waitcnt vmcnt(0)" : "+v"(raw) : : "memory"); };
    fetch_dt(0);
    fetch(0);
    sizes(0);
    fetch_dt(1);
    fetch(1);
    sizes(1);
    fetch_dt(2);
    rows_there();
    __syncthreads();
    scores(0);
    __syncthreads();
    for (int k = 0; k < nch; ++k) {
      fetch(k + 2);
      sizes(k + 2);
      fetch_dt(k + 3);
      scores(k + 1);
      rows_there();
      __syncthreads();
    }
    return;
  }

  St S;
  const size_t slot = (size_t)(w.item - p.li) * kSubs * a.H + h;   // of the next part's start
  if (!p.first) S.load(a.seg + (slot - (size_t)kSubs * a.H) * sd);
  else if (a.start && !p.last) S.load(a.start + slot * sd);
  else if (a.h0) S.load(a.h0 + ((size_t)p.n * a.H + h) * sd);
  else S.zero();
  const float dskip = a.D ? a.D[h] : 0.f;
  const size_t yld = (size_t)a.H * DV;
  T* y = (T*)a.y + ((p.start + p.t0) * (size_t)a.H + h) * DV;
  const typename TK::RowBase rowb = TK::row_base();
  __syncthreads();
  __syncthreads();
  for (int k = 0; k < nch; ++k) {
    const int buf = k % 3;
    const T *tc = sm.c[buf], *tb = sm.b[buf], *tx = sm.x[buf];
    const typename Lds::Sizes& z = sm.z[buf];
    const Slab<T>* tm = sm.m[k & 1];
    const int n = min(p.t1 - p.t0 - kQ * k, kQ);
    Slab<T> xs[2][NT];
    St::template slabs<TV>(tx, xs);
    Split<T> xw[2][NT];
    St::weigh(xs, z.wdt, xw);
    // S^T C
    f32x4 acc[4][NT];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[it][q] = zero4();
#pragma unroll
    for (int y4 = 0; y4 < DK / 32; ++y4) {
      Slab<T> ss[NT];
#pragma unroll
      for (int q = 0; q < NT; ++q) ss[q] = make_slab<T>(S.s[2 * y4][q], S.s[2 * y4 + 1][q]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const Slab<T> cs = TK::row(tc, rowb, it, y4);
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[it][q] = mma(ss[q], cs, acc[it][q]);
      }
    }
    // a product with zeros is NaN exactly where x is not finite: the masked
    // entries of M would then spread later tokens' values to earlier ones
    f32x4 probe = zero4();
#pragma unroll
    for (int js = 0; js < 2; ++js)
#pragma unroll
      for (int q = 0; q < NT; ++q) probe = mma(Slab<T>{}, xs[js][q], probe);
    const bool finite = !__any(probe[0] != probe[0]);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const float e = z.ecum[16 * it + l16];
#pragma unroll
      for (int q = 0; q < NT; ++q) acc[it][q] *= e;
    }
    const int col = wave * St::CPW + 4 * NT * g;
    if (finite) {
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int js = 0; js <= it / 2; ++js) {
          const Slab<T> m = tm[m_slab(it, js) * 64 + lane];
#pragma unroll
          for (int q = 0; q < NT; ++q) acc[it][q] = mma(xs[js][q], m, acc[it][q]);
        }
    } else {   // token by token, later ones left out
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll 1
        for (int j = 0; j <= 16 * it + l16; ++j) {
          const T* mp = reinterpret_cast<const T*>(tm + m_slab(it, j >> 5) * 64 + ((j >> 2) & 3) * 16 + l16);
          const float m = to_f32(mp[4 * ((j >> 4) & 1) + (j & 3)]);
#pragma unroll
          for (int q = 0; q < NT; ++q) acc[it][q] += m * widen4(load4(tx + TV::at(j, col + 4 * q)));
        }
    }
    S.template update<TK>(sm.el[buf], tb, xw);
    if (a.D) {
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[it][q] += dskip * TV::four(tx, 16 * it, col + 4 * q);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = 16 * it + l16;
      float o[4 * NT];
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[4 * q + r] = acc[it][q][r];
      if (i < n) Rows<T, 4 * NT>::store(y + (size_t)(kQ * k + i) * yld + col, o);
    }
    __syncthreads();
  }
  if (p.last && a.ht) S.store(a.ht + ((size_t)p.n * a.H + h) * sd);
}

template <typename T, int DK, int DV>
hipError_t fwd_go(const SsmArgs& a, const SeqTab& s, int seqs, bool split, hipStream_t st) {
  const dim3 grid = item_head_grid(s.items, a.H);
  if (split) {
    SweepArgs w{};
    w.f = a;
    w.cols = a.x;
    w.ldcols = a.ldx;
    w.rows = a.B;
    w.ldrows = a.ldb;
    w.from = a.h0;
    w.subs = kSubs;
    hipError_t e = launch_sweep<T, DK, DV, false, false, false>(w, s, st);
    if (e == hipSuccess) e = launch_chain(w, s, seqs, DK * DV, false, st);
    if (e != hipSuccess) return e;
  }
  if constexpr (sizeof(T) == 2)
    hipLaunchKernelGGL((ssm_pipe_kernel<DK, DV>), grid, dim3(kPipeThreads), 0, st, a, s);
  else
    hipLaunchKernelGGL((ssm_chunk_kernel<DK, DV>), grid, dim3(kSsmThreads), 0, st, a, s);
  return hipGetLastError();
}

}  // namespace

int ssm_part(long long tokens, int H, int wgs) {
  // a part is at least four chunks, so that the extra pass and the chaining
  // stay small beside it (1000 tokens x 32 heads: 42 us; at least two 47, eight
  // 48; 4 heads would like two: 30 against 27, fp32 85 against 53), and a whole
  // number of chunks for each of its shares
  const long long want = (tokens * H + wgs - 1) / wgs, unit = (long long)kQ * kSubs;
  const long long part = (want + unit - 1) / unit * unit;
  return (int)(part < 256 ? 256 : part > (1 << 30) ? (1 << 30) : part);
}

// Cutting a sequence adds a pass that costs about half of the one it shortens,
// and two launches: a longest sequence of up to 1.5 parts + 256 tokens stays
// whole, and with it every other one; of up to 2 parts + 256 where the parts
// would be more than the work-groups that run at once.  Whole against cut, us
// (bf16, 32 heads, lengths behind the name of the work-groups' share of the
// tokens): 256: 640 33 against 35, 1000 47 against 42; 1024: 1500 + 7 x 928 77
// against 130, 2000 + 7 x 864 94 against 128; 2048: 3600 + 13 x 950 198
// against 212.
int ssm_part_of(int H, int wgs, const int* cu, int N, int B, int T) {
  const int part = ssm_part((long long)B * T, H, wgs);
  long long longest = T, parts = 0;
  if (cu) {
    longest = 0;
    for (int n = 0; n < N; ++n) {
      const long long len = cu[n + 1] - cu[n];
      longest = longest > len ? longest : len;
      parts += (len + part - 1) / part;
    }
  } else {
    parts = (long long)B * ((T + part - 1) / part);
  }
  const long long whole = (long long)part + (parts * H > wgs ? part : part / 2) + 256, unit = (long long)kQ * kSubs;
  return longest > part && longest <= whole ? (int)((longest + unit - 1) / unit * unit) : part;
}

size_t ssm_seg_bytes(long long tokens, int H, int dk, int dv) {
  const size_t slots = kSubs * ssm_slots(tokens, H, kScanWgs);
  return ((slots * (2 * (size_t)dk * dv * sizeof(float) + sizeof(double))) + 255) & ~(size_t)255;
}

hipError_t launch_ssm_fwd(int is_bf16, const SsmArgs& a0, int dk, int dv, const int* cu, int N, int B, int T, void* workspace,
                          hipStream_t st) {
  const long long tokens = (long long)B * T;
  const int part = ssm_part_of(a0.H, kScanWgs, cu, N, B, T), end = cu ? N : B;
  if (!seq_tabs_fit(cu, N, B, T, part, most_items(a0.H))) return hipErrorInvalidConfiguration;
  SsmArgs a = a0;
  a.seg = static_cast<float*>(workspace);
  const size_t states = kSubs * ssm_slots(tokens, a.H, kScanWgs) * (size_t)dk * dv;
  a.start = a.ht && a.ht == a.h0 ? a.seg + states : nullptr;
  a.sum = reinterpret_cast<double*>(a.seg + 2 * states);
  for (int n = 0; n < end;) {
    SeqTab s;
    const int n0 = n;
    n = make_seq_tab(s, cu, N, n, B, T, part);
    const bool split = s.items > n - n0;   // some sequence has more than one part
    hipError_t e;
#define KDA_SSM_GO(T_, K_, V_) e = fwd_go<T_, K_, V_>(a, s, n - n0, split, st)
    if (is_bf16) {
      if (dk == 128 && dv == 128) KDA_SSM_GO(bf16, 128, 128);
      else if (dk == 128) KDA_SSM_GO(bf16, 128, 64);
      else if (dv == 128) KDA_SSM_GO(bf16, 64, 128);
      else KDA_SSM_GO(bf16, 64, 64);
    } else {
      if (dk == 128 && dv == 128) KDA_SSM_GO(float, 128, 128);
      else if (dk == 128) KDA_SSM_GO(float, 128, 64);
      else if (dv == 128) KDA_SSM_GO(float, 64, 128);
      else KDA_SSM_GO(float, 64, 64);
    }
#undef KDA_SSM_GO
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Single token.  Bound by the state, read once and written once: a thread
// keeps four value columns of DK / RG rows in registers, all rows' loads
// issued first; the sums over the state channels are joined through LDS.  256
// sequences x 32 heads of 128 x 128: 193 us (5.6 TB/s).
namespace {

constexpr int kStepThreads = 512;

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kStepThreads) void ssm_step_kernel(const SsmArgs a) {
  constexpr int CG = DV / 4, RG = kStepThreads / CG, RPT = DK / RG;
  static_assert(RPT >= 1 && DK % RG == 0, "shape");
  __shared__ float sb[DK], sc[DK], sx[DV];
  __shared__ f32x4 red[RG][CG];
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H, grp = h / (a.H / a.G);
  const size_t at = (size_t)blockIdx.x * (DK * DV);
  const f32x4* src = reinterpret_cast<const f32x4*>(a.h0 + at) + cg;
  f32x4* dst = reinterpret_cast<f32x4*>(a.ht + at) + cg;
  f32x4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = __builtin_nontemporal_load(src + (size_t)(rg + RG * i) * CG);
  const float bias = a.bias ? a.bias[h] : 0.f;
  const StepSize st = step_size(to_f32(((const T*)a.dt)[(size_t)b * (size_t)a.lddt + h]), bias, a.softplus,
                                (double)a.A[h] * 1.4426950408889634074);
  const float dec = exp2_of(st.a);
  if (tid < DK) {
    sb[tid] = to_f32(((const T*)a.B)[(size_t)b * (size_t)a.ldb + (size_t)grp * DK + tid]) * st.dt;
    sc[tid] = to_f32(((const T*)a.C)[(size_t)b * (size_t)a.ldc + (size_t)grp * DK + tid]);
  }
  if (tid < DV) sx[tid] = to_f32(((const T*)a.x)[(size_t)b * (size_t)a.ldx + (size_t)h * DV + tid]);
  __syncthreads();
  const f32x4 x4 = load4(sx + 4 * cg);
  f32x4 y = zero4();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
    s[i] = s[i] * dec + sb[r] * x4;
    y += sc[r] * s[i];
    __builtin_nontemporal_store(s[i], dst + (size_t)r * CG);
  }
  red[rg][cg] = y;
  __syncthreads();
  if (tid < DV) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) v += red[r][tid >> 2][tid & 3];
    if (a.D) v = fmaf(a.D[h], sx[tid], v);
    ((T*)a.y)[(size_t)blockIdx.x * DV + tid] = from_f32<T>(v);
  }
}

template <typename T>
hipError_t step_go(const SsmArgs& a, int dk, int dv, int B, hipStream_t st) {
  const dim3 grid((unsigned)B * (unsigned)a.H), th(kStepThreads);
  if (dk == 128 && dv == 128) hipLaunchKernelGGL((ssm_step_kernel<T, 128, 128>), grid, th, 0, st, a);
  else if (dk == 128) hipLaunchKernelGGL((ssm_step_kernel<T, 128, 64>), grid, th, 0, st, a);
  else if (dv == 128) hipLaunchKernelGGL((ssm_step_kernel<T, 64, 128>), grid, th, 0, st, a);
  else hipLaunchKernelGGL((ssm_step_kernel<T, 64, 64>), grid, th, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_step(int is_bf16, const SsmArgs& a, int dk, int dv, int B, hipStream_t st) {
  if ((long long)B * a.H > max_groups(kStepThreads)) return hipErrorInvalidConfiguration;
  return is_bf16 ? step_go<bf16>(a, dk, dv, B, st) : step_go<float>(a, dk, dv, B, st);
}

}  // namespace kda
