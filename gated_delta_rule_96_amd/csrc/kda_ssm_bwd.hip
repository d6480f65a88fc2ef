// Gradients of the state space scan.
//
// Per head, in a chunk with entering state S, gradient dS of the state behind
// it, cum_i / cum_Q the decay sums, E_ij = exp(cum_i - cum_j) for j <= i,
// P = C B^T, Qm = dy x^T, w_j = exp(cum_Q - cum_j):
//   dC_i = exp(cum_i) S dy_i + sum_j E_ij dt_j Qm_ij B_j
//   dB_j = sum_i E_ij dt_j Qm_ij C_i + w_j dt_j dS x_j
//   dx_j = dt_j (sum_i E_ij P_ij dy_i + w_j dS^T B_j) + D dy_j
// With R_ij = E_ij P_ij Qm_ij, u_i = exp(cum_i) C_i . (S dy_i) and V_j = w_j
// B_j . (dS x_j), the gradient of the decay exponent a_t = dt_t A is what
// crosses token t:
//   da_t = sum_{i>=t>j} R_ij dt_j + sum_{i>=t} u_i + sum_{j<t} V_j dt_j
//          + exp(cum_Q) <dS, S>
//   ddt_t = A da_t + sum_i R_it + V_t,   dA = sum dt_t da_t,
//   dD = sum_t Qm_tt
// and a softplus multiplies ddt by Sigmoid(raw + bias).  dB and dC sum over
// the heads of a group.
//
// Four steps, as many kernels (kda_ssm_sweep.h): the states entering every
// chunk, along the tokens; the state gradients behind every chunk, against
// them; one work-group per chunk and group (or share of its heads) that walks
// the heads with P and the sums of dB and dC in registers; sums of dA, dD,
// d(dt_bias) over the chunks.  Everything is written once: no atomics, the
// same result every time.
//
// A state and its gradient per chunk and head, written and read once (2 dk dv 4
// bytes each way), are the bulk of the traffic beside the inputs.
// Measured (4 x 8192 tokens, 16 heads of 128 x 128, one group, bf16): 870 us:
// this kernel 474, sweeps that keep states 125 + 129 (0.54 GB written each, 4.2
// TB/s), own sums of the parts 57 + 61, chaining 23, last sums 5.  This kernel
// reads 1.1 GB of states (2.3 TB/s); it is bound by waits: for the states,
// which the registers only allow to be fetched two slabs of 32 columns ahead,
// and at the four barriers of a head.
//
// Rounding (bf16): the elementwise weights of the products that end in dx, dB
// and dC (bf16 outputs) are rounded to bf16 once, dS^T B's operand dS too; S
// dy and dS x feed fp32 sums (dA, and ddt through differences of large sums)
// and take S and dS in three bf16 parts (24 bits).
#include "kda_ssm_sweep.h"

namespace kda {

namespace {

// Two sweep work-groups per CU (32K tokens x 16 heads: 885 us in all; one 954,
// four 929).
constexpr int kSweepWgs = 512;
// Eight waves a chunk: with four, the sums over the heads and the products of
// one head do not fit the registers (32K tokens x 16 heads, as first written:
// 1101 us in all, with eight 1018).
constexpr int kBwdWaves = 8, kBwdThreads = 64 * kBwdWaves;

struct ChunkBwd {
  SsmBwdArgs b;
  const float *S, *dS;     // [chunks][H][dk][dv]
  float* part;             // [chunks][3][H]: dA, dD, d(dt_bias) of the chunk
  float *dBp, *dCp;        // shares > 1: [shares][tokens][G][dk]
  size_t tokens;
  int shares;              // work-groups the heads of a group are split over
};

template <typename T, int DK, int DV>
struct BwdLds {
  static constexpr int PK = RowTile<T, DK>::kPitch, PV = RowTile<T, DV>::kPitch, PM = kQ + LdsRow<T>::pad;
  T c[kQ * PK];
  T b[kQ * PK];
  union {
    T x[kQ * PV];
    struct {   // when x has been used up: sums of the waves
      float u[DK / 16][kQ], v[DK / 16][kQ], diag[kQ], qd[kQ], g[kBwdWaves];
    } s;
  };
  double col[4][kQ], row[2][kQ];   // R's sums over 16 rows i, and over two column tiles j
  T dy[kQ * PV];
  T m[kQ * PM];              // E dt Qm, then E P: [i][j]
  // dS rounded to T, [state channel][value column] (fp32: read from memory
  // again, as there is no room)
  static constexpr bool kKeepDS = sizeof(T) == 2;
  T ds[kKeepDS ? DK * PV : 1];
  double cum[kQ];
  float ecum[kQ], w[kQ], dt[kQ], slope[kQ];   // slope: of the softplus (or 1)
};

// Sum over the 16 lanes of a row of lanes, by lane permutations.
__device__ __forceinline__ double sum16(double x) {
  x += dpp_zero<0xB1>(x);    // quad_perm [1,0,3,2]
  x += dpp_zero<0x4E>(x);    // quad_perm [2,3,0,1]
  x += dpp_zero<0x141>(x);   // row_half_mirror
  x += dpp_zero<0x140>(x);   // row_mirror
  return x;
}
// Sum over the four lane groups that hold one column of a tile.
template <typename F>
__device__ __forceinline__ F sum_groups(F x) {
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kBwdThreads, 2) void ssm_bwd_kernel(const ChunkBwd a, const SeqTab sq) {
  typedef BwdLds<T, DK, DV> Lds;
  constexpr int PK = Lds::PK, PV = Lds::PV, PM = Lds::PM;
  // A wave's part of an output [tokens x D]: 16 columns of NK / NV token tiles.
  constexpr int KT = DK / 16, VT = DV / 16, NK = 4 * KT / kBwdWaves, NV = 4 * VT / kBwdWaves;
  __shared__ __align__(16) char smem[sizeof(Lds)];
  Lds& sm = *reinterpret_cast<Lds*>(smem);
  const SsmBwdArgs& b = a.b;
  const SsmArgs& f = b.f;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int HG = f.H / f.G;
  const int item = (int)(blockIdx.x / (unsigned)(f.G * a.shares)), rest = (int)(blockIdx.x - (unsigned)item * (unsigned)(f.G * a.shares));
  const int share = rest / f.G, grp = rest - share * f.G;
  const int per = (HG + a.shares - 1) / a.shares;
  const int h0 = grp * HG + min(share * per, HG), h1 = grp * HG + min((share + 1) * per, HG);
  const SeqPart p = seq_part(sq, item);   // a part is a chunk
  const int n = p.t1 - p.t0;
  if (n <= 0) {   // an empty sequence's item: it adds nothing
    if (tid < 3)
      for (int h = h0; h < h1; ++h) a.part[((size_t)item * 3 + tid) * f.H + h] = 0.f;
    return;
  }
  const size_t tok = p.start + p.t0;   // the chunk's first token
  const T* x = (const T*)f.x + tok * (size_t)f.ldx;
  const T* dyp = (const T*)b.dy + tok * (size_t)f.H * DV;
  const T* dt = (const T*)f.dt + tok * (size_t)f.lddt;
  const long long vld = (long long)f.H * DV;

  const int k0 = 16 * (wave % KT), tk = KT == kBwdWaves ? 0 : NK * (wave / KT);   // first state channel and token tile
  const int c0 = 16 * (wave % VT), tv = VT == kBwdWaves ? 0 : NV * (wave / VT);   // first value column and token tile
  // Half strips of the token x token products: tiles (is, 2 jh) and (is, 2 jh + 1).
  const int is = wave & 3, jh = wave >> 2;

  RowTile<T, DV, kBwdThreads> rx, ry;
  float raw = 0.f;
  auto fetch = [&](int h) {
    rx.load(x + (size_t)h * DV, f.ldx, n, tid);
    ry.load(dyp + (size_t)h * DV, vld, n, tid);
    raw = lane < n ? to_f32(dt[(size_t)lane * (size_t)f.lddt + h]) : 0.f;
  };
  {
    RowTile<T, DK, kBwdThreads> rc, rb;
    rc.load((const T*)f.C + tok * (size_t)f.ldc + (size_t)grp * DK, f.ldc, n, tid);
    rb.load((const T*)f.B + tok * (size_t)f.ldb + (size_t)grp * DK, f.ldb, n, tid);
    if (h0 < h1) fetch(h0);
    rc.store(sm.c, tid);
    rb.store(sm.b, tid);
  }
  __syncthreads();
  // P of the wave's half strip, transposed tiles (rows j, columns i), for all heads
  f32x4 pt[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    pt[q] = zero4();
    const int jt = 2 * jh + q;
    if (jt > is) continue;
#pragma unroll
    for (int k = 0; k < DK / 32; ++k) pt[q] = mma(slab_any(sm.b, PK, 16 * jt, 32 * k), slab_any(sm.c, PK, 16 * is, 32 * k), pt[q]);
  }
  f32x4 dC[NK], dB[NK];   // transposed: rows state channels, columns tokens
#pragma unroll
  for (int t = 0; t < NK; ++t) dC[t] = dB[t] = zero4();

  for (int h = h0; h < h1; ++h) {
    // the lane's places, formed anew for every head: kept over the loop they
    // would take about a hundred registers and spill
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int g = ln >> 4, l16 = ln & 15, i_own = 16 * is + l16;
    T* m_own = sm.m + i_own * PM + LdsRow<T>::shift(i_own);
    const RowLanes rk = row_lanes<T>(PK, ln), rv = row_lanes<T>(PV, ln), rm = row_lanes<T>(PM, ln);
    // S and dS, 16 rows a wave, in slabs of 32 value columns loaded two ahead of
    // their use (all of them at once, or a head ahead, spill, and a reload
    // from scratch waits for every load before it)
    const size_t st = ((size_t)item * f.H + h) * (size_t)(DK * DV);
    f32x4 sS[DV / 32][2], sD[DV / 32][2];
    auto fetch_states = [&](int k) {
      const float *pS = a.S + st + (size_t)k0 * DV + 32 * k, *pD = a.dS + st + (size_t)k0 * DV + 32 * k;
      const unsigned off = (unsigned)(l16 * DV + 4 * g);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        sS[k][q] = load4(pS + off + 16 * q);
        sD[k][q] = load4(pD + off + 16 * q);
      }
    };
    fetch_states(0);
    fetch_states(1);
    const double a2 = (double)f.A[h] * 1.4426950408889634074;
    const float bias = f.bias ? f.bias[h] : 0.f;
    StepSize s = step_size(raw, bias, f.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const float slope = f.softplus ? sigmoid_fast(raw + bias) : 1.f;
    const bool cut = s.a == kNothing;   // nothing crosses this token
    const double cum = wave_scan(s.a), last = lane63(cum);
    __syncthreads();   // the head before is done with LDS
    rx.store(sm.x, tid);
    ry.store(sm.dy, tid);
    if (wave == 0) sm.cum[lane] = cum;
    else if (wave == 1) sm.ecum[lane] = exp2_of(cum);
    else if (wave == 2) sm.w[lane] = exp2_of(last - cum);
    else if (wave == 3) sm.dt[lane] = s.dt;
    else if (wave == 4) sm.slope[lane] = slope;
    if (h + 1 < h1) fetch(h + 1);
    __syncthreads();

    // half strip of Qm, and from it R's sums, E dt Qm (to LDS) and E P (kept).
    // A token's decay gradient is a difference of R's row and column sums: both
    // in 64 bits, or their roundings do not cancel and dt_t times them is dA
    double row = 0.0;
    float diag = 0.f, qd = 0.f;
    V4<T> ep[2];
    {
      Slab<T> ys[DV / 32];
#pragma unroll
      for (int k = 0; k < DV / 32; ++k) ys[k] = slab_any(sm.dy, PV, 16 * is, 32 * k, ln);
      const double ci = sm.cum[i_own];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int jt = 2 * jh + q;
        ep[q] = narrow4<T>(zero4());
        if (jt > (is | 1)) continue;   // tile is + 1 of an even strip: zeros complete its slab
        f32x4 nn = zero4(), mm = zero4();
        if (jt <= is) {
          f32x4 acc = zero4();
#pragma unroll
          for (int k = 0; k < DV / 32; ++k) acc = mma(slab_any(sm.x, PV, 16 * jt, 32 * k, ln), ys[k], acc);
          const int j = 16 * jt + 4 * g;
          const f32x4 dj = load4(sm.dt + j);
          double col[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = j + r <= i_own, on = j + r == i_own;
            const float e = exp2_of(ci - sm.cum[j + r]);
            const float m = in ? e * pt[q][r] : 0.f;
            const float rr = in ? m * acc[r] : 0.f;
            mm[r] = m;
            nn[r] = in ? e * dj[r] * acc[r] : 0.f;
            if (on) {
              diag = rr;
              qd = acc[r];
            }
            col[r] = on ? 0.0 : (double)rr;
            row = fma(col[r], (double)dj[r], row);
            col[r] = sum16(col[r]);
          }
          if (l16 == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sm.col[is][j + r] = col[r];
          }
        }
        ep[q] = narrow4<T>(mm);
        store4(m_own + 16 * jt + 4 * g, narrow4<T>(nn));
      }
      row = sum_groups(row);
      if (g == 0) sm.row[jh][i_own] = row;
      diag = sum_groups(diag);   // one lane of a column holds it
      qd = sum_groups(qd);
    }

    // S dy and dS x (transposed: rows the wave's state channels)
    float su[NK], sv[NK], gs;
    {
      f32x4 U[NK], Z[NK], g4 = zero4();
#pragma unroll
      for (int t = 0; t < NK; ++t) U[t] = Z[t] = zero4();
      T* dsp = sm.ds + (k0 + l16) * PV + LdsRow<T>::shift(l16) + 4 * g;
#pragma unroll
      for (int k = 0; k < DV / 32; ++k) {
        if (k + 2 < DV / 32) fetch_states(k + 2);
        const f32x4 s0 = sS[k][0], s1 = sS[k][1], d0 = sD[k][0], d1 = sD[k][1];
#pragma unroll
        for (int r = 0; r < 4; ++r) g4[r] = fmaf(s0[r], d0[r], fmaf(s1[r], d1[r], g4[r]));
        if constexpr (Lds::kKeepDS) {   // (waves that share the rows write the same values)
          store4(dsp + 32 * k, narrow4<T>(d0));
          store4(dsp + 32 * k + 16, narrow4<T>(d1));
        }
        // one operand's parts at a time: more do not fit the registers
        Split<T> sp;
        split_of(s0, s1, sp);
#pragma unroll
        for (int t = 0; t < NK; ++t) U[t] = mma_split(sp, slab_row(sm.dy, rv, 16 * (tk + t) * PV + 32 * k), U[t]);
        __builtin_amdgcn_sched_barrier(0);
        split_of(d0, d1, sp);
#pragma unroll
        for (int t = 0; t < NK; ++t) Z[t] = mma_split(sp, slab_row(sm.x, rv, 16 * (tk + t) * PV + 32 * k), Z[t]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // waves that share state channels (other tokens) hold the same sum
      gs = tk == 0 ? (g4[0] + g4[1]) + (g4[2] + g4[3]) : 0.f;
#pragma unroll
      for (int t = 0; t < NK; ++t) {
        const int it = tk + t, i = 16 * it + l16;
        const float e = sm.ecum[i], w = sm.w[i], wd = w * sm.dt[i];
        const f32x4 c4 = four_of_row(sm.c, PK, 16 * it, k0 + 4 * g, ln), b4 = four_of_row(sm.b, PK, 16 * it, k0 + 4 * g, ln);
        float uu = 0.f, vv = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uu = fmaf(c4[r], U[t][r], uu);
          vv = fmaf(b4[r], Z[t][r], vv);
        }
        dC[t] += e * U[t];
        dB[t] += wd * Z[t];
        su[t] = e * sum_groups(uu);
        sv[t] = w * sum_groups(vv);
      }
    }
    for (int off = 32; off >= 1; off >>= 1) gs += __shfl_xor(gs, off);
    __syncthreads();   // x is used up; E dt Qm is complete
    if (g == 0) {
#pragma unroll
      for (int t = 0; t < NK; ++t) {
        sm.s.u[wave % KT][16 * (tk + t) + l16] = su[t];
        sm.s.v[wave % KT][16 * (tk + t) + l16] = sv[t];
      }
      if (jh == is / 2) {
        sm.s.diag[i_own] = diag;
        sm.s.qd[i_own] = qd;
      }
    }
    if (lane == 0) sm.s.g[wave] = gs;

    // dC += (E dt Qm) B, dB += (E dt Qm)^T C
#pragma unroll
    for (int js = 0; js < 2; ++js) {
      const Slab<T> bs = slab_tr<T>(sm.b, PK, 32 * js, k0, 4, ln), cs = slab_tr<T>(sm.c, PK, 32 * js, k0, 4, ln);
#pragma unroll
      for (int t = 0; t < NK; ++t) {
        const int it = tk + t;
        if (js <= it / 2) dC[t] = mma(bs, slab_row(sm.m, rm, 16 * it * PM + 32 * js), dC[t]);
        if (js >= it / 2) dB[t] = mma(cs, slab_tr<T>(sm.m, PM, 32 * js, 16 * it, 4, ln), dB[t]);
      }
    }
    // dS^T B (transposed: rows the wave's value columns, columns tokens j)
    f32x4 dx[NV];
#pragma unroll
    for (int t = 0; t < NV; ++t) dx[t] = zero4();
#pragma unroll
    for (int k = 0; k < DK / 32; ++k) {
      Slab<T> ds;
      if constexpr (Lds::kKeepDS) {
        ds = slab_tr<T>(sm.ds, PV, 32 * k, c0, 4, ln);
      } else {
        const float* dp = a.dS + st + (size_t)(32 * k + 4 * g) * DV + c0 + l16;
        f32x4 lo, hi;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          lo[r] = dp[r * DV];
          hi[r] = dp[(16 + r) * DV];
        }
        ds = make_slab<T>(lo, hi);
      }
#pragma unroll
      for (int t = 0; t < NV; ++t) dx[t] = mma(ds, slab_row(sm.b, rk, 16 * (tv + t) * PK + 32 * k), dx[t]);
    }
    __syncthreads();   // E dt Qm is used up; the sums are complete
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (2 * jh + q <= (is | 1)) store4(m_own + 16 * (2 * jh + q) + 4 * g, ep[q]);
    __syncthreads();
    // dx
    const float dskip = f.D ? f.D[h] : 0.f;
    const Slab<T> y0 = slab_tr<T>(sm.dy, PV, 0, c0, 4, ln), y1 = slab_tr<T>(sm.dy, PV, 32, c0, 4, ln);
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      const int it = tv + t, j = 16 * it + l16, c = c0 + 4 * g;
      const float dj = sm.dt[j];
      dx[t] *= sm.w[j];
      if (it < 2) dx[t] = mma(y0, slab_tr<T>(sm.m, PM, 0, 16 * it, 4, ln), dx[t]);
      dx[t] = mma(y1, slab_tr<T>(sm.m, PM, 32, 16 * it, 4, ln), dx[t]);
      f32x4 o = dj * dx[t];
      if (f.D) o += dskip * four_of_row(sm.dy, PV, 16 * it, c, ln);
      const float ov[4] = {o[0], o[1], o[2], o[3]};
      if (j < n) Rows<T, 4>::store((T*)b.dx + (tok + j) * (size_t)vld + (size_t)h * DV + c, ov);
    }
    if (wave == 0) {
      // the chunk's per-token sums: lane = token
      double u = 0.0, v = 0.0, cs = 0.0, gsum = 0.0;
#pragma unroll
      for (int q = 0; q < KT; ++q) {
        u += (double)sm.s.u[q][lane];
        v += (double)sm.s.v[q][lane];
      }
      // a strip before token j's tile has no entry of column j
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q >= lane >> 4) cs += sm.col[q][lane];
#pragma unroll
      for (int q = 0; q < kBwdWaves; ++q) gsum += (double)sm.s.g[q];
      const double dts = (double)sm.dt[lane], vd = v * dts;
      const double net = (sm.row[0][lane] + sm.row[1][lane]) + u - cs * dts - vd;
      const double incl = wave_scan(net);
      const double all = lane63(incl) + lane63(wave_scan(vd)) + (double)exp2_of(sm.cum[kQ - 1]) * gsum;
      // (what is left of the sums at a cut is their rounding; dt_t is large there)
      const double da = cut ? 0.0 : all - (incl - net);
      double d = ((double)f.A[h] * da + cs + sm.s.diag[lane] + v) * (double)sm.slope[lane];
      if (lane >= n) d = 0.0;
      if (lane < n) ((T*)b.ddt)[(tok + lane) * (size_t)f.H + h] = from_f32<T>((float)d);
      const double sA = lane63(wave_scan(da * dts)), sD = lane63(wave_scan((double)sm.s.qd[lane])), sb = lane63(wave_scan(d));
      if (lane == 0) {
        float* o = a.part + (size_t)item * 3 * f.H + h;
        o[0] = (float)sA;
        o[f.H] = (float)sD;
        o[2 * f.H] = (float)sb;
      }
    }
  }
  // sums over the heads
#pragma unroll
  for (int t = 0; t < NK; ++t) {
    const int i = 16 * (tk + t) + l16;
    if (i >= n) continue;
    const size_t at = ((tok + i) * (size_t)f.G + grp) * DK + k0 + 4 * g;
    const float oc[4] = {dC[t][0], dC[t][1], dC[t][2], dC[t][3]}, ob[4] = {dB[t][0], dB[t][1], dB[t][2], dB[t][3]};
    if (a.shares > 1) {
      const size_t sh = (size_t)share * a.tokens * f.G * DK;
      Rows<float, 4>::store(a.dCp + sh + at, oc);
      Rows<float, 4>::store(a.dBp + sh + at, ob);
    } else {
      Rows<T, 4>::store((T*)b.dC + at, oc);
      Rows<T, 4>::store((T*)b.dB + at, ob);
    }
  }
}

// dB and dC from the shares of a group's heads, eight elements a thread.
template <typename T>
__global__ __launch_bounds__(256) void ssm_shares_kernel(const float* __restrict__ bp, const float* __restrict__ cp, T* __restrict__ dB,
                                                         T* __restrict__ dC, size_t n8, int shares) {
  const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= 2 * n8) return;
  const float* src = id < n8 ? bp : cp;
  const size_t at = (id < n8 ? id : id - n8) * 8;
  float s[8] = {}, v[8];
  for (int k = 0; k < shares; ++k) {
    Rows<float, 8>::load(src + (size_t)k * n8 * 8 + at, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += v[i];
  }
  Rows<T, 8>::store((id < n8 ? dB : dC) + at, s);
}

// Work-groups a group's heads are split over: enough for about one per CU (1000
// tokens x 32 heads: 128 us; for two per CU, the sums over the shares make it
// 140).
int head_shares(long long chunks, int H, int G) {
  long long s = 1;
  while (s < H / G && chunks * G * s < 256) s *= 2;
  return (int)(s < H / G ? s : H / G);
}

struct BwdLayout {
  size_t seg, sum, S, dS, part, dBp, dCp, total, chunks;
  int shares;
};
BwdLayout bwd_layout(int is_packed, int N, int B, int T, int H, int G, int dk, int dv) {
  const size_t tokens = (size_t)B * T, sd = (size_t)dk * dv * sizeof(float), slots = ssm_slots((long long)tokens, H, kSweepWgs);
  BwdLayout L{};
  L.chunks = is_packed ? (size_t)T / kQ + N : (size_t)B * (((size_t)T + kQ - 1) / kQ);
  L.shares = head_shares((long long)L.chunks, H, G);
  size_t off = 0;
  auto put = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  L.seg = put(slots * sd);
  L.sum = put(slots * sizeof(double));
  L.S = put(L.chunks * H * sd);
  L.dS = put(L.chunks * H * sd);
  L.part = put(L.chunks * 3 * H * sizeof(float));
  const size_t share = L.shares > 1 ? (size_t)L.shares * tokens * G * dk * sizeof(float) : 0;
  L.dBp = put(share);
  L.dCp = put(share);
  L.total = off;
  return L;
}

template <typename T, int DK, int DV>
hipError_t bwd_go(const SsmBwdArgs& b, const BwdLayout& L, const int* cu, int N, int B, int Tn, char* ws, hipStream_t st) {
  const long long tokens = (long long)B * Tn;
  const int part = ssm_part_of(b.f.H, kSweepWgs, cu, N, B, Tn), end = cu ? N : B;
  ChunkBwd a{};
  a.b = b;
  a.b.f.seg = reinterpret_cast<float*>(ws + L.seg);
  a.b.f.sum = reinterpret_cast<double*>(ws + L.sum);
  a.b.f.start = nullptr;
  a.tokens = (size_t)tokens;
  a.shares = L.shares;
  a.dBp = reinterpret_cast<float*>(ws + L.dBp);
  a.dCp = reinterpret_cast<float*>(ws + L.dCp);
  size_t done = 0;   // chunks of the launches before
  for (int n = 0; n < end;) {
    SeqTab s, sc;
    const int n0 = n;
    n = make_seq_tab(s, cu, N, n0, B, Tn, part);
    make_seq_tab(sc, cu, N, n0, B, Tn, kQ);
    const bool split = s.items > n - n0;
    const size_t at = done * (size_t)b.f.H;
    float* S = reinterpret_cast<float*>(ws + L.S) + at * (DK * DV);
    float* dS = reinterpret_cast<float*>(ws + L.dS) + at * (DK * DV);
    SweepArgs w{};
    w.f = a.b.f;
    w.rows = b.f.B;
    w.ldrows = b.f.ldb;
    w.cols = b.f.x;
    w.ldcols = b.f.ldx;
    w.from = b.f.h0;
    w.at = S;
    w.subs = 1;
    hipError_t e = hipSuccess;
    if (split) {
      e = launch_sweep<T, DK, DV, false, false, true>(w, s, st);
      if (e == hipSuccess) e = launch_chain(w, s, n - n0, DK * DV, false, st);
      if (e != hipSuccess) return e;
    }
    if ((e = launch_sweep<T, DK, DV, false, true, true>(w, s, st)) != hipSuccess) return e;
    w.rows = b.f.C;
    w.ldrows = b.f.ldc;
    w.cols = b.dy;
    w.ldcols = (long long)b.f.H * DV;
    w.from = b.dht;
    w.to = b.dh0;
    w.at = dS;
    if (split) {
      e = launch_sweep<T, DK, DV, true, false, true>(w, s, st);
      if (e == hipSuccess) e = launch_chain(w, s, n - n0, DK * DV, true, st);
      if (e != hipSuccess) return e;
    }
    if ((e = launch_sweep<T, DK, DV, true, true, true>(w, s, st)) != hipSuccess) return e;
    a.S = S;
    a.dS = dS;
    a.part = reinterpret_cast<float*>(ws + L.part) + at * 3;
    const dim3 grid((unsigned)sc.items * (unsigned)(b.f.G * a.shares));
    hipLaunchKernelGGL((ssm_bwd_kernel<T, DK, DV>), grid, dim3(kBwdThreads), 0, st, a, sc);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    done += (size_t)sc.items;
  }
  if (a.shares > 1) {
    const size_t n8 = (size_t)tokens * b.f.G * DK / 8;
    // (several shares: fewer than 256 chunks)
    hipLaunchKernelGGL((ssm_shares_kernel<T>), dim3((unsigned)((2 * n8 + 255) / 256)), dim3(256), 0, st, a.dBp, a.dCp, (T*)b.dB, (T*)b.dC,
                       n8, a.shares);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_sum_rows(reinterpret_cast<float*>(ws + L.part), done, (unsigned)b.f.H, (unsigned)b.f.H, (unsigned)b.f.H, b.dA, b.dD,
                         b.dbias, st);
}

template <typename T>
hipError_t bwd_dims(const SsmBwdArgs& b, int dk, int dv, const BwdLayout& L, const int* cu, int N, int B, int Tn, char* ws, hipStream_t st) {
  if (dk == 128 && dv == 128) return bwd_go<T, 128, 128>(b, L, cu, N, B, Tn, ws, st);
  if (dk == 128) return bwd_go<T, 128, 64>(b, L, cu, N, B, Tn, ws, st);
  if (dv == 128) return bwd_go<T, 64, 128>(b, L, cu, N, B, Tn, ws, st);
  return bwd_go<T, 64, 64>(b, L, cu, N, B, Tn, ws, st);
}

}  // namespace

size_t ssm_bwd_workspace_bytes(int is_packed, int N, int B, int T, int H, int G, int dk, int dv) {
  return bwd_layout(is_packed, N, B, T, H, G, dk, dv).total;
}

hipError_t launch_ssm_bwd(int is_bf16, const SsmBwdArgs& a, int dk, int dv, const int* cu, int N, int B, int T, void* workspace,
                          hipStream_t st) {
  // parts are longer than chunks, and a chunk has at most one work-group a head
  if (!seq_tabs_fit(cu, N, B, T, kQ, most_items(a.f.H))) return hipErrorInvalidConfiguration;
  const BwdLayout L = bwd_layout(cu != nullptr, N, B, T, a.f.H, a.f.G, dk, dv);
  char* ws = static_cast<char*>(workspace);
  return is_bf16 ? bwd_dims<bf16>(a, dk, dv, L, cu, N, B, T, ws, st) : bwd_dims<float>(a, dk, dv, L, cu, N, B, T, ws, st);
}

}  // namespace kda
