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
// Bound by HBM: a state and its gradient per chunk and head, written and read
// (4 dk dv 4 bytes each way), are the bulk beside the inputs.
//
// Rounding (bf16): the elementwise weights of the products that end in dx, dB
// and dC (bf16 outputs) are rounded to bf16 once, dS^T B's operand dS too; S
// dy and dS x feed fp32 sums (dA, and ddt through differences of large sums)
// and take S and dS in three bf16 parts (24 bits).
#include "kda_ssm_sweep.h"

namespace kda {

namespace {

constexpr int kSweepWgs = 512;   // two sweep work-groups per CU

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
    struct {   // when x has been used up: sums of the four waves
      float u[kSsmWaves][kQ], v[kSsmWaves][kQ], col[kSsmWaves][kQ], row[kQ], diag[kQ], qd[kQ], g[kSsmWaves];
    } s;
  };
  T dy[kQ * PV];
  T m[kQ * PM];              // E dt Qm, then E P: [i][j]
  double cum[kQ];
  float ecum[kQ], w[kQ], dt[kQ];
};

// Sum over the 16 lanes of a row of lanes, by lane permutations.
__device__ __forceinline__ float sum16(float x) {
  x += dpp_f<0xB1>(x);    // quad_perm [1,0,3,2]
  x += dpp_f<0x4E>(x);    // quad_perm [2,3,0,1]
  x += dpp_f<0x141>(x);   // row_half_mirror
  x += dpp_f<0x140>(x);   // row_mirror
  return x;
}
// Sum over the four lane groups that hold one column of a tile.
__device__ __forceinline__ float sum_groups(float x) {
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kSsmThreads, sizeof(T) == 2 ? 2 : 1) void ssm_bwd_kernel(const ChunkBwd a, const SeqTab sq) {
  typedef BwdLds<T, DK, DV> Lds;
  constexpr int PK = Lds::PK, PV = Lds::PV, PM = Lds::PM;
  constexpr int CPK = DK / kSsmWaves, NK = CPK / 16, CPV = DV / kSsmWaves, NV = CPV / 16;
  __shared__ __align__(16) char smem[sizeof(Lds)];
  Lds& sm = *reinterpret_cast<Lds*>(smem);
  const SsmBwdArgs& b = a.b;
  const SsmArgs& f = b.f;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
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

  // The output rows (state channels, value columns) of this lane in a
  // transposed tile: rows m of tile t are base + 4 N (m/4) + 4t + m%4.
  const int k0 = wave * CPK, c0 = wave * CPV;
  const int i_own = 16 * wave + l16;   // column of the strip this wave forms
  T* m_own = sm.m + i_own * PM + LdsRow<T>::shift(i_own);

  RowTile<T, DV> rx, ry;
  float raw = 0.f;
  auto fetch = [&](int h) {
    rx.load(x + (size_t)h * DV, f.ldx, n, tid);
    ry.load(dyp + (size_t)h * DV, vld, n, tid);
    raw = lane < n ? to_f32(dt[(size_t)lane * (size_t)f.lddt + h]) : 0.f;
  };
  {
    RowTile<T, DK> rc, rb;
    rc.load((const T*)f.C + tok * (size_t)f.ldc + (size_t)grp * DK, f.ldc, n, tid);
    rb.load((const T*)f.B + tok * (size_t)f.ldb + (size_t)grp * DK, f.ldb, n, tid);
    if (h0 < h1) fetch(h0);
    rc.store(sm.c, tid);
    rb.store(sm.b, tid);
  }
  __syncthreads();
  // P of the wave's strip, transposed tiles (rows j, columns i), for all heads
  f32x4 pt[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    pt[jt] = zero4();
    if (jt > wave) continue;
#pragma unroll
    for (int k = 0; k < DK / 32; ++k)
      pt[jt] = mma(slab_any(sm.b, PK, 16 * jt, 32 * k), slab_any(sm.c, PK, 16 * wave, 32 * k), pt[jt]);
  }
  f32x4 dC[4][NK], dB[4][NK];   // transposed: rows state channels, columns tokens
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int q = 0; q < NK; ++q) dC[it][q] = dB[it][q] = zero4();

  for (int h = h0; h < h1; ++h) {
    const double a2 = (double)f.A[h] * 1.4426950408889634074;
    const float bias = f.bias ? f.bias[h] : 0.f, rawv = raw;
    StepSize s = step_size(raw, bias, f.softplus, a2);
    if (lane >= n) s = StepSize{0.f, 0.0};
    const double cum = wave_scan(s.a), last = lane63(cum);
    __syncthreads();   // the head before is done with LDS
    rx.store(sm.x, tid);
    ry.store(sm.dy, tid);
    if (wave == 0) sm.cum[lane] = cum;
    else if (wave == 1) sm.ecum[lane] = exp2_of(cum);
    else if (wave == 2) sm.w[lane] = exp2_of(last - cum);
    else sm.dt[lane] = s.dt;
    if (h + 1 < h1) fetch(h + 1);
    __syncthreads();

    // strip of Qm, and from it R's sums, E dt Qm (to LDS) and E P (kept)
    float row = 0.f, diag = 0.f, qd = 0.f;
    f32x4 col[4];
    V4<T> ep[4];
    {
      Slab<T> ys[DV / 32];
#pragma unroll
      for (int k = 0; k < DV / 32; ++k) ys[k] = slab_any(sm.dy, PV, 16 * wave, 32 * k);
      const double ci = sm.cum[i_own];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        col[jt] = zero4();
        ep[jt] = narrow4<T>(zero4());
        if (jt > (wave | 1)) continue;   // tile wave + 1 of an even strip: zeros complete its slab
        f32x4 nn = zero4(), mm = zero4();
        if (jt <= wave) {
          f32x4 acc = zero4();
#pragma unroll
          for (int k = 0; k < DV / 32; ++k) acc = mma(slab_any(sm.x, PV, 16 * jt, 32 * k), ys[k], acc);
          const int j = 16 * jt + 4 * g;
          const f32x4 dj = load4(sm.dt + j);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = j + r <= i_own, on = j + r == i_own;
            const float e = exp2_of(ci - sm.cum[j + r]);
            const float m = in ? e * pt[jt][r] : 0.f;
            const float rr = in ? m * acc[r] : 0.f;
            mm[r] = m;
            nn[r] = in ? e * dj[r] * acc[r] : 0.f;
            if (on) {
              diag = rr;
              qd = acc[r];
            } else {
              row = fmaf(rr, dj[r], row);
              col[jt][r] = rr;
            }
          }
        }
        ep[jt] = narrow4<T>(mm);
        store4(m_own + 16 * jt + 4 * g, narrow4<T>(nn));
      }
      row = sum_groups(row);
      diag = sum_groups(diag);   // one lane of a column holds it
      qd = sum_groups(qd);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt)
#pragma unroll
        for (int r = 0; r < 4; ++r) col[jt][r] = sum16(col[jt][r]);
    }

    // S dy and dS x (transposed: rows the wave's state channels)
    const size_t st = ((size_t)item * f.H + h) * (size_t)(DK * DV);
    float su[4], sv[4], gs;
    {
      f32x4 U[4][NK], Z[4][NK], g4 = zero4();
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int q = 0; q < NK; ++q) U[it][q] = Z[it][q] = zero4();
#pragma unroll 1
      for (int k = 0; k < DV / 32; ++k) {
        Split<T> ss[NK], ds[NK];
#pragma unroll
        for (int q = 0; q < NK; ++q) {
          const size_t at = st + (size_t)(k0 + 4 * NK * (l16 >> 2) + 4 * q + (l16 & 3)) * DV + 32 * k + 4 * g;
          const f32x4 s0 = load4(a.S + at), s1 = load4(a.S + at + 16), d0 = load4(a.dS + at), d1 = load4(a.dS + at + 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) g4[r] = fmaf(s0[r], d0[r], fmaf(s1[r], d1[r], g4[r]));
          split_of(s0, s1, ss[q]);
          split_of(d0, d1, ds[q]);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const Slab<T> ys = slab_row(sm.dy, PV, 16 * it, 32 * k), xs = slab_row(sm.x, PV, 16 * it, 32 * k);
#pragma unroll
          for (int q = 0; q < NK; ++q) {
            U[it][q] = mma_split(ss[q], ys, U[it][q]);
            Z[it][q] = mma_split(ds[q], xs, Z[it][q]);
          }
        }
      }
      gs = (g4[0] + g4[1]) + (g4[2] + g4[3]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int i = 16 * it + l16;
        const float e = sm.ecum[i], w = sm.w[i], wd = w * sm.dt[i];
        float uu = 0.f, vv = 0.f;
#pragma unroll
        for (int q = 0; q < NK; ++q) {
          const f32x4 c4 = four_of_row(sm.c, PK, 16 * it, k0 + 4 * NK * g + 4 * q), b4 = four_of_row(sm.b, PK, 16 * it, k0 + 4 * NK * g + 4 * q);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uu = fmaf(c4[r], U[it][q][r], uu);
            vv = fmaf(b4[r], Z[it][q][r], vv);
          }
          dC[it][q] += e * U[it][q];
          dB[it][q] += wd * Z[it][q];
        }
        su[it] = e * sum_groups(uu);
        sv[it] = w * sum_groups(vv);
      }
    }
    __syncthreads();   // x is used up; E dt Qm is complete
    if (g == 0) {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        sm.s.u[wave][16 * it + l16] = su[it];
        sm.s.v[wave][16 * it + l16] = sv[it];
      }
      sm.s.row[i_own] = row;
      sm.s.diag[i_own] = diag;
      sm.s.qd[i_own] = qd;
    }
    if (l16 == 0) {
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) store4(&sm.s.col[wave][16 * jt + 4 * g], col[jt]);
    }
    for (int off = 32; off >= 1; off >>= 1) gs += __shfl_xor(gs, off);
    if (lane == 0) sm.s.g[wave] = gs;

    // dC += (E dt Qm) B, dB += (E dt Qm)^T C
#pragma unroll
    for (int js = 0; js < 2; ++js) {
#pragma unroll
      for (int q = 0; q < NK; ++q) {
        const Slab<T> bs = slab_tr<T>(sm.b, PK, 32 * js, k0 + 4 * q, 4 * NK), cs = slab_tr<T>(sm.c, PK, 32 * js, k0 + 4 * q, 4 * NK);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          if (js <= it / 2) dC[it][q] = mma(bs, slab_row(sm.m, PM, 16 * it, 32 * js), dC[it][q]);
          if (js >= it / 2) dB[it][q] = mma(cs, slab_tr<T>(sm.m, PM, 32 * js, 16 * it, 4), dB[it][q]);
        }
      }
    }
    // dS^T B (transposed: rows the wave's value columns, columns tokens j)
    f32x4 dx[4][NV];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int q = 0; q < NV; ++q) dx[it][q] = zero4();
#pragma unroll 1
    for (int k = 0; k < DK / 32; ++k) {
      Slab<T> ds[NV];
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const float* dp = a.dS + st + (size_t)(32 * k + 4 * g) * DV + c0 + 4 * NV * (l16 >> 2) + 4 * q + (l16 & 3);
        f32x4 lo, hi;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          lo[r] = dp[(size_t)r * DV];
          hi[r] = dp[(size_t)(16 + r) * DV];
        }
        ds[q] = make_slab<T>(lo, hi);
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const Slab<T> bs = slab_row(sm.b, PK, 16 * it, 32 * k);
#pragma unroll
        for (int q = 0; q < NV; ++q) dx[it][q] = mma(ds[q], bs, dx[it][q]);
      }
    }
    __syncthreads();   // E dt Qm is used up; the sums are complete
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= (wave | 1)) store4(m_own + 16 * jt + 4 * g, ep[jt]);
    if (wave == 0) {
      // the chunk's per-token sums: lane = token
      const double u = ((double)sm.s.u[0][lane] + sm.s.u[1][lane]) + ((double)sm.s.u[2][lane] + sm.s.u[3][lane]);
      const double v = ((double)sm.s.v[0][lane] + sm.s.v[1][lane]) + ((double)sm.s.v[2][lane] + sm.s.v[3][lane]);
      double cs = 0.0;   // a strip before token j's tile has no entry of column j
#pragma unroll
      for (int q = 0; q < kSsmWaves; ++q)
        if (q >= lane >> 4) cs += (double)sm.s.col[q][lane];
      const double vd = v * s.dt;
      const double net = (double)sm.s.row[lane] + u - cs * s.dt - vd;
      const double gsum = ((double)sm.s.g[0] + sm.s.g[1]) + ((double)sm.s.g[2] + sm.s.g[3]);
      const double incl = wave_scan(net);
      const double all = lane63(incl) + lane63(wave_scan(vd)) + (double)exp2_of(last) * gsum;
      const double da = all - (incl - net);
      double d = (double)f.A[h] * da + cs + sm.s.diag[lane] + v;
      if (f.softplus) d *= (double)sigmoid_fast(rawv + bias);
      if (lane >= n) d = 0.0;
      if (lane < n) ((T*)b.ddt)[(tok + lane) * (size_t)f.H + h] = from_f32<T>((float)d);
      const double sA = lane63(wave_scan(da * s.dt)), sD = lane63(wave_scan((double)sm.s.qd[lane])), sb = lane63(wave_scan(d));
      if (lane == 0) {
        float* o = a.part + (size_t)item * 3 * f.H + h;
        o[0] = (float)sA;
        o[f.H] = (float)sD;
        o[2 * f.H] = (float)sb;
      }
    }
    __syncthreads();
    // dx
    const float dskip = f.D ? f.D[h] : 0.f;
    Slab<T> ysT[2][NV];
#pragma unroll
    for (int js = 0; js < 2; ++js)
#pragma unroll
      for (int q = 0; q < NV; ++q) ysT[js][q] = slab_tr<T>(sm.dy, PV, 32 * js, c0 + 4 * q, 4 * NV);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int j = 16 * it + l16, c = c0 + 4 * NV * g;
      const float w = sm.w[j], dj = sm.dt[j];
#pragma unroll
      for (int q = 0; q < NV; ++q) dx[it][q] *= w;
#pragma unroll
      for (int js = it / 2; js < 2; ++js) {
        const Slab<T> ms = slab_tr<T>(sm.m, PM, 32 * js, 16 * it, 4);
#pragma unroll
        for (int q = 0; q < NV; ++q) dx[it][q] = mma(ysT[js][q], ms, dx[it][q]);
      }
      float o[4 * NV];
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const f32x4 yj = four_of_row(sm.dy, PV, 16 * it, c + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[4 * q + r] = f.D ? fmaf(dskip, yj[r], dj * dx[it][q][r]) : dj * dx[it][q][r];
      }
      if (j < n) Rows<T, 4 * NV>::store((T*)b.dx + (tok + j) * (size_t)vld + (size_t)h * DV + c, o);
    }
  }
  // sums over the heads
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int i = 16 * it + l16;
    if (i >= n) continue;
    const size_t at = ((tok + i) * (size_t)f.G + grp) * DK + k0 + 4 * NK * g;
    float oc[4 * NK], ob[4 * NK];
#pragma unroll
    for (int q = 0; q < NK; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        oc[4 * q + r] = dC[it][q][r];
        ob[4 * q + r] = dB[it][q][r];
      }
    if (a.shares > 1) {
      const size_t sh = (size_t)share * a.tokens * f.G * DK;
      Rows<float, 4 * NK>::store(a.dCp + sh + at, oc);
      Rows<float, 4 * NK>::store(a.dBp + sh + at, ob);
    } else {
      Rows<T, 4 * NK>::store((T*)b.dC + at, oc);
      Rows<T, 4 * NK>::store((T*)b.dB + at, ob);
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

// Work-groups a group's heads are split over: enough for about two per CU.
int head_shares(long long chunks, int H, int G) {
  long long s = 1;
  while (s < H / G && chunks * G * s < 512) s *= 2;
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
  const int part = ssm_part(tokens, b.f.H, kSweepWgs), end = cu ? N : B;
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
    if (s.items < 0 || sc.items < 0) return hipErrorInvalidConfiguration;
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
    const long long blocks = (long long)sc.items * b.f.G * a.shares;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssm_bwd_kernel<T, DK, DV>), dim3((unsigned)blocks), dim3(kSsmThreads), 0, st, a, sc);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    done += (size_t)sc.items;
  }
  if (a.shares > 1) {
    const size_t n8 = (size_t)tokens * b.f.G * DK / 8;
    if (2 * n8 / 256 + 1 > 0x7fffffffULL) return hipErrorInvalidConfiguration;
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
  const BwdLayout L = bwd_layout(cu != nullptr, N, B, T, a.f.H, a.f.G, dk, dv);
  char* ws = static_cast<char*>(workspace);
  return is_bf16 ? bwd_dims<bf16>(a, dk, dv, L, cu, N, B, T, ws, st) : bwd_dims<float>(a, dk, dv, L, cu, N, B, T, ws, st);
}

}  // namespace kda
