// Short causal depthwise convolution of the projections in front of a
// recurrence, with its carried state, gradients and single-token step.
//
//   z[t, c] = bias[c] + sum_j w[c, j] x[t - (W-1-j), c],   j = 0 .. W-1
//   y = z, or z Sigmoid(z)
// Tokens before a sequence's first come from its state (W-1 rows, oldest
// first; zero without one); the state behind a sequence is its last W-1
// inputs.  Rows [state, tokens] together are numbered e = 0 .. len+W-2:
// token t reads rows t .. t+W-1, and the final state is rows len .. len+W-2.
//
// Bound by HBM: every input once, every output once, 2W operations each.
// One thread owns VE = 4 neighbouring channels (their weights are 16 bytes a
// channel: with eight channels a thread a wave's weights lie in twice as many
// cache lines per load) of a strip of tokens and walks it with the last W-1
// rows in registers, eight rows' loads in flight; only the W-1 rows before a
// strip are read twice (from the caches).  All sums in fp32, one rounding to the output type.
// Measured (bf16): 65536 tokens x 4096 channels 195 us (5.5 TB/s); 8191 packed
// tokens x 4352 channels 30 us (4.7 TB/s, rows of a wider tensor); gradients of
// 32768 tokens x 2048 channels from fp32 dy 114 us (4.7 TB/s); a token for 256
// sequences x 4352 channels 4.5 us (3.9 TB/s), twice that through the Python
// binding.  Eight channels a thread took 207, 34 and 123 us where four took
// 199, 32 and 114.
#include "kda_rows.h"

namespace kda {

namespace {

constexpr int kConvThreads = 256;
// Rows loaded together: forward (64K tokens x 4096 channels: 203 us, 16K: 46;
// four 214 and 46, sixteen 200 and 51), and x and dy rows of the backward (32K x
// 2048: 115 us, 16K of fp32: 84; four 153 and 78, one 114 and 104).
constexpr int kFwdRows = 8;
constexpr int kBwdRows = 2;

__device__ __forceinline__ float act_of(float z, int silu) { return silu ? z * sigmoid_fast(z) : z; }

// Row e of [state, tokens] of sequence p, channels c ..
template <typename T, int VE>
__device__ __forceinline__ void ext_row(const ConvArgs& a, const SeqPart& p, int e, int c, float (&x)[VE]) {
  const int W1 = a.W - 1;
  if (e >= W1) {
    Rows<T, VE>::load((const T*)a.x + (p.start + (size_t)(e - W1)) * (size_t)a.ldx + c, x);
  } else if (a.s0) {
    Rows<T, VE>::load((const T*)a.s0 + ((size_t)p.n * W1 + e) * a.D + c, x);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = 0.f;
  }
}

template <int W, int VE>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, float (&w)[W][VE], float (&b)[VE]) {
#pragma unroll
  for (int i = 0; i < VE; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = a.w[(size_t)(c + i) * W + j];
    b[i] = a.bias ? a.bias[c + i] : 0.f;
  }
}

// The state behind sequence p: rows len .. len+W-2.  Row r comes from a later
// row (or the same one), so a state may be replaced in place by one thread.
template <typename T, int VE>
__device__ __forceinline__ void final_state(const ConvArgs& a, const SeqPart& p, int c) {
  for (int r = 0; r < a.W - 1; ++r) {
    float x[VE];
    ext_row<T, VE>(a, p, p.len + r, c, x);
    Rows<T, VE>::store((T*)a.st + ((size_t)p.n * (a.W - 1) + r) * a.D + c, x);
  }
}

template <typename T, int W, int VE>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const ConvArgs a, const SeqTab s, unsigned CG) {
  const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
  const unsigned item = id / CG;
  if (item >= (unsigned)s.items) return;
  const int c = (int)(id - item * CG) * VE;
  const SeqPart p = seq_part(s, (int)item);
  float w[W][VE], b[VE];
  load_taps<W, VE>(a, c, w, b);
  float buf[W - 1 + kFwdRows][VE];   // rows t .. of [state, tokens]
#pragma unroll
  for (int k = 0; k < W - 1; ++k) ext_row<T, VE>(a, p, p.t0 + k, c, buf[k]);
  const T* x = (const T*)a.x + p.start * (size_t)a.ldx + c;
  T* y = (T*)a.y + p.start * (size_t)a.D + c;
  for (int t = p.t0; t < p.t1; t += kFwdRows) {
    // rows past the strip re-read its last one and are not stored
#pragma unroll
    for (int u = 0; u < kFwdRows; ++u)
      Rows<T, VE>::load(x + (size_t)min(t + u, p.t1 - 1) * (size_t)a.ldx, buf[W - 1 + u]);
#pragma unroll
    for (int u = 0; u < kFwdRows; ++u) {
      float o[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        float z = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) z = fmaf(w[j][i], buf[u + j][i], z);
        o[i] = act_of(z, a.silu);
      }
      if (t + u < p.t1) Rows<T, VE>::store(y + (size_t)(t + u) * a.D, o);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i) buf[k][i] = buf[kFwdRows + k][i];
  }
  if (a.st && p.last) final_state<T, VE>(a, p, c);
}

// Final states alone (the in-place carry of sequences of several strips,
// after the forward has read the old states).
template <typename T, int VE>
__global__ __launch_bounds__(kConvThreads) void conv_state_kernel(const ConvArgs a, const SeqTab s, unsigned CG) {
  const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
  const unsigned item = id / CG;
  if (item >= (unsigned)s.items) return;
  final_state<T, VE>(a, seq_part(s, (int)item), (int)(id - item * CG) * VE);
}

// One token per sequence: y from the state's rows and x, and the state moved
// on by one row (st may be s0: a thread reads all its rows first).  A thread
// takes one channel, so that a wave's weights are one contiguous piece, of S
// sequences, whose weights it loads once.
template <typename T, int W, int S>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(const ConvArgs a, unsigned B) {
  const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
  const unsigned D = (unsigned)a.D, n0 = id / D * S;
  if (n0 >= B) return;
  const int c = (int)(id % D);
  float r[S][W], w[W][1], b[1];
#pragma unroll
  for (int q = 0; q < S; ++q) {
    // a sequence past the last re-reads that one and is not stored
    const size_t n = min(n0 + q, B - 1);
    const T* s0 = (const T*)a.s0 + n * (W - 1) * D + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) r[q][k] = to_f32(s0[(size_t)k * D]);
    r[q][W - 1] = to_f32(((const T*)a.x)[n * (size_t)a.ldx + c]);
  }
  load_taps<W, 1>(a, c, w, b);
#pragma unroll
  for (int q = 0; q < S; ++q) {
    const size_t n = n0 + q;
    if (n >= B) return;
    float z = b[0];
#pragma unroll
    for (int j = 0; j < W; ++j) z = fmaf(w[j][0], r[q][j], z);
    ((T*)a.y)[n * D + c] = from_f32<T>(act_of(z, a.silu));
    T* st = (T*)a.st + n * (W - 1) * D + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) st[(size_t)k * D] = from_f32<T>(r[q][k + 1]);
  }
}

// Gradients.  With dz = dy act'(z) (z recomputed from x), row e of [state,
// tokens] gets
//   sum_j w[j] dz[e - j]  (+ the final state's gradient, row e - len)
// which is dx of token e-(W-1), or ds0 of row e for e < W-1.  A thread walks
// e = t0 .. t1+W-2 of its strip with the last W rows of x and of dz in
// registers, and sums dw[j] = sum_t dz[t] x[t+j] and dbias over its own
// tokens.  Threads of a work-group that share channels add their sums through
// lane moves and LDS in a fixed order, one partial row a work-group;
// sum_rows_kernel adds those in order: no atomics, the same result every time.
template <typename T, typename TG, int W, int VE>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const ConvBwdArgs a, const SeqTab s, unsigned CG, unsigned LC,
                                                                unsigned cblocks) {
  constexpr int kWaves = kConvThreads / 64;
  __shared__ float red[kWaves][64 * VE * (W + 1)];
  const ConvArgs& f = a.f;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned grp = blockIdx.x / cblocks, cb = blockIdx.x - grp * cblocks;
  const unsigned cg = cb * LC + (lane & (LC - 1));
  const unsigned per = 64u / LC * kWaves;   // strips of a work-group
  const unsigned item = grp * per + wave * (64u / LC) + lane / LC;
  const bool live = cg < CG && item < (unsigned)s.items;
  const int c = (int)(live ? cg : 0) * VE;
  float dw[W][VE], db[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  if (live) {
    const SeqPart p = seq_part(s, (int)item);
    float w[W][VE], b[VE];
    load_taps<W, VE>(f, c, w, b);
    float buf[W - 1 + kBwdRows][VE], dz[W - 1 + kBwdRows][VE];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      ext_row<T, VE>(f, p, p.t0 + k, c, buf[k]);
#pragma unroll
      for (int i = 0; i < VE; ++i) dz[k][i] = 0.f;
    }
    const T* x = (const T*)f.x + p.start * (size_t)f.ldx + c;
    const TG* dy = (const TG*)a.dy + p.start * (size_t)f.D + c;
    T* dx = (T*)a.dx + p.start * (size_t)f.D + c;
    const int e1 = p.t1 + W - 1;              // rows e < e1
    const int tl = min(e1, p.len);            // tokens whose dz this strip needs
    for (int t = p.t0; t < e1; t += kBwdRows) {
      float g[kBwdRows][VE];
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        if (t + u < tl) {
          Rows<T, VE>::load(x + (size_t)(t + u) * (size_t)f.ldx, buf[W - 1 + u]);
          Rows<TG, VE>::load(dy + (size_t)(t + u) * f.D, g[u]);
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i) buf[W - 1 + u][i] = g[u][i] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        const bool mine = t + u < p.t1;
        float o[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          float d = g[u][i];
          if (f.silu) {
            float z = b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) z = fmaf(w[j][i], buf[u + j][i], z);
            const float sg = sigmoid_fast(z);
            // act'(z) = sg (1 + z (1 - sg)); a token past the end has no gradient
            d = t + u < tl ? d * (sg * fmaf(z, 1.f - sg, 1.f)) : 0.f;
          }
          dz[W - 1 + u][i] = d;
          if (mine) {
            db[i] += d;
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][i] = fmaf(d, buf[u + j][i], dw[j][i]);
          }
          float v = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) v = fmaf(w[j][i], dz[W - 1 + u - j][i], v);
          o[i] = v;
        }
        const int e = t + u;
        if (e < e1) {
          if (a.dst && e >= p.len) {
            float q[VE];
            Rows<T, VE>::load((const T*)a.dst + ((size_t)p.n * (W - 1) + (e - p.len)) * f.D + c, q);
#pragma unroll
            for (int i = 0; i < VE; ++i) o[i] += q[i];
          }
          if (e >= p.t0 + W - 1) Rows<T, VE>::store(dx + (size_t)(e - (W - 1)) * f.D, o);
          else if (p.first && a.ds0) Rows<T, VE>::store((T*)a.ds0 + ((size_t)p.n * (W - 1) + e) * f.D + c, o);
        }
      }
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          buf[k][i] = buf[kBwdRows + k][i];
          dz[k][i] = dz[kBwdRows + k][i];
        }
    }
  }
  // sums over the strips of a wave that share channels, then over the waves
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      float v = j < W ? dw[j < W ? j : 0][i] : db[i];
      for (unsigned off = LC; off < 64; off <<= 1) v += __shfl_xor(v, (int)off);
      if ((unsigned)lane < LC) red[wave][(j * 64 + lane) * VE + i] = v;
    }
  __syncthreads();
  const unsigned cols = LC * VE;
  for (unsigned k = threadIdx.x; k < cols * (W + 1); k += kConvThreads) {
    const unsigned j = k / cols, cc = k - j * cols;
    const unsigned ch = cb * cols + cc;
    if (ch >= (unsigned)f.D) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kWaves; ++q) v += red[q][j * 64 * VE + cc];
    // a partial row is [dw as D x W, dbias as D]
    a.part[(size_t)grp * (W + 1) * f.D + (j < (unsigned)W ? (size_t)ch * W + j : (size_t)W * f.D + ch)] = v;
  }
}

// Four channels a thread where every row starts on the size of four elements
// (channels and the token stride a multiple of 4, all tensors aligned); one
// channel otherwise (16384 tokens x 4096 channels: 46 us; of rows 13 elements
// wider: 67).
bool on_four(const void* p, int is_bf16) { return reinterpret_cast<uintptr_t>(p) % (is_bf16 ? 8u : 16u) == 0; }
int vec_of(const ConvArgs& a, int is_bf16) {
  return a.D % 4 == 0 && a.ldx % 4 == 0 && on_four(a.x, is_bf16) && on_four(a.s0, is_bf16) && on_four(a.st, is_bf16) &&
                 on_four(a.y, is_bf16)
             ? 4
             : 1;
}
int vec_of(const ConvBwdArgs& a, int is_bf16) {
  return on_four(a.dy, a.dy_bf16) && on_four(a.dst, is_bf16) && on_four(a.dx, is_bf16) && on_four(a.ds0, is_bf16) ? vec_of(a.f, is_bf16)
                                                                                                              : 1;
}

// Tokens of a strip: long strips re-read fewer rows, short ones keep the card
// busy on short inputs.  Forward at most 128 (64K tokens x 4096 channels: 203
// us; 64 209), fewer below 256K threads (16384 x 4096: 46 us; 512K 55, 128K 54).
// Backward at most 64 (32K x 2048: 115 us; 32 120, 128 152), fewer below 128K
// threads (4096 x 4352: 42 us; 64K 62, 256K 46).
int fwd_strip(long long rows, int cg) {
  int part = 128;
  while (part > kFwdRows && rows * cg / part < 256LL * 1024) part >>= 1;
  return part;
}
int bwd_strip(long long rows, int cg) {
  int part = 64;
  while (part > 8 && rows * cg / part < 256LL * 512) part >>= 1;
  return part;
}
unsigned pow2_lanes(unsigned cg) {
  unsigned l = 1;
  while (l < cg && l < 64) l <<= 1;
  return l;
}

template <typename T, int VE>
hipError_t fwd_go(const ConvArgs& a, const SeqTab& s, hipStream_t st) {
  const unsigned CG = (unsigned)(a.D / VE);
  const dim3 grid(((unsigned)s.items * CG + kConvThreads - 1) / kConvThreads);
  if (a.W == 2) hipLaunchKernelGGL((conv_fwd_kernel<T, 2, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG);
  else if (a.W == 3) hipLaunchKernelGGL((conv_fwd_kernel<T, 3, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG);
  else hipLaunchKernelGGL((conv_fwd_kernel<T, 4, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG);
  return hipGetLastError();
}
template <typename T, int VE>
hipError_t state_go(const ConvArgs& a, const SeqTab& s, hipStream_t st) {
  const unsigned CG = (unsigned)(a.D / VE);
  const dim3 grid(((unsigned)s.items * CG + kConvThreads - 1) / kConvThreads);
  hipLaunchKernelGGL((conv_state_kernel<T, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG);
  return hipGetLastError();
}
// Sequences of a token step's thread: more where enough threads are left (256
// x 4352 channels: two 4.5 us, one 4.9, four 4.5; 1024 x 4352: four 11.9, two
// 12.7, one 14.0; 64 x 4352: one 2.5, two 2.7).
template <typename T, int W>
hipError_t step_go(const ConvArgs& a, int B, hipStream_t st) {
  const long long all = (long long)B * a.D;
  const int S = all < (1 << 19) ? 1 : all < (1 << 21) ? 2 : 4;
  const long long n = ((long long)B + S - 1) / S * a.D;
  if (n > 0x7fffffffLL) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)((n + kConvThreads - 1) / kConvThreads)), th(kConvThreads);
  if (S == 1) hipLaunchKernelGGL((conv_step_kernel<T, W, 1>), grid, th, 0, st, a, (unsigned)B);
  else if (S == 2) hipLaunchKernelGGL((conv_step_kernel<T, W, 2>), grid, th, 0, st, a, (unsigned)B);
  else hipLaunchKernelGGL((conv_step_kernel<T, W, 4>), grid, th, 0, st, a, (unsigned)B);
  return hipGetLastError();
}
template <typename T>
hipError_t step_type(const ConvArgs& a, int B, hipStream_t st) {
  return a.W == 2 ? step_go<T, 2>(a, B, st) : a.W == 3 ? step_go<T, 3>(a, B, st) : step_go<T, 4>(a, B, st);
}
// Work-groups along the items of a launch (partial rows it writes).
unsigned bwd_groups(unsigned items, unsigned LC) {
  const unsigned per = 64u / LC * (kConvThreads / 64);
  return (items + per - 1) / per;
}
template <typename T, typename TG, int VE>
hipError_t bwd_go(const ConvBwdArgs& a, const SeqTab& s, unsigned* rows, hipStream_t st) {
  const unsigned CG = (unsigned)(a.f.D / VE), LC = pow2_lanes(CG), cb = (CG + LC - 1) / LC;
  const unsigned ng = bwd_groups((unsigned)s.items, LC);
  const dim3 grid(ng * cb);
  if (a.f.W == 2) hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 2, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG, LC, cb);
  else if (a.f.W == 3) hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 3, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG, LC, cb);
  else hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 4, VE>), grid, dim3(kConvThreads), 0, st, a, s, CG, LC, cb);
  *rows = ng;
  return hipGetLastError();
}

}  // namespace

int make_seq_tab(SeqTab& s, const int* cu, int N, int n0, int B, int T, int part) {
  s.n0 = n0;
  s.T = T;
  s.part = part;
  s.chunks = (T + kSeqChunk - 1) / kSeqChunk;
  if (!cu) {
    s.n = 0;
    s.parts = (T + part - 1) / part;
    s.items = B * s.parts;
    return B;
  }
  s.n = N - n0 < kMaxVarSeq ? N - n0 : kMaxVarSeq;
  s.parts = 0;
  long long items = 0, chunks = 0;
  for (int i = 0; i <= s.n; ++i) {
    s.cu[i] = cu[n0 + i];
    s.cc[i] = (int)items;
    s.cb[i] = (int)chunks;
    if (i == s.n) break;
    const long long len = cu[n0 + i + 1] - cu[n0 + i];
    items += len > 0 ? (len + part - 1) / part : 1;
    chunks += len > 0 ? (len + kSeqChunk - 1) / kSeqChunk : 1;
  }
  s.items = (int)items;
  return n0 + s.n;
}

bool seq_tabs_fit(const int* cu, int N, int B, int T, int part, long long most) {
  if (!cu) return (long long)B * ((T + part - 1) / part) <= most;
  if ((long long)T / part + N <= most) return true;
  for (int n = 0; n < N;) {
    long long items = 0;
    for (const int end = N - n < kMaxVarSeq ? N : n + kMaxVarSeq; n < end; ++n) {
      const long long len = cu[n + 1] - cu[n];
      items += len > 0 ? (len + part - 1) / part : 1;
    }
    if (items > most) return false;
  }
  return true;
}

constexpr int kSumThreads = 1024;
// out[c]: sum of column c of part [nrows][n0 + n1 + n2] over its rows, the
// columns in three outputs.  A work-group takes 64 columns; its 16 waves take
// every 16th row and are joined through LDS, always in the same order.
__global__ __launch_bounds__(kSumThreads) void sum_rows_kernel(const float* __restrict__ part, size_t nrows, unsigned n0, unsigned n1,
                                                        unsigned n2, float* __restrict__ out0, float* __restrict__ out1,
                                                        float* __restrict__ out2) {
  __shared__ double red[16][64];
  const unsigned l = threadIdx.x & 63, q = threadIdx.x >> 6, col = blockIdx.x * 64 + l, cols = n0 + n1 + n2;
  double v = 0.0;
  if (col < cols)
#pragma unroll 8
    for (size_t r = q; r < nrows; r += 16) v += (double)part[r * cols + col];
  red[q][l] = v;
  __syncthreads();
  if (q != 0 || col >= cols) return;
  v = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += red[k][l];
  float* out = col < n0 ? out0 : col < n0 + n1 ? out1 : out2;
  if (out) out[col - (col < n0 ? 0 : col < n0 + n1 ? n0 : n0 + n1)] = (float)v;
}

hipError_t launch_sum_rows(const float* part, size_t nrows, unsigned n0, unsigned n1, unsigned n2, float* out0, float* out1,
                           float* out2, hipStream_t st) {
  hipLaunchKernelGGL(sum_rows_kernel, dim3((n0 + n1 + n2 + 63) / 64), dim3(kSumThreads), 0, st, part, nrows, n0, n1, n2, out0, out1, out2);
  return hipGetLastError();
}

hipError_t launch_conv_fwd(int is_bf16, const ConvArgs& a, const int* cu, int N, int B, int T, hipStream_t st) {
  const int ve = vec_of(a, is_bf16), part = fwd_strip((long long)B * T, a.D / ve), end = cu ? N : B;
  if (!seq_tabs_fit(cu, N, B, T, part, 0x7fffffffLL / (a.D / ve))) return hipErrorInvalidConfiguration;
  // a state replaced in place is written by a launch of its own where another
  // strip still has to read the old one
  const bool later = a.st && a.st == a.s0 && T > part;
  for (int pass = 0; pass < (later ? 2 : 1); ++pass) {
    ConvArgs b = a;
    if (later && pass == 0) b.st = nullptr;
    for (int n = 0; n < end;) {
      SeqTab s;
      n = make_seq_tab(s, cu, N, n, B, T, pass ? T : part);
      hipError_t e;
      if (pass) {
        if (is_bf16) e = ve == 4 ? state_go<bf16, 4>(b, s, st) : state_go<bf16, 1>(b, s, st);
        else e = ve == 4 ? state_go<float, 4>(b, s, st) : state_go<float, 1>(b, s, st);
      } else {
        if (is_bf16) e = ve == 4 ? fwd_go<bf16, 4>(b, s, st) : fwd_go<bf16, 1>(b, s, st);
        else e = ve == 4 ? fwd_go<float, 4>(b, s, st) : fwd_go<float, 1>(b, s, st);
      }
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t launch_conv_step(int is_bf16, const ConvArgs& a, int B, hipStream_t st) {
  return is_bf16 ? step_type<bf16>(a, B, st) : step_type<float>(a, B, st);
}

size_t conv_bwd_workspace_bytes(int is_packed, int N, int B, int T, int D, int W) {
  // the larger of the two channel widths' needs: strides and alignment decide at the call
  size_t most = 0;
  for (int ve : {4, 1}) {
    if (D % ve) continue;
    const int cg = D / ve, part = bwd_strip((long long)B * T, cg);
    const size_t items = (is_packed ? (size_t)T / part + N : (size_t)B * (((size_t)T + part - 1) / part));
    const unsigned LC = pow2_lanes((unsigned)cg);
    const size_t per = 64u / LC * (kConvThreads / 64);
    const size_t rows = items / per + 1 + (is_packed ? (size_t)N / kMaxVarSeq + 1 : 0);
    const size_t bytes = rows * (size_t)(W + 1) * D * sizeof(float);
    most = bytes > most ? bytes : most;
  }
  return (most + 255) & ~(size_t)255;
}

hipError_t launch_conv_bwd(int is_bf16, const ConvBwdArgs& a, const int* cu, int N, int B, int T, hipStream_t st) {
  const int ve = vec_of(a, is_bf16), part = bwd_strip((long long)B * T, a.f.D / ve), end = cu ? N : B;
  const unsigned CG = (unsigned)(a.f.D / ve), LC = pow2_lanes(CG), cb = (CG + LC - 1) / LC;
  if (!seq_tabs_fit(cu, N, B, T, part, max_groups(kConvThreads) / cb * (64 / LC * (kConvThreads / 64))) ||
      ((long long)a.f.D * (a.f.W + 1) + 63) / 64 > max_groups(kSumThreads))
    return hipErrorInvalidConfiguration;
  size_t rows = 0;
  for (int n = 0; n < end;) {
    SeqTab s;
    n = make_seq_tab(s, cu, N, n, B, T, part);
    ConvBwdArgs b = a;
    b.part = a.part + rows * (size_t)(a.f.W + 1) * a.f.D;
    unsigned r = 0;
    hipError_t e;
    if (!is_bf16) e = ve == 4 ? bwd_go<float, float, 4>(b, s, &r, st) : bwd_go<float, float, 1>(b, s, &r, st);
    else if (a.dy_bf16) e = ve == 4 ? bwd_go<bf16, bf16, 4>(b, s, &r, st) : bwd_go<bf16, bf16, 1>(b, s, &r, st);
    else e = ve == 4 ? bwd_go<bf16, float, 4>(b, s, &r, st) : bwd_go<bf16, float, 1>(b, s, &r, st);
    if (e != hipSuccess) return e;
    rows += r;
  }
  return launch_sum_rows(a.part, rows, (unsigned)(a.f.W * a.f.D), (unsigned)a.f.D, 0, a.dw, a.dbias, nullptr, st);
}

}  // namespace kda
