// Gated linear recurrence with one state a channel (kda_lru_dev.h has the
// formulas): prompts, packed prompts, single tokens.
//
// A wave holds R tokens of 64 NC channels in registers, a work-group kWaves
// runs of them, one behind the other: a part of a sequence.  Its (P, H) are
// joined over the waves in LDS.  Every input is read once: the parts of a
// sequence hand their states on inside the one launch.
//
// Bound by HBM: 65536 x 4096 bf16 416 us (8 bytes an element, 5.2 TB/s), 8191
// packed tokens x 4096 fp32 119 us (4.5 TB/s); a token for each of 256 x 4096
// channels is bound by the launch, few channels by the hops from part to part.
// The tile: runs of 8, 24 or 32 tokens, 4 or 16 waves, four channels a lane, a look
// back over 2 or 8 parts were all slower or the same; so were a work-group for all
// parts of a short sequence (4 parts 27 us, a chain of parts 15).
#include "kda_lru_dev.h"

namespace kda {

namespace {

constexpr int kWaves = 8, kR = 16, kPart = kWaves * kR;
constexpr int kBack = 4;   // parts that a wave looks back over
constexpr int kPolls = 1 << 21;   // of a wait, a few seconds

// a and u of a wave's run of R tokens from token t on (the same for all
// lanes); tokens past the part's end leave the state as it is.
template <typename T, int NC, int R, bool kFull>
__device__ __forceinline__ void load_run(const LruArgs& g, const SeqPart& p, const LruLane& l, int t, float (&a)[R][NC], float (&u)[R][NC]) {
  typedef LruPack<T, NC> Pk;
  const int n = p.t1 - t;
  if (n <= 0) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        a[k][j] = 1.f;
        u[k][j] = 0.f;
      }
    return;
  }
  float c[NC];
  lru_coef<NC>(g, l, c);
  Pk x[R], r[R], i[R];
  const size_t row = p.start + (size_t)t;
  const T *px = (const T*)g.x + row * (size_t)g.ldx, *pr = (const T*)g.r + row * (size_t)g.ldr, *pi = (const T*)g.i + row * (size_t)g.ldi;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int q = min(k, n - 1);
    x[k] = *reinterpret_cast<const Pk*>(px + q * g.ldx + l.cl);
    r[k] = *reinterpret_cast<const Pk*>(pr + q * g.ldr + l.cl);
  }
  if (kFull || g.i)
#pragma unroll
    for (int k = 0; k < R; ++k) i[k] = *reinterpret_cast<const Pk*>(pi + min(k, n - 1) * g.ldi + l.cl);
  const LruMode md = lru_mode<kFull>(g);
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int j = 0; j < NC; ++j)
      lru_gate<T>(md, c[j], x[k].at(j), r[k].at(j), md.igate ? i[k].at(j) : 0.f, a[k][j], u[k][j]);
  if (n < R)
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (k >= n)
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          a[k][j] = 1.f;
          u[k][j] = 0.f;
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

// What a part hands to the parts behind it, a word pair or word a channel in
// the workspace: `own` its (P, H), `into` the state behind it.  A word is valid
// once it is not all ones (a fill that every call does first), so that a word is
// its own flag: relaxed accesses at device scope are enough, and nothing is
// ordered by fences, which would write back the caches.
struct Words {
  unsigned* ticket;             // parts and slices given out so far
  unsigned* status;             // not 0: a wait of this call has expired (kda_fwd_status)
  unsigned long long* own;      // [items][D]
  unsigned* into;               // [items][D]
};
constexpr unsigned kNone = 0xffffffffu;
// Bits of x as a word: a NaN of all ones becomes the usual one.
__device__ __forceinline__ unsigned word_of(float x) {
  const unsigned b = __float_as_uint(x);
  return b == kNone ? 0x7fc00000u : b;
}
__device__ __forceinline__ Words words_at(void* ws, size_t n) {
  Words w;
  w.ticket = static_cast<unsigned*>(ws);
  w.status = w.ticket + 8;
  w.own = reinterpret_cast<unsigned long long*>(w.ticket + 64);
  w.into = reinterpret_cast<unsigned*>(w.own + n);
  return w;
}
// `begin`: a call's first launch, which clears the status.
__global__ __launch_bounds__(256) void lru_fill_kernel(unsigned* ws, size_t n, int begin) {   // n words of ones behind the ticket
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x, step = (size_t)gridDim.x * 256;
  if (id == 0) {
    ws[0] = 0;
    if (begin) ws[8] = 0;
  }
  for (size_t q = id; q < n / 4; q += step) reinterpret_cast<u32x4*>(ws + 64)[q] = u32x4{kNone, kNone, kNone, kNone};
  if (id < n % 4) ws[64 + n / 4 * 4 + id] = kNone;
}

// How a part gets the state in front of it.
//   kOne: every sequence is one part
//   kNear, kFar: it looks back over kBack parts, or its waves over kBack each
enum LruWay { kOne, kNear, kFar };

// What the parts d0 + 1 .. d0 + kBack before a part have published (bit d of the
// result: part d0 + d + 1 its state; bit 8 + d: its own P and H).
template <int NC> struct LruBack {
  unsigned in[kBack][NC];
  unsigned long long own[kBack][NC];
};
template <int NC> __device__ __forceinline__ unsigned look_back(const Words& w, size_t at, int D, int parts_before, int d0, bool live, LruBack<NC>& b) {
#pragma unroll
  for (int d = 0; d < kBack; ++d) {
    const size_t from = at - (size_t)min(d0 + d + 1, parts_before) * D;   // (the first part publishes its state only)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      b.in[d][j] = __hip_atomic_load(w.into + from + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      b.own[d][j] = __hip_atomic_load(w.own + from + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  unsigned bits = 0;
#pragma unroll
  for (int d = 0; d < kBack; ++d) {
    bool got = true, has = true;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      got &= b.in[d][j] != kNone;
      has &= b.own[d][j] != ~0ull;
    }
    bits |= (__all(got || !live) ? 1u << d : 0u) | (__all(has || !live) ? 256u << d : 0u);
  }
  return bits;
}
// How many parts back the nearest state is, if the parts in between have their
// own P and H there (else 0).
__device__ __forceinline__ int found_back(unsigned got, unsigned has) {
  if (!got) return 0;
  const int d = __builtin_ctz(got);
  const unsigned between = (1u << d) - 1;
  return (has & between) == between ? d + 1 : 0;
}
// The state behind a part with own (P, H) from that in front of it.
__device__ __forceinline__ float carry_over(unsigned long long own, float h) {
  return fmaf(__uint_as_float((unsigned)own), h, __uint_as_float((unsigned)(own >> 32)));
}

__device__ __forceinline__ void expired(const Words& w, int lane) {
  if (lane == 0) __hip_atomic_store(w.status, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Outputs.  kNear and kFar: each work-group takes the next (part, slice) by a
// ticket and waits for parts before its own only, all of which have lower
// tickets: the lowest ticket that is not done waits for nothing, so every wait
// ends, however many work-groups run at once.  A part publishes its own (P, H),
// goes back to the nearest part that has its state published, if the (P, H) of
// those in between are, and carries the state over them one by one, as each of
// them does, so that the bits do not depend on which was found.  A wait is bounded
// all the same: the states behind one that expires are NaN, and the status says so.
template <typename T, int NC, LruWay kWay, bool kFull>
__global__ __launch_bounds__(64 * kWaves, 4) void lru_out_kernel(const LruArgs g, const SeqTab s, unsigned slices, void* ws, int begin) {
  constexpr bool kChain = kWay == kNear || kWay == kFar;
  __shared__ float red[2][kWaves][64 * NC];
  __shared__ float carry[64 * NC];
  __shared__ unsigned given;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  unsigned id = blockIdx.x;
  const Words w = words_at(ws, (size_t)s.items * g.D);
  if (kChain) {
    if (threadIdx.x == 0) given = __hip_atomic_fetch_add(w.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(given);
    if (id >= gridDim.x) return;
  } else if (begin && blockIdx.x == 0 && threadIdx.x == 0) {
    *w.status = 0;
  }
  unsigned item = id / slices;
  const LruLane l = lru_lane<NC>((int)(id - item * slices), g.D);
  // (equal sequences take turns, so that their chains run side by side)
  if (kChain && s.n == 0) item = item % (unsigned)(s.items / s.parts) * s.parts + item / (unsigned)(s.items / s.parts);
  const SeqPart p = seq_part(s, (int)item);
  float a[kR][NC], u[kR][NC], P[NC], H[NC], h[NC];
  load_run<T, NC, kR, kFull>(g, p, l, p.t0 + wave * kR, a, u);
  run_sum<NC, kR>(a, u, P, H);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    red[0][wave][lane * NC + j] = P[j];
    red[1][wave][lane * NC + j] = H[j];
  }
  __syncthreads();
  const size_t at = (size_t)item * g.D + l.cl;
  if (wave == 0) {
#pragma unroll
    for (int q = 1; q < kWaves; ++q)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float f = red[0][q][lane * NC + j];
        H[j] = fmaf(f, H[j], red[1][q][lane * NC + j]);
        P[j] *= f;
      }
    if (kChain && !p.first && !p.last && l.live)
#pragma unroll
      for (int j = 0; j < NC; ++j)
        __hip_atomic_store(w.own + at + j, (unsigned long long)word_of(H[j]) << 32 | word_of(P[j]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (kWay == kOne || p.first) {
#pragma unroll
    for (int j = 0; j < NC; ++j) h[j] = g.h0 ? g.h0[(size_t)p.n * g.D + l.cl + j] : 0.f;
  } else if (kWay == kNear) {
    if (wave == 0) {
      LruBack<NC> b;
      int found = 0;
      for (int poll = 0;; ++poll) {
        const unsigned bits = look_back<NC>(w, at, g.D, p.t0 / kPart, 0, l.live, b);
        found = found_back(bits & 255, bits >> 8);
        if (found || poll == kPolls) break;
        __builtin_amdgcn_s_sleep(1);
      }
      if (!found) {
        expired(w, lane);
#pragma unroll
        for (int j = 0; j < NC; ++j) h[j] = __builtin_nanf("");
      }
#pragma unroll
      for (int d = kBack - 1; d >= 0; --d)
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          if (d + 1 == found) h[j] = __uint_as_float(b.in[d][j]);
          else if (d + 1 < found) h[j] = carry_over(b.own[d][j], h[j]);
        }
    }
  } else if (kWay == kFar) {
    __shared__ unsigned long long far[kWaves * kBack][64 * NC];
    __shared__ unsigned seen[2][kWaves];
    LruBack<NC> b;
    int found = 0;
    for (int poll = 0;; ++poll) {   // (two sets of bits by turns: one barrier a poll is enough)
      const unsigned bits = look_back<NC>(w, at, g.D, p.t0 / kPart, wave * kBack, l.live, b);
      if (lane == 0) seen[poll & 1][wave] = bits;
      __syncthreads();
      unsigned got = 0, has = 0;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) {
        const unsigned m = __builtin_amdgcn_readfirstlane(seen[poll & 1][q]);
        got |= (m & 255) << (q * kBack);
        has |= (m >> 8) << (q * kBack);
      }
      found = found_back(got, has);
      if (found || poll == kPolls) break;
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int d = 0; d < kBack; ++d)
      if (wave * kBack + d < found)
#pragma unroll
        for (int j = 0; j < NC; ++j) far[wave * kBack + d][lane * NC + j] = wave * kBack + d + 1 == found ? b.in[d][j] : b.own[d][j];
    __syncthreads();
    if (wave == 0) {
      if (!found) expired(w, lane);
#pragma unroll
      for (int j = 0; j < NC; ++j) h[j] = found ? __uint_as_float((unsigned)far[max(found, 1) - 1][lane * NC + j]) : __builtin_nanf("");
#pragma unroll 4
      for (int d = found - 2; d >= 0; --d)
#pragma unroll
        for (int j = 0; j < NC; ++j) h[j] = carry_over(far[d][lane * NC + j], h[j]);
    }
  }
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      carry[lane * NC + j] = h[j];
      const float behind = fmaf(P[j], h[j], H[j]);
      if (!l.live) continue;
      if (kChain && !p.last)
        __hip_atomic_store(w.into + (size_t)item * g.D + l.c + j, word_of(behind), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (p.last && g.ht) g.ht[(size_t)p.n * g.D + l.c + j] = behind;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NC; ++j) h[j] = carry[lane * NC + j];
  for (int q = 0; q < wave; ++q)
#pragma unroll
    for (int j = 0; j < NC; ++j) h[j] = fmaf(red[0][q][lane * NC + j], h[j], red[1][q][lane * NC + j]);
  const int t = p.t0 + wave * kR;
  T* y = (T*)g.y + (p.start + (size_t)t) * g.D;
#pragma unroll
  for (int k = 0; k < kR; ++k) {
    LruPack<T, NC> o;
#pragma unroll
    for (int j = 0; j < NC; ++j) h[j] = fmaf(a[k][j], h[j], u[k][j]);
    o.set(h);
    if (l.live && t + k < p.t1) *reinterpret_cast<LruPack<T, NC>*>(y + (long long)k * g.D + l.c) = o;
  }
}

// One token per sequence.
template <typename T, int NC>
__global__ __launch_bounds__(256) void lru_step_kernel(const LruArgs g, unsigned B, unsigned CG) {
  const unsigned id = blockIdx.x * 256 + threadIdx.x, n = id / CG;
  if (n >= B) return;
  const int ch = (int)(id - n * CG) * NC;
  typedef LruPack<T, NC> Pk;
  float c[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) c[j] = g.c ? g.c[ch + j] : 0.f;
  Pk x, r, i, o;
  x = *reinterpret_cast<const Pk*>((const T*)g.x + n * (size_t)g.ldx + ch);
  r = *reinterpret_cast<const Pk*>((const T*)g.r + n * (size_t)g.ldr + ch);
  i = x;
  if (g.i) i = *reinterpret_cast<const Pk*>((const T*)g.i + n * (size_t)g.ldi + ch);
  const size_t at = (size_t)n * g.D + ch;
  const LruPack<float, NC> h0 = *reinterpret_cast<const LruPack<float, NC>*>(g.h0 + at);
  LruPack<float, NC> ht;
  const LruMode md = lru_mode<false>(g);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float a, u;
    lru_gate<T>(md, c[j], x.at(j), r.at(j), i.at(j), a, u);
    ht.v[j] = fmaf(a, h0.v[j], u);
  }
  o.set(ht.v);
  *reinterpret_cast<Pk*>((T*)g.y + at) = o;
  *reinterpret_cast<LruPack<float, NC>*>(g.ht + at) = ht;
}

// Whether rows and states may be read and written two channels at a time.
bool pairs(const LruArgs& a, size_t esz) {
  if (a.D % 2 || a.ldx % 2 || a.ldr % 2 || (a.i && a.ldi % 2) || reinterpret_cast<uintptr_t>(a.h0) % 8 || reinterpret_cast<uintptr_t>(a.ht) % 8)
    return false;
  for (const void* p : {a.x, a.r, a.i, (const void*)a.y})
    if (reinterpret_cast<uintptr_t>(p) % (2 * esz)) return false;
  return true;
}

template <typename T, int NC, bool kFull>
hipError_t fwd_go(const LruArgs& a, const int* cu, int N, int B, int T_, void* ws, hipStream_t st) {
  const unsigned slices = (unsigned)((a.D + 64 * NC - 1) / (64 * NC));
  if (!seq_tabs_fit(cu, N, B, T_, kPart, max_groups(64 * kWaves) / slices)) return hipErrorInvalidConfiguration;
  const int end = cu ? N : B;
  for (int n = 0; n < end;) {
    SeqTab s;
    const int begin = n == 0;
    n = make_seq_tab(s, cu, N, n, B, T_, kPart);
    const unsigned seqs = (unsigned)(s.n ? s.n : B);
    const dim3 grid((unsigned)s.items * slices), th(64 * kWaves);
    if ((unsigned)s.items == seqs) {   // no sequence has a second part
      hipLaunchKernelGGL((lru_out_kernel<T, NC, kOne, kFull>), grid, th, 0, st, a, s, slices, ws, begin);
    } else {
      const size_t words = (size_t)s.items * a.D * 3, groups = (words + 1023) / 1024;
      hipLaunchKernelGGL(lru_fill_kernel, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, st, static_cast<unsigned*>(ws), words, begin);
      // Few chains at once wait for their states, hop by hop (65536 tokens of 512
      // channels: 87 us by kFar, 167 by kNear; 1024: 157 and 180); with many the
      // words read count (2048: 269 and 244; 4096: 492 and 425).
      if (seqs * slices <= 8) hipLaunchKernelGGL((lru_out_kernel<T, NC, kFar, kFull>), grid, th, 0, st, a, s, slices, ws, begin);
      else hipLaunchKernelGGL((lru_out_kernel<T, NC, kNear, kFull>), grid, th, 0, st, a, s, slices, ws, begin);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t fwd_type(const LruArgs& a, const int* cu, int N, int B, int T_, void* ws, hipStream_t st) {
  if (pairs(a, sizeof(T))) return lru_full(a) ? fwd_go<T, 2, true>(a, cu, N, B, T_, ws, st) : fwd_go<T, 2, false>(a, cu, N, B, T_, ws, st);
  return lru_full(a) ? fwd_go<T, 1, true>(a, cu, N, B, T_, ws, st) : fwd_go<T, 1, false>(a, cu, N, B, T_, ws, st);
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
  return (256 + items * 3 * D * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_lru_fwd(int is_bf16, const LruArgs& a, const int* cu, int N, int B, int T, void* workspace, hipStream_t st) {
  if (is_bf16) return fwd_type<bf16>(a, cu, N, B, T, workspace, st);
  return fwd_type<float>(a, cu, N, B, T, workspace, st);
}

hipError_t launch_lru_step(int is_bf16, const LruArgs& a, int B, hipStream_t st) {
  if (is_bf16) return pairs(a, 2) ? step_go<bf16, 2>(a, B, st) : step_go<bf16, 1>(a, B, st);
  return pairs(a, 4) ? step_go<float, 2>(a, B, st) : step_go<float, 1>(a, B, st);
}

}  // namespace kda
