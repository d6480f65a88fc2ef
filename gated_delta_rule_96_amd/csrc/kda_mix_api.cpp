// C ABI of the operators around the recurrence (declared in include/kda.h):
// short causal convolution, norms of query and key heads with the position
// rotation, state space scan.  Synchronous argument checks, then the launches on the caller's
// stream; nothing is allocated and no state is kept.
#include <hip/hip_runtime.h>

#include "kda_check.h"
#include "kda_launch.h"

using kda::aligned16;
using kda::elem_size;
using kda::overlap;
using kda::size_ok;
using kda::valid_dtype;

namespace {

constexpr int kMaxT = 1 << 30;
// Heads are numbered in 32 bits, up to a wave's 32 beyond the last one.
constexpr int kMaxHeads = 1 << 24;

// A span of memory an argument covers.
struct Span {
  const void* p;
  size_t n;
};
// Whether an output overlaps an input or another output; an output that
// starts where inputs[same] starts and covers the same bytes is that input
// replaced in place (same < 0: never).
template <int NI, int NO>
bool spans_apart(const Span (&in)[NI], const Span (&out)[NO], const int (&same)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i) {
      if (i == same[o] && in[i].p == out[o].p && in[i].n == out[o].n) continue;
      if (overlap(in[i].p, in[i].n, out[o].p, out[o].n)) return false;
    }
    for (int k = 0; k < o; ++k)
      if (overlap(out[k].p, out[k].n, out[o].p, out[o].n)) return false;
  }
  return true;
}
// Bytes from the first to the last element of `rows` rows of n elements, ld
// apart.
size_t rows_bytes(size_t rows, long long ld, size_t n, size_t esz) { return ((rows - 1) * (size_t)ld + n) * esz; }

int check_cu(const int* cu, int N, int B, int T) {
  if (!cu) return KDA_OK;
  if (B != 1 || N <= 0 || cu[0] != 0 || cu[N] != T) return KDA_ERR_SHAPE;
  for (int i = 0; i < N; ++i)
    if (cu[i + 1] < cu[i]) return KDA_ERR_SHAPE;
  return KDA_OK;
}

// (hipErrorInvalidConfiguration: sizes beyond a launch's, see max_groups)
int hip_status(hipError_t e) {
  return e == hipSuccess ? KDA_OK : e == hipErrorInvalidConfiguration ? KDA_ERR_SHAPE : KDA_ERR_HIP;
}

// Sizes and strides of the convolution's x.
int check_conv(const void* x, long long ldx, const float* w, const float* bias, int flags, int dtype, int B, int T, int D, int W) {
  if (!valid_dtype(dtype)) return KDA_ERR_DTYPE;
  if (B <= 0 || T <= 0 || T > kMaxT || D <= 0 || ldx < D || (flags & ~KDA_CONV_SILU) || !size_ok(B, T, ldx, 8))
    return KDA_ERR_SHAPE;
  if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
  if ((long long)D * (W + 1) > 0x7fffffffLL) return KDA_ERR_SHAPE;
  if (!x || !w) return KDA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(x) % elem_size(dtype) || !aligned16(w) || !aligned16(bias)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

// Tokens or states of D channels without gaps: from any element where rows of
// D are no whole 16 bytes.
bool conv_aligned(const void* p, int D, int dtype) {
  const size_t esz = elem_size(dtype);
  return reinterpret_cast<uintptr_t>(p) % ((size_t)D * esz % 16 == 0 ? 16 : esz) == 0;
}

}  // namespace

extern "C" {

int kda_conv_fwd(const void* x, long long ldx, const float* w, const float* bias, const void* s0, void* st, void* y, int flags,
                 int dtype, int B, int T, int D, int W, const int* cu_seqlens, int N, void* stream) {
  int e = check_conv(x, ldx, w, bias, flags, dtype, B, T, D, W);
  if (e != KDA_OK) return e;
  if (!y) return KDA_ERR_NULL;
  if (!conv_aligned(s0, D, dtype) || !conv_aligned(st, D, dtype) || !conv_aligned(y, D, dtype)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, ns = (size_t)(cu_seqlens ? N : B) * (W - 1) * D * esz;
  const Span in[] = {{x, rows_bytes(rows, ldx, D, esz)}, {s0, ns}, {w, (size_t)D * W * 4}, {bias, (size_t)D * 4}};
  const Span out[] = {{y, rows * D * esz}, {st, ns}};
  if (!spans_apart(in, out, {-1, 1})) return KDA_ERR_OVERLAP;
  const kda::ConvArgs a{x, ldx, w, bias, s0, st, y, flags & KDA_CONV_SILU, D, W};
  return hip_status(kda::launch_conv_fwd(dtype == KDA_BF16, a, cu_seqlens, N, B, T, static_cast<hipStream_t>(stream)));
}

int kda_conv_step(const void* x, long long ldx, const float* w, const float* bias, const void* state, void* state_out, void* y,
                  int flags, int dtype, int B, int D, int W, void* stream) {
  const int e = check_conv(x, ldx, w, bias, flags, dtype, B, 1, D, W);
  if (e != KDA_OK) return e;
  if (!state || !state_out || !y) return KDA_ERR_NULL;
  if (!conv_aligned(state, D, dtype) || !conv_aligned(state_out, D, dtype) || !conv_aligned(y, D, dtype)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), ns = (size_t)B * (W - 1) * D * esz;
  const Span in[] = {{x, rows_bytes(B, ldx, D, esz)}, {state, ns}, {w, (size_t)D * W * 4}, {bias, (size_t)D * 4}};
  const Span out[] = {{y, (size_t)B * D * esz}, {state_out, ns}};
  if (!spans_apart(in, out, {-1, 1})) return KDA_ERR_OVERLAP;
  const kda::ConvArgs a{x, ldx, w, bias, state, state_out, y, flags & KDA_CONV_SILU, D, W};
  return hip_status(kda::launch_conv_step(dtype == KDA_BF16, a, B, static_cast<hipStream_t>(stream)));
}

size_t kda_conv_bwd_workspace_bytes(int B, int T, int D, int W, int N) {
  if (B <= 0 || T <= 0 || T > kMaxT || D <= 0 || W < 2 || W > 4 || N < 0 || (N > 0 && B != 1) || !size_ok(B, T, D, 8) ||
      (long long)D * (W + 1) > 0x7fffffffLL)
    return 0;
  return kda::conv_bwd_workspace_bytes(N > 0, N, B, T, D, W);
}

int kda_conv_bwd(const void* x, long long ldx, const float* w, const float* bias, const void* s0, const void* dy, int dy_dtype,
                 const void* dst, void* dx, float* dw, float* dbias, void* ds0, int flags, int dtype, int B, int T, int D, int W,
                 const int* cu_seqlens, int N, void* workspace, size_t workspace_bytes, void* stream) {
  int e = check_conv(x, ldx, w, bias, flags, dtype, B, T, D, W);
  if (e != KDA_OK) return e;
  if (!valid_dtype(dy_dtype) || (dtype == KDA_F32 && dy_dtype != KDA_F32)) return KDA_ERR_DTYPE;
  if (!dy || !dx || !dw) return KDA_ERR_NULL;
  for (const void* p : {s0, dst, (const void*)dx, (const void*)ds0})
    if (!conv_aligned(p, D, dtype)) return KDA_ERR_ALIGN;
  if (!conv_aligned(dy, D, dy_dtype) || !aligned16(dw) || !aligned16(dbias)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  const size_t need = kda_conv_bwd_workspace_bytes(B, T, D, W, cu_seqlens ? N : 0);
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, ns = (size_t)(cu_seqlens ? N : B) * (W - 1) * D * esz;
  const Span in[] = {{x, rows_bytes(rows, ldx, D, esz)}, {s0, ns}, {w, (size_t)D * W * 4}, {bias, (size_t)D * 4},
                     {dy, rows * D * elem_size(dy_dtype)}, {dst, ns}};
  const Span out[] = {{dx, rows * D * esz}, {dw, (size_t)D * W * 4}, {dbias, (size_t)D * 4}, {ds0, ns}, {workspace, need}};
  if (!spans_apart(in, out, {-1, -1, -1, -1, -1})) return KDA_ERR_OVERLAP;
  const kda::ConvBwdArgs a{{x, ldx, w, bias, s0, nullptr, nullptr, flags & KDA_CONV_SILU, D, W}, dy, dy_dtype == KDA_BF16, dst, dx,
                           dw, dbias, ds0, static_cast<float*>(workspace)};
  return hip_status(kda::launch_conv_bwd(dtype == KDA_BF16, a, cu_seqlens, N, B, T, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int check_qk(const void* q, long long ldq, const void* k, long long ldk, const float* wq, const float* wk, const float* cos,
             const float* sin, const int* pos, int pos0, int n_pos, float eps, int flags, int dtype, int B, int T, int Hq, int Hk,
             int d, int rot) {
  if (!valid_dtype(dtype)) return KDA_ERR_DTYPE;
  if (B <= 0 || T <= 0 || T > kMaxT || Hq <= 0 || Hq > kMaxHeads || Hk < 0 || Hk > kMaxHeads || d <= 0 || rot < 0 || (flags & ~(KDA_QK_RMS | KDA_QK_INTERLEAVED)) ||
      !(eps >= 0.f) || !size_ok(B, T, (long long)Hq + Hk, 8LL * d) || (long long)B * T > (1LL << 40))
    return KDA_ERR_SHAPE;
  if (d % 8 || d > 512 || rot % 8 || rot > d) return KDA_ERR_UNSUPPORTED;
  if (ldq < (long long)Hq * d || (Hk && ldk < (long long)Hk * d) || !size_ok(B, T, ldq, 8) || (Hk && !size_ok(B, T, ldk, 8)))
    return KDA_ERR_SHAPE;
  if (!q || (Hk && !k) || (rot && (!cos || !sin))) return KDA_ERR_NULL;
  if (rot && (n_pos <= 0 || (!pos && (pos0 < 0 || (long long)pos0 + T > n_pos)))) return KDA_ERR_SHAPE;
  const size_t esz = elem_size(dtype);
  for (const void* p : {q, k, (const void*)wq, (const void*)wk, (const void*)cos, (const void*)sin})
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  if ((ldq * esz) % 16 || (Hk && (ldk * esz) % 16) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

kda::QkArgs qk_args(const void* q, long long ldq, const void* k, long long ldk, const float* wq, const float* wk, const float* cos,
                    const float* sin, const int* pos, int pos0, int n_pos, float eps, int flags, int B, int T, int Hq, int Hk, int d,
                    int rot) {
  kda::QkArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.ld[0] = ldq;
  a.ld[1] = ldk;
  a.w[0] = wq;
  a.w[1] = wk;
  a.H[0] = Hq;
  a.H[1] = Hk;
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  a.pos0 = pos0;
  a.n_pos = n_pos;
  a.rms = (flags & KDA_QK_RMS) != 0;
  a.inter = (flags & KDA_QK_INTERLEAVED) != 0;
  a.d = d;
  a.rot = rot;
  a.eps = eps;
  a.tokens = (long long)B * T;
  a.T = T;
  return a;
}

}  // namespace

extern "C" {

int kda_qk_norm_rope(const void* q, long long ldq, const void* k, long long ldk, const float* wq, const float* wk, const float* cos,
                     const float* sin, const int* pos, int pos0, int n_pos, float eps, void* q_out, void* k_out, int flags,
                     int dtype, int B, int T, int Hq, int Hk, int d, int rot, void* stream) {
  const int e = check_qk(q, ldq, k, ldk, wq, wk, cos, sin, pos, pos0, n_pos, eps, flags, dtype, B, T, Hq, Hk, d, rot);
  if (e != KDA_OK) return e;
  if (!q_out || (Hk && !k_out)) return KDA_ERR_NULL;
  if (!aligned16(q_out) || !aligned16(k_out)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, table = rot ? (size_t)n_pos * (rot / 2) * 4 : 0;
  const Span in[] = {{q, rows_bytes(rows, ldq, (size_t)Hq * d, esz)}, {k, Hk ? rows_bytes(rows, ldk, (size_t)Hk * d, esz) : 0},
                     {wq, (size_t)d * 4}, {wk, (size_t)d * 4}, {cos, table}, {sin, table}, {pos, rows * 4}};
  const Span out[] = {{q_out, rows * Hq * d * esz}, {k_out, rows * Hk * d * esz}};
  if (!spans_apart(in, out, {0, 1})) return KDA_ERR_OVERLAP;
  kda::QkArgs a = qk_args(q, ldq, k, ldk, wq, wk, cos, sin, pos, pos0, n_pos, eps, flags, B, T, Hq, Hk, d, rot);
  a.y[0] = q_out;
  a.y[1] = k_out;
  return hip_status(kda::launch_qk_fwd(dtype == KDA_BF16, a, static_cast<hipStream_t>(stream)));
}

size_t kda_qk_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d) {
  if (B <= 0 || T <= 0 || T > kMaxT || Hq <= 0 || Hq > kMaxHeads || Hk < 0 || Hk > kMaxHeads || d <= 0 || d % 8 || d > 512 ||
      !size_ok(B, T, (long long)Hq + Hk, 8LL * d) || (long long)B * T > (1LL << 40))
    return 0;
  return kda::qk_bwd_workspace_bytes((long long)B * T, Hq, Hk, d);
}

int kda_qk_norm_rope_bwd(const void* q, long long ldq, const void* k, long long ldk, const float* wq, const float* wk,
                         const float* cos, const float* sin, const int* pos, int pos0, int n_pos, float eps, const void* dq_out,
                         const void* dk_out, int dy_dtype, void* dq, void* dk, float* dwq, float* dwk, int flags, int dtype, int B,
                         int T, int Hq, int Hk, int d, int rot, void* workspace, size_t workspace_bytes, void* stream) {
  const int e = check_qk(q, ldq, k, ldk, wq, wk, cos, sin, pos, pos0, n_pos, eps, flags, dtype, B, T, Hq, Hk, d, rot);
  if (e != KDA_OK) return e;
  if (!valid_dtype(dy_dtype) || (dtype == KDA_F32 && dy_dtype != KDA_F32)) return KDA_ERR_DTYPE;
  if (!dq_out || !dq || (Hk && (!dk_out || !dk))) return KDA_ERR_NULL;
  for (const void* p : {dq_out, dk_out, (const void*)dq, (const void*)dk, (const void*)dwq, (const void*)dwk})
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  const size_t need = dwq || dwk ? kda_qk_bwd_workspace_bytes(B, T, Hq, Hk, d) : 0;
  if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), gsz = elem_size(dy_dtype), rows = (size_t)B * T, nq = rows * Hq * d, nk = rows * Hk * d;
  const size_t table = rot ? (size_t)n_pos * (rot / 2) * 4 : 0, nw = (size_t)d * 4;
  const Span in[] = {{q, rows_bytes(rows, ldq, (size_t)Hq * d, esz)}, {k, Hk ? rows_bytes(rows, ldk, (size_t)Hk * d, esz) : 0},
                     {wq, nw}, {wk, nw}, {cos, table}, {sin, table}, {pos, rows * 4}, {dq_out, nq * gsz}, {dk_out, nk * gsz}};
  const Span out[] = {{dq, nq * esz}, {dk, nk * esz}, {dwq, nw}, {dwk, nw}, {workspace, need}};
  if (!spans_apart(in, out, {-1, -1, -1, -1, -1})) return KDA_ERR_OVERLAP;
  kda::QkArgs a = qk_args(q, ldq, k, ldk, wq, wk, cos, sin, pos, pos0, n_pos, eps, flags, B, T, Hq, Hk, d, rot);
  a.y[0] = dq;
  a.y[1] = dk;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.part = static_cast<float*>(workspace);
  return hip_status(kda::launch_qk_bwd(dtype == KDA_BF16, dy_dtype == KDA_BF16, a, dwq, dwk, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// The scan's sizes, strides and inputs.
int check_ssm(const kda::SsmArgs& a, int flags, int dtype, int B, int T, int dk, int dv) {
  if (!valid_dtype(dtype)) return KDA_ERR_DTYPE;
  if (B <= 0 || T <= 0 || T > kMaxT || a.H <= 0 || a.G <= 0 || dk <= 0 || dv <= 0 || a.H % a.G || (flags & ~KDA_SSM_SOFTPLUS) ||
      !size_ok(B, T, a.H, 8LL * dv) || !size_ok(B, a.H, dk, 4LL * dv) || (long long)B * T > (1LL << 40) ||
      (long long)B * a.H > 0x7fffffffLL)
    return KDA_ERR_SHAPE;
  if (!kda::supported_d(dk) || !kda::supported_d(dv)) return KDA_ERR_UNSUPPORTED;
  if (a.ldx < (long long)a.H * dv || a.lddt < a.H || a.ldb < (long long)a.G * dk || a.ldc < (long long)a.G * dk) return KDA_ERR_SHAPE;
  for (long long ld : {a.ldx, a.lddt, a.ldb, a.ldc})   // 32-bit offsets within a few rows
    if (ld > (1 << 24) || !size_ok(B, T, ld, 8)) return KDA_ERR_SHAPE;
  if (!a.x || !a.dt || !a.A || !a.B || !a.C) return KDA_ERR_NULL;
  const size_t esz = elem_size(dtype);
  for (const void* p : {a.x, a.B, a.C, (const void*)a.A, (const void*)a.D, (const void*)a.bias, (const void*)a.h0})
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(a.dt) % esz || (a.ldx * esz) % 16 || (a.ldb * esz) % 16 || (a.ldc * esz) % 16) return KDA_ERR_ALIGN;
  return KDA_OK;
}
// The memory the scan's inputs cover.
struct SsmSpans {
  Span s[8];
};
SsmSpans ssm_spans(const kda::SsmArgs& a, size_t rows, size_t ns, int dk, int dv, size_t esz) {
  return SsmSpans{{{a.x, rows_bytes(rows, a.ldx, (size_t)a.H * dv, esz)}, {a.dt, rows_bytes(rows, a.lddt, a.H, esz)},
                   {a.B, rows_bytes(rows, a.ldb, (size_t)a.G * dk, esz)}, {a.C, rows_bytes(rows, a.ldc, (size_t)a.G * dk, esz)},
                   {a.A, (size_t)a.H * 4}, {a.D, (size_t)a.H * 4}, {a.bias, (size_t)a.H * 4}, {a.h0, ns}}};
}

}  // namespace

extern "C" {

size_t kda_ssm_workspace_bytes(int B, int T, int H, int dk, int dv, int dtype) {
  if (!valid_dtype(dtype) || B <= 0 || T <= 0 || T > kMaxT || H <= 0 || !kda::supported_d(dk) || !kda::supported_d(dv) ||
      !size_ok(B, T, H, 8LL * dv) || (long long)B * T > (1LL << 40))
    return 0;
  return kda::ssm_seg_bytes((long long)B * T, H, dk, dv);
}

int kda_ssm_fwd_chunked(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* Bm, long long ldb,
                        const void* Cm, long long ldc, const float* D, const float* dt_bias, const float* h0, float* ht, void* y,
                        int flags, int dtype, int B, int T, int H, int G, int dk, int dv, const int* cu_seqlens, int N,
                        void* workspace, size_t workspace_bytes, void* stream) {
  kda::SsmArgs a{};
  a.x = x, a.dt = dt, a.B = Bm, a.C = Cm;
  a.ldx = ldx, a.lddt = lddt, a.ldb = ldb, a.ldc = ldc;
  a.A = A, a.D = D, a.bias = dt_bias, a.h0 = h0, a.ht = ht, a.y = y;
  a.softplus = flags & KDA_SSM_SOFTPLUS, a.H = H, a.G = G;
  int e = check_ssm(a, flags, dtype, B, T, dk, dv);
  if (e != KDA_OK) return e;
  if (!y) return KDA_ERR_NULL;
  if (!aligned16(ht) || !aligned16(y)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  if (cu_seqlens && (long long)N * H > 0x7fffffffLL) return KDA_ERR_SHAPE;
  const size_t need = kda_ssm_workspace_bytes(B, T, H, dk, dv, dtype);
  if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, ns = (size_t)(cu_seqlens ? N : B) * H * dk * dv * 4;
  const SsmSpans in = ssm_spans(a, rows, ns, dk, dv, esz);
  const Span out[] = {{y, rows * H * dv * esz}, {ht, ns}, {workspace, need}};
  if (!spans_apart(in.s, out, {-1, 7, -1})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_ssm_fwd(dtype == KDA_BF16, a, dk, dv, cu_seqlens, N, B, T, workspace, static_cast<hipStream_t>(stream)));
}

int kda_ssm_step(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* Bm, long long ldb,
                 const void* Cm, long long ldc, const float* D, const float* dt_bias, const float* state, float* state_out, void* y,
                 int flags, int dtype, int B, int H, int G, int dk, int dv, void* stream) {
  kda::SsmArgs a{};
  a.x = x, a.dt = dt, a.B = Bm, a.C = Cm;
  a.ldx = ldx, a.lddt = lddt, a.ldb = ldb, a.ldc = ldc;
  a.A = A, a.D = D, a.bias = dt_bias, a.h0 = state, a.ht = state_out, a.y = y;
  a.softplus = flags & KDA_SSM_SOFTPLUS, a.H = H, a.G = G;
  const int e = check_ssm(a, flags, dtype, B, 1, dk, dv);
  if (e != KDA_OK) return e;
  if (!state || !state_out || !y) return KDA_ERR_NULL;
  if (!aligned16(state_out) || !aligned16(y)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rows = (size_t)B, ns = rows * H * dk * dv * 4;
  const SsmSpans in = ssm_spans(a, rows, ns, dk, dv, esz);
  const Span out[] = {{y, rows * H * dv * esz}, {state_out, ns}};
  if (!spans_apart(in.s, out, {-1, 7})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_ssm_step(dtype == KDA_BF16, a, dk, dv, B, static_cast<hipStream_t>(stream)));
}

size_t kda_ssm_bwd_workspace_bytes(int B, int T, int H, int G, int dk, int dv, int dtype, int N) {
  if (!valid_dtype(dtype) || B <= 0 || T <= 0 || T > kMaxT || H <= 0 || G <= 0 || H % G || !kda::supported_d(dk) ||
      !kda::supported_d(dv) || N < 0 || (N > 0 && B != 1) || !size_ok(B, T, H, 8LL * dk * dv) || (long long)B * T > (1LL << 40) ||
      (long long)N * H > 0x7fffffffLL)
    return 0;
  return kda::ssm_bwd_workspace_bytes(N > 0, N, B, T, H, G, dk, dv);
}

int kda_ssm_bwd_chunked(const void* x, long long ldx, const void* dt, long long lddt, const float* A, const void* Bm, long long ldb,
                        const void* Cm, long long ldc, const float* D, const float* dt_bias, const float* h0, const void* dy,
                        const float* dht, void* dx, void* ddt, float* dA, void* dBm, void* dCm, float* dD, float* ddt_bias,
                        float* dh0, int flags, int dtype, int B, int T, int H, int G, int dk, int dv, const int* cu_seqlens, int N,
                        void* workspace, size_t workspace_bytes, void* stream) {
  kda::SsmBwdArgs a{};
  kda::SsmArgs& f = a.f;
  f.x = x, f.dt = dt, f.B = Bm, f.C = Cm;
  f.ldx = ldx, f.lddt = lddt, f.ldb = ldb, f.ldc = ldc;
  f.A = A, f.D = D, f.bias = dt_bias, f.h0 = h0;
  f.softplus = flags & KDA_SSM_SOFTPLUS, f.H = H, f.G = G;
  a.dy = dy, a.dht = dht, a.dx = dx, a.ddt = ddt, a.dA = dA, a.dB = dBm, a.dC = dCm, a.dD = dD, a.dbias = ddt_bias, a.dh0 = dh0;
  int e = check_ssm(f, flags, dtype, B, T, dk, dv);
  if (e != KDA_OK) return e;
  if (!dy || !dx || !ddt || !dA || !dBm || !dCm) return KDA_ERR_NULL;
  for (const void* p : {dy, (const void*)dht, (const void*)dx, (const void*)ddt, (const void*)dA, (const void*)dBm, (const void*)dCm,
                        (const void*)dD, (const void*)ddt_bias, (const void*)dh0})
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  const size_t need = kda_ssm_bwd_workspace_bytes(B, T, H, G, dk, dv, dtype, cu_seqlens ? N : 0);
  if (need == 0) return KDA_ERR_SHAPE;
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, ns = (size_t)(cu_seqlens ? N : B) * H * dk * dv * 4;
  const size_t nv = rows * H * dv * esz, nk = rows * G * dk * esz, nh = (size_t)H * 4;
  const SsmSpans fs = ssm_spans(f, rows, ns, dk, dv, esz);
  const Span in[] = {fs.s[0], fs.s[1], fs.s[2], fs.s[3], fs.s[4], fs.s[5], fs.s[6], fs.s[7], {dy, nv}, {dht, ns}};
  const Span out[] = {{dx, nv}, {ddt, rows * H * esz}, {dA, nh}, {dBm, nk}, {dCm, nk}, {dD, nh}, {ddt_bias, nh}, {dh0, ns}, {workspace, need}};
  if (!spans_apart(in, out, {-1, -1, -1, -1, -1, -1, -1, -1, -1})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_ssm_bwd(dtype == KDA_BF16, a, dk, dv, cu_seqlens, N, B, T, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
