// C ABI of the operators of a recurrent block (declared in include/kda.h):
// norm of the residual stream, product of 8-bit rows and weights, gated linear
// recurrence.  Synchronous argument checks, then the launches on the caller's
// stream; nothing is allocated and no state is kept.
#include <hip/hip_runtime.h>

#include "kda_check.h"
#include "kda_launch.h"

using kda::aligned16;
using kda::check_cu;
using kda::elem_size;
using kda::hip_status;
using kda::kMaxT;
using kda::rows_bytes;
using kda::size_ok;
using kda::Span;
using kda::spans_apart;
using kda::valid_dtype;

namespace {

constexpr long long kMaxRows = 1LL << 40;
constexpr int kMaxNormD = 16384;
// Channels of the recurrence and outputs of the product are numbered in 32
// bits, a tile beyond the last.
constexpr int kMaxWidth = 1 << 30;
// Bytes between two rows of the product's operands, and scales between two
// rows': a tile of 256 rows is addressed in 32 bits.
constexpr int kMaxStride8 = 1 << 24, kMaxScaleStride = 1 << 20;

int check_norm(long long rows, int D, float eps) {
  if (rows <= 0 || rows > kMaxRows || D <= 0 || !(eps >= 0.f)) return KDA_ERR_SHAPE;
  return D % 8 || D > kMaxNormD ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

int check_rows(const void* p, long long ld, long long rows, int D, int dtype) {
  if (ld < D || !size_ok(rows, ld, 8, 1)) return KDA_ERR_SHAPE;
  if (!p) return KDA_ERR_NULL;
  return !aligned16(p) || (rows > 1 && (ld * elem_size(dtype)) % 16) ? KDA_ERR_ALIGN : KDA_OK;
}

}  // namespace

extern "C" {

int kda_add_rms_norm(const void* x, long long ldx, const void* res, long long ldr, int res_dtype, const float* w, float eps, void* sum,
                     void* y, float* scale, int dtype, long long rows, int D, void* stream) {
  if (!valid_dtype(dtype) || (res && (!valid_dtype(res_dtype) || (dtype == KDA_F32 && res_dtype != KDA_F32)))) return KDA_ERR_DTYPE;
  int e = check_norm(rows, D, eps);
  if (e != KDA_OK || (e = check_rows(x, ldx, rows, D, dtype)) != KDA_OK) return e;
  if (res && (e = check_rows(res, ldr, rows, D, res_dtype)) != KDA_OK) return e;
  if (!y || (res && !sum)) return KDA_ERR_NULL;
  if (!aligned16(w) || !aligned16(y) || !aligned16(sum) || !aligned16(scale)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), rsz = elem_size(res_dtype), n = (size_t)rows * D;
  const Span in[] = {{x, rows_bytes(rows, ldx, D, esz)}, {res, res ? rows_bytes(rows, ldr, D, rsz) : 0}, {w, (size_t)D * 4}};
  const Span out[] = {{sum, res ? n * rsz : 0}, {y, scale ? n : n * esz}, {scale, (size_t)rows * ((D + 127) / 128) * 4}};
  if (!spans_apart(in, out, {1, -1, -1})) return KDA_ERR_OVERLAP;
  const kda::NormArgs a{x, ldx, res, ldr, w, sum, y, scale, nullptr, nullptr, rows, D, eps};
  return hip_status(kda::launch_norm_fwd(dtype == KDA_BF16, res_dtype == KDA_BF16, a, static_cast<hipStream_t>(stream)));
}

size_t kda_add_rms_norm_bwd_workspace_bytes(long long rows, int D) {
  return check_norm(rows, D, 0.f) != KDA_OK || !size_ok(rows, D, 8, 1) ? 0 : kda::norm_bwd_workspace_bytes(rows, D);
}

int kda_add_rms_norm_bwd(const void* h, long long ldh, const float* w, float eps, const void* dy, int dy_dtype, const void* dh, void* dx,
                         float* dw, int dtype, long long rows, int D, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(dy_dtype)) return KDA_ERR_DTYPE;
  int e = check_norm(rows, D, eps);
  if (e != KDA_OK || (e = check_rows(h, ldh, rows, D, dtype)) != KDA_OK) return e;
  if (!dy || !dx) return KDA_ERR_NULL;
  for (const void* p : {(const void*)w, dy, dh, (const void*)dx, (const void*)dw})
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  const size_t need = dw ? kda_add_rms_norm_bwd_workspace_bytes(rows, D) : 0;
  if (need && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return KDA_ERR_ALIGN;
  const size_t esz = elem_size(dtype), n = (size_t)rows * D;
  const Span in[] = {{h, rows_bytes(rows, ldh, D, esz)}, {w, (size_t)D * 4}, {dy, n * elem_size(dy_dtype)}, {dh, n * esz}};
  const Span out[] = {{dx, n * esz}, {dw, (size_t)D * 4}, {need ? workspace : nullptr, need}};
  if (!spans_apart(in, out, {3, -1, -1})) return KDA_ERR_OVERLAP;
  const kda::NormArgs a{h, ldh, dh, D, w, nullptr, dx, nullptr, dy, dw ? static_cast<float*>(workspace) : nullptr, rows, D, eps};
  return hip_status(kda::launch_norm_bwd(dtype == KDA_BF16, dy_dtype == KDA_BF16, a, dw, static_cast<hipStream_t>(stream)));
}

int kda_gemm_fp8(const void* a, long long lda, const float* sa, long long lsa, const void* w, const float* sw, void* c, int c_dtype,
                 long long M, int N, int K, void* stream) {
  if (!valid_dtype(c_dtype)) return KDA_ERR_DTYPE;
  if (M <= 0 || M > kMaxRows || N <= 0 || N > kMaxWidth || K <= 0 || K > kMaxStride8 || lda > kMaxStride8) return KDA_ERR_SHAPE;
  if (K % 16) return KDA_ERR_UNSUPPORTED;
  const int KB = (K + 127) / 128;
  if (lda < K || lsa < KB || lsa > kMaxScaleStride || !size_ok(M, lda, 8, 1) || !size_ok(M, lsa, 8, 1) || !size_ok(M, N, 8, 1)) return KDA_ERR_SHAPE;
  if (!a || !sa || !w || !sw || !c) return KDA_ERR_NULL;
  if (!aligned16(a) || (M > 1 && lda % 16) || !aligned16(w) || !aligned16(c)) return KDA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(sa) & 3u) || (reinterpret_cast<uintptr_t>(sw) & 3u)) return KDA_ERR_ALIGN;
  const Span in[] = {{a, rows_bytes(M, lda, K, 1)}, {sa, rows_bytes(M, lsa, KB, 4)}, {w, (size_t)N * K}, {sw, (size_t)((N + 127) / 128) * KB * 4}};
  const Span out[] = {{c, (size_t)M * N * elem_size(c_dtype)}};
  if (!spans_apart(in, out, {-1})) return KDA_ERR_OVERLAP;
  const kda::Gemm8Args g{static_cast<const unsigned char*>(a), lda, sa, lsa, static_cast<const unsigned char*>(w), sw, c, M, N, N, K};
  return hip_status(kda::launch_gemm8(c_dtype == KDA_BF16, g, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int check_lru(const kda::LruArgs& a, int flags, int dtype, int B, int T) {
  if (!valid_dtype(dtype)) return KDA_ERR_DTYPE;
  if (B <= 0 || T <= 0 || T > kMaxT || a.D <= 0 || a.D > kMaxWidth || (flags & ~KDA_LRU_UNIT) || (long long)B * T > kMaxRows) return KDA_ERR_SHAPE;
  if (a.ldx < a.D || a.ldr < a.D || (a.i && a.ldi < a.D) || !size_ok(B, T, a.ldx, 8) || !size_ok(B, T, a.ldr, 8) || (a.i && !size_ok(B, T, a.ldi, 8)))
    return KDA_ERR_SHAPE;
  if (!a.x || !a.r) return KDA_ERR_NULL;
  const size_t esz = elem_size(dtype);
  for (const void* p : {a.x, a.r, a.i})
    if (reinterpret_cast<uintptr_t>(p) % esz) return KDA_ERR_ALIGN;
  return aligned16(a.c) ? KDA_OK : KDA_ERR_ALIGN;
}

// Tokens or states of D channels without gaps: from any element where rows of
// D are no whole 16 bytes.
bool dense_aligned(const void* p, int D, size_t esz) { return reinterpret_cast<uintptr_t>(p) % ((size_t)D * esz % 16 == 0 ? 16 : esz) == 0; }

}  // namespace

extern "C" {

size_t kda_lru_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T <= 0 || T > kMaxT || D <= 0 || D > kMaxWidth || N < 0 || (N > 0 && B != 1) || (long long)B * T > kMaxRows || !size_ok(B, T, D, 8) ||
      !size_ok(N ? N : B, D, 16, 1))
    return 0;
  return kda::lru_workspace_bytes(N > 0, N, B, T, D);
}

int kda_lru_fwd(const void* x, long long ldx, const void* r, long long ldr, const void* i, long long ldi, const float* c, const float* h0,
                float* ht, void* y, int flags, int dtype, int B, int T, int D, const int* cu_seqlens, int N, void* workspace,
                size_t workspace_bytes, void* stream) {
  const kda::LruArgs a{x, r, i, ldx, ldr, ldi, c, h0, ht, y, flags & KDA_LRU_UNIT, D};
  int e = check_lru(a, flags, dtype, B, T);
  if (e != KDA_OK) return e;
  if (!y) return KDA_ERR_NULL;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T;
  if (!dense_aligned(y, D, esz) || !dense_aligned(h0, D, 4) || !dense_aligned(ht, D, 4)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  const size_t need = kda_lru_workspace_bytes(B, T, D, cu_seqlens ? N : 0), ns = (size_t)(cu_seqlens ? N : B) * D * 4;
  if (!need) return KDA_ERR_SHAPE;
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_ALIGN;
  const Span in[] = {{x, rows_bytes(rows, ldx, D, esz)}, {r, rows_bytes(rows, ldr, D, esz)}, {i, i ? rows_bytes(rows, ldi, D, esz) : 0},
                     {c, (size_t)D * 4}, {h0, ns}};
  const Span out[] = {{y, rows * D * esz}, {ht, ns}, {workspace, need}};
  if (!spans_apart(in, out, {-1, 4, -1})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_lru_fwd(dtype == KDA_BF16, a, cu_seqlens, N, B, T, workspace, static_cast<hipStream_t>(stream)));
}

int kda_lru_step(const void* x, long long ldx, const void* r, long long ldr, const void* i, long long ldi, const float* c,
                 const float* state, float* state_out, void* y, int flags, int dtype, int B, int D, void* stream) {
  const kda::LruArgs a{x, r, i, ldx, ldr, ldi, c, state, state_out, y, flags & KDA_LRU_UNIT, D};
  const int e = check_lru(a, flags, dtype, B, 1);
  if (e != KDA_OK) return e;
  if (!state || !state_out || !y) return KDA_ERR_NULL;
  const size_t esz = elem_size(dtype), ns = (size_t)B * D * 4;
  if (!dense_aligned(y, D, esz) || !dense_aligned(state, D, 4) || !dense_aligned(state_out, D, 4)) return KDA_ERR_ALIGN;
  const Span in[] = {{x, rows_bytes(B, ldx, D, esz)}, {r, rows_bytes(B, ldr, D, esz)}, {i, i ? rows_bytes(B, ldi, D, esz) : 0},
                     {c, (size_t)D * 4}, {state, ns}};
  const Span out[] = {{y, (size_t)B * D * esz}, {state_out, ns}};
  if (!spans_apart(in, out, {-1, 4})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_lru_step(dtype == KDA_BF16, a, B, static_cast<hipStream_t>(stream)));
}

size_t kda_lru_bwd_workspace_bytes(int B, int T, int D, int N) {
  return kda_lru_workspace_bytes(B, T, D, N) ? kda::lru_bwd_workspace_bytes(N > 0, N, B, T, D) : 0;
}

int kda_lru_bwd(const void* x, long long ldx, const void* r, long long ldr, const void* i, long long ldi, const float* c, const float* h0,
                const void* dy, const float* dht, void* dx, void* dr, void* di, float* dc, float* dh0, int flags, int dtype, int B, int T,
                int D, const int* cu_seqlens, int N, void* workspace, size_t workspace_bytes, void* stream) {
  const kda::LruBwdArgs b{{x, r, i, ldx, ldr, ldi, c, h0, nullptr, nullptr, flags & KDA_LRU_UNIT, D}, dy, dht, dx, dr, di, dc, dh0};
  int e = check_lru(b.f, flags, dtype, B, T);
  if (e != KDA_OK) return e;
  if (!dy || !dx || !dr || (i && !di) || (!i && di) || (!c && dc)) return KDA_ERR_NULL;
  const size_t esz = elem_size(dtype), rows = (size_t)B * T, n = rows * D * esz;
  for (const void* p : {dy, (const void*)dx, (const void*)dr, (const void*)di})
    if (!dense_aligned(p, D, esz)) return KDA_ERR_ALIGN;
  if (!dense_aligned(h0, D, 4) || !dense_aligned(dht, D, 4) || !dense_aligned(dh0, D, 4) || !aligned16(dc)) return KDA_ERR_ALIGN;
  if ((e = check_cu(cu_seqlens, N, B, T)) != KDA_OK) return e;
  const size_t need = kda_lru_bwd_workspace_bytes(B, T, D, cu_seqlens ? N : 0), ns = (size_t)(cu_seqlens ? N : B) * D * 4;
  if (!need) return KDA_ERR_SHAPE;
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_ALIGN;
  const Span in[] = {{x, rows_bytes(rows, ldx, D, esz)}, {r, rows_bytes(rows, ldr, D, esz)}, {i, i ? rows_bytes(rows, ldi, D, esz) : 0},
                     {c, (size_t)D * 4}, {h0, ns}, {dy, n}, {dht, ns}};
  const Span out[] = {{dx, n}, {dr, n}, {di, di ? n : 0}, {dc, (size_t)D * 4}, {dh0, ns}, {workspace, need}};
  if (!spans_apart(in, out, {-1, -1, -1, -1, -1, -1})) return KDA_ERR_OVERLAP;
  return hip_status(kda::launch_lru_bwd(dtype == KDA_BF16, b, cu_seqlens, N, B, T, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
