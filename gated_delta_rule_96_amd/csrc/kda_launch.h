// Internal host-side launch interface between the C ABI (kda_api.cpp) and
// the kernel translation units.  Arguments are already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Decay preparation: gate (z != nullptr; softplus != 0 selects the unbounded
// -Softplus gate instead of gmin * Sigmoid) and/or chunk-local cumsum.
hipError_t launch_prepare_decay(int is_bf16, const void* z, const float* A, float gmin, void* g,
                                float* gcum, int B, int T, int H, int dk, int chunk, int softplus,
                                hipStream_t stream);

// Opt-in range check of a log-decay input (KDA_VALIDATE=1 in the
// environment: validate_requested()).  bounded != 0: every g in [gmin, 0];
// otherwise g <= 0; finite in both cases.  With gcum != nullptr the per-row
// decays it encodes are checked instead of g.  g / gcum are [B, T, HD]
// (HD = H * dk).  Synchronises `stream`; *in_range = 1 if every value passes.
bool validate_requested();
hipError_t validate_decay(int is_bf16, const void* g, const float* gcum, int bounded, float gmin, int B, int T,
                          int HD, int chunk, hipStream_t stream, int* in_range);

// Bytes of one per-chunk record of the prefill workspace.
size_t fwd_record_bytes(int is_bf16, int dk, int dv);
// Workspace of the fused single-pass schedule (ring buffers + control words).
size_t fwd_fused_workspace_bytes(int is_bf16, int nbh, int dk, int dv);

// Up to kMaxVarSeq packed sequences of one variable-length prefill, carried
// in the fused kernel's launch arguments: sequence i is tokens cu[i] ..
// cu[i+1]-1 of the packed axis, its chunks (every chunk starts at the
// sequence start) are stream chunks cc[i] .. cc[i+1]-1 of every head, and its
// first snapshot is snapshot sb[i].  n = 0: one plain sequence per (b, h).
constexpr int kMaxVarSeq = 128;
struct VarSeg {
  int n;
  int cu[kMaxVarSeq + 1];
  int cc[kMaxVarSeq + 1];
  int sb[kMaxVarSeq + 1];
};

// Chunked prefill, fused schedule (one persistent kernel per batch of heads).
// unbounded != 0: the decay may go below -5 (diagonal tiles by position pairs).
// snap != nullptr, snap_every > 0: states after every snap_every chunks
// (excluding the end) to snap[j][b * H + h][dk][dv].
// var != nullptr (B = 1): the packed sequences above, h0 / ht [n][H][dk][dv]
// (h0 nullable), snapshots numbered per sequence from sb[i]; sequences
// without tokens are not touched.
// layer_flags (1: g is z, gate with A fused into the scan; 2: q/k rows L2
// normalised in-kernel) and og (output gate pre-activation, nullable).
hipError_t launch_fwd_fused(int is_bf16, const void* q, const void* k, const void* v, const void* g,
                            const float* gcum, const void* beta, float scale, const float* h0, float* ht, float* o,
                            int B, int T, int H, int dk, int dv, void* workspace, size_t workspace_bytes,
                            int unbounded, float* snap, int snap_every, const float* A, const void* og,
                            int layer_flags, hipStream_t stream, const VarSeg* var = nullptr);

// Chunked prefill, two-stage schedule: bit 0 intra-chunk kernel, bit 1 state pass.
hipError_t launch_fwd_stages(int is_bf16, const void* q, const void* k, const void* v, const void* g,
                             const float* gcum, const void* beta, float scale, const float* h0, float* ht, float* o,
                             int B, int T, int H, int dk, int dv, void* workspace, int stages, int unbounded,
                             float* snap, int snap_every, hipStream_t stream);

// Zero-fills nwords 4-byte words on the stream (a kernel, not a memset node).
hipError_t launch_zero_words(void* p, size_t nwords, hipStream_t stream);

// Zeroes the status words (the first 16 ints, error word at [8]) of a
// prefill workspace; called once per API call, before its launches.
hipError_t launch_clear_status(void* ws, hipStream_t stream);

// Library-owned scratch of the allocation-free prefill (a file-scope device
// array, one per GPU): its device address on the current device, fetched
// with hipGetSymbolAddress on the first call there.  40 MiB hold the ring of
// 34 heads with fp32 inputs at dk = dv = 128 (the largest record, 1.16 MB per
// head) and 70 heads with bf16 inputs; larger batches of heads run as
// further launches of the same kernel.
constexpr size_t kNoAllocScratchBytes = (size_t)40 << 20;
hipError_t noalloc_scratch(void** ptr);


// The decode step's layer steps: g holds z and the gate is formed from
// A [H] fp32; flags & kDecodeLayerNormQK normalises the q and k rows; og
// [B,H,dv] of the input type (or null) gates the output.
constexpr int kDecodeLayerNormQK = 2;
struct DecodeLayer {
  const float* A;
  const void* og;
  int flags;
};

// One decode token per (b, h), state updated in place (lay: the layer
// variant, or null for the plain step).
hipError_t launch_decode_step(int is_bf16, const void* q, const void* k, const void* v,
                              const void* g, const void* beta, float scale, float* state, float* o,
                              int B, int H, int dk, int dv, hipStream_t stream,
                              const DecodeLayer* lay = nullptr);

// Backward: fp32 words of one per-chunk record, and the three kernels after
// a forward pass that kept the state entering every chunk in snap
// ([chunk - 1][b * H + h][dk][dv]).  rec, dN ([chunk][dk][dv] per head) and
// dU ([chunk][64][dv] per head) are workspace.
size_t bwd_record_words(int dk, int dv);
hipError_t launch_bwd_chunks(int is_bf16, const void* q, const void* k, const void* v, const void* g,
                             const void* beta, const float* dO, float scale, const float* h0, const float* dht,
                             const float* snap, float* rec, float* dN, float* dU, int B, int T, int H, int dk,
                             int dv, float* dq, float* dk_, float* dv_, float* dg, float* dbeta, float* dh0,
                             hipStream_t st);

// The sequences of one launch of the token-walking operators (short
// convolution, state space scan).  n = 0: sequences of T tokens each, packed
// one behind the other, `parts` parts each.  n > 0: packed sequences n0 ..
// n0+n-1 of the call (at most kMaxVarSeq a launch): sequence n0+i is rows
// cu[i] .. cu[i+1]-1, its parts are items cc[i] .. cc[i+1]-1 of the launch.
// Chunks of kSeqChunk tokens are numbered the same way (an empty sequence has
// one): `chunks` each, or cb[i] .. of packed ones.
constexpr int kSeqChunk = 64;
struct SeqTab {
  int n, n0, T, parts, part, items, chunks;
  int cu[kMaxVarSeq + 1];
  int cc[kMaxVarSeq + 1];
  int cb[kMaxVarSeq + 1];
};
// The table of sequences n0 .. of a call, cut into parts of `part` tokens:
// B sequences of T (cu == nullptr, one launch), or N packed ones from n0 on
// (as many as one launch carries).  Returns the first sequence not covered.
int make_seq_tab(SeqTab& s, const int* cu, int N, int n0, int B, int T, int part);
// Whether none of a call's tables has more than `most` items.
bool seq_tabs_fit(const int* cu, int N, int B, int T, int part, long long most);
// Work-groups of `threads` that one launch may have: a launch of 2^32 threads
// or more runs only a part of them, without an error.  Sizes beyond it are
// hipErrorInvalidConfiguration before a call's first launch.
constexpr long long max_groups(int threads) { return 0xffffffffLL / threads; }

// out[0][c], then out[1], out[2]: column sums of part [nrows][n0 + n1 + n2], in
// a fixed order (any output may be null).  Up to 2^31 columns, in several launches
// where one has not the work-groups.
hipError_t launch_sum_rows(const float* part, size_t nrows, unsigned n0, unsigned n1, unsigned n2, float* out0, float* out1,
                           float* out2, hipStream_t stream);

// Short causal convolution: see kda_conv.hip.  dtypes: 0 fp32, 1 bf16.
struct ConvArgs {
  const void* x;
  long long ldx;       // elements between tokens of x
  const float* w;      // [D][W]
  const float* bias;   // [D] or null
  const void* s0;      // [N][W-1][D] or null
  void* st;            // [N][W-1][D] or null
  void* y;             // [rows][D]
  int silu, D, W;
};
hipError_t launch_conv_fwd(int is_bf16, const ConvArgs& a, const int* cu, int N, int B, int T, hipStream_t stream);
hipError_t launch_conv_step(int is_bf16, const ConvArgs& a, int B, hipStream_t stream);
struct ConvBwdArgs {
  ConvArgs f;          // y unused
  const void* dy;      // [rows][D]
  int dy_bf16;
  const void* dst;     // [N][W-1][D] or null
  void* dx;            // [rows][D]
  float* dw;           // [D][W]
  float* dbias;        // [D] or null
  void* ds0;           // [N][W-1][D] or null
  float* part;         // workspace
};
size_t conv_bwd_workspace_bytes(int is_packed, int N, int B, int T, int D, int W);
hipError_t launch_conv_bwd(int is_bf16, const ConvBwdArgs& a, const int* cu, int N, int B, int T, hipStream_t stream);

// Norms of query and key heads with the position rotation: see kda_qknorm.hip.
struct QkArgs {
  const void* x[2];      // q, k: [tokens][H][d] with token strides ld
  long long ld[2];
  const float* w[2];     // [d] or null
  void* y[2];            // [tokens][H][d]: normed rows, or dq / dk (backward)
  const void* dy[2];     // backward: [tokens][H][d]
  int H[2];              // H[1] may be 0
  const float *cos, *sin;   // [n_pos][rot / 2]
  const int* pos;        // [tokens] or null: pos0 + t
  int pos0, n_pos;
  int rms, inter, d, rot;
  float eps;
  long long tokens;
  int T;
  float* part;           // backward workspace
};
hipError_t launch_qk_fwd(int is_bf16, const QkArgs& a, hipStream_t stream);
size_t qk_bwd_workspace_bytes(long long tokens, int Hq, int Hk, int d);
hipError_t launch_qk_bwd(int is_bf16, int dy_bf16, const QkArgs& a, float* dwq, float* dwk, hipStream_t stream);

// State space scan with one decay per head: see kda_ssm.hip.
struct SsmArgs {
  const void *x, *dt, *B, *C;        // rows [tokens][H][dv], [H], [G][dk], [G][dk]
  long long ldx, lddt, ldb, ldc;
  const float *A, *D, *bias;         // [H]; D and bias may be null
  const float* h0;                   // [N][H][dk][dv] or null
  float* ht;                         // [N][H][dk][dv] or null
  void* y;                           // [tokens][H][dv]
  int softplus, H, G;
  float* seg;                        // workspace: states between a sequence's parts
  float* start;                      // copies of h0 where ht replaces it (or null)
  double* sum;                       // workspace: their decay sums
};
// Tokens of a part for about `wgs` (part, head) work-groups.  A sequence of n
// parts keeps n - 1 states; n - 1 <= its tokens / part.
int ssm_part(long long tokens, int H, int wgs);
// The same, but long enough for the longest sequence where that pays (in
// kda_ssm.hip).
int ssm_part_of(int H, int wgs, const int* cu, int N, int B, int T);
inline size_t ssm_slots(long long tokens, int H, int wgs) { return (size_t)(tokens / ssm_part(tokens, H, wgs)) * H; }
// Workspace bytes of the forward.
size_t ssm_seg_bytes(long long tokens, int H, int dk, int dv);
hipError_t launch_ssm_fwd(int is_bf16, const SsmArgs& a, int dk, int dv, const int* cu, int N, int B, int T, void* workspace,
                          hipStream_t stream);
// One token per sequence: state h0 -> ht (may be the same).
hipError_t launch_ssm_step(int is_bf16, const SsmArgs& a, int dk, int dv, int B, hipStream_t stream);

// Gradients of the scan: see kda_ssm_bwd.hip.  f: the forward's inputs.
struct SsmBwdArgs {
  SsmArgs f;
  const void* dy;              // [tokens][H][dv]
  const float* dht;            // [N][H][dk][dv] or null
  void *dx, *ddt, *dB, *dC;    // of the inputs' type, contiguous
  float *dA, *dD, *dbias;      // [H]; dD and dbias may be null
  float* dh0;                  // or null
};
size_t ssm_bwd_workspace_bytes(int is_packed, int N, int B, int T, int H, int G, int dk, int dv);
hipError_t launch_ssm_bwd(int is_bf16, const SsmBwdArgs& a, int dk, int dv, const int* cu, int N, int B, int T, void* workspace,
                          hipStream_t stream);

// Norm of the residual stream with the residual's addition: see kda_rmsnorm.hip.
struct NormArgs {
  const void* x;         // rows: the addend (forward), h (backward)
  long long ldx;
  const void* res;       // forward: rows of the stream or null; backward: dh, contiguous, or null
  long long ldr;
  const float* w;        // [D] or null
  void* sum;             // forward: h, contiguous
  void* y;               // forward: the norm (8-bit with scale); backward: dx
  float* scale;          // forward: [rows][blocks of 128], or null
  const void* dy;        // backward
  float* part;           // backward workspace, or null
  long long rows;
  int D;
  float eps;
};
hipError_t launch_norm_fwd(int is_bf16, int sum_bf16, const NormArgs& a, hipStream_t stream);
size_t norm_bwd_workspace_bytes(long long rows, int D);
hipError_t launch_norm_bwd(int is_bf16, int dy_bf16, const NormArgs& a, float* dw, hipStream_t stream);

// Product of 8-bit rows and weights with scales by blocks: see kda_gemm8.hip.
struct Gemm8Args {
  const unsigned char* a;   // rows [M][K]
  long long lda;
  const float* sa;          // rows [M][KB]
  long long lsa;
  const unsigned char* w;   // [N][K]
  const float* sw;          // [NB][KB]
  void* c;                  // rows [M][N], ldc apart
  long long M, ldc;
  int N, K;
};
hipError_t launch_gemm8(int out_bf16, const Gemm8Args& g, hipStream_t stream);

// Gated linear recurrence, one state a channel: see kda_lru.hip, kda_lru_bwd.hip.
struct LruArgs {
  const void *x, *r, *i;             // rows [tokens][D]; i may be null
  long long ldx, ldr, ldi;
  const float* c;                    // [D] or null
  const float* h0;                   // [N][D] or null
  float* ht;                         // [N][D] or null
  void* y;                           // [tokens][D]
  int unit, D;
};
size_t lru_workspace_bytes(int is_packed, int N, int B, int T, int D);
hipError_t launch_lru_fwd(int is_bf16, const LruArgs& a, const int* cu, int N, int B, int T, void* workspace, hipStream_t stream);
// One token per sequence: state h0 -> ht (may be the same).
hipError_t launch_lru_step(int is_bf16, const LruArgs& a, int B, hipStream_t stream);
struct LruBwdArgs {
  LruArgs f;                         // ht and y unused
  const void* dy;                    // [tokens][D]
  const float* dht;                  // [N][D] or null
  void *dx, *dr, *di;                // [tokens][D]; di null without i
  float* dc;                         // [D] or null
  float* dh0;                        // [N][D] or null
};
size_t lru_bwd_workspace_bytes(int is_packed, int N, int B, int T, int D);
hipError_t launch_lru_bwd(int is_bf16, const LruBwdArgs& a, const int* cu, int N, int B, int T, void* workspace, hipStream_t stream);

}  // namespace kda
