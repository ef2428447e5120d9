// Internal declarations shared by the host API and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qlora_nf4.h"

namespace qn {

// Tables handed to the codec kernels by value (they live in the kernel argument
// segment; kernels copy what they index dynamically into LDS), one per 4-bit
// type (QN_NF4, QN_FP4).
//   code[16]      the table's values by code (fp32).
//   thr[33], base[33], lohi[33]  bucket table for the nearest-value search: a
//   normalised value n in [-1, 1 + 2^-23] falls into bucket b = floor(16 n +
//   16) (0 .. 32; bucket 32 holds n >= 1); its level is base[b] + (n >=
//   thr[b]) among the distinct values in ascending order, and its code is
//   byte (n >= thr[b]) of lohi[b].  For NF4 the code of a level is the level
//   itself.
constexpr int kBuckets = 33;
struct CodecTables {
  float code[16];
  float thr[kBuckets];
  uint32_t base[kBuckets];
  uint32_t lohi[kBuckets];
};

// Host: the tables of a 4-bit type (codebook.cpp).  Idempotent, thread-safe.
const CodecTables &codec_tables(int qtype = QN_NF4);
// False if a decision table failed its self-check (never expected).
bool codec_tables_ok();

// Host: fp64 NF4 rows before rounding (exposed for the library's own checks).
void nf4_rows_f64(double out[16]);

// Compute units of the current device (device.cpp); cached per device, thread-safe.
int device_cus();

// Kernel-level timing (trace.cpp).  While tracing is enabled, an object of this
// type records a start event on construction and a stop event on destruction,
// on the given stream, and logs the pair under `kind` (QN_TRACE_* codes).
class TraceScope {
 public:
  TraceScope(int kind, hipStream_t s);
  ~TraceScope();
  TraceScope(const TraceScope &) = delete;
  TraceScope &operator=(const TraceScope &) = delete;

 private:
  int kind_;
  hipStream_t stream_;
  hipEvent_t start_ = nullptr, stop_ = nullptr;
};

// Kernel launchers (return hipError_t of the launch).
// Quantise n weights; with absmax_q and scale2 non-null the same launch also
// double-quantises the block scales (a workgroup per group of 256 blocks).
hipError_t launch_quantize(const void *W, int w_is_bf16, int64_t n, int qtype, uint8_t *codes,
                           float *absmax, uint8_t *absmax_q, float *scale2, hipStream_t s);
hipError_t launch_double_quant(const float *absmax, int64_t nb, uint8_t *absmax_q,
                               float *scale2, hipStream_t s);
hipError_t launch_dequant(const qn_nf4_weight &W, void *out, int out_bf16, hipStream_t s);
// One 8-bit AdamW step (k_adamw8.hip): the fp32 constants of the step, with
// c1 = 1 - b1, c2 = 1 - b2, bc1 = 1 - b1^t, bc2 = 1 - b2^t formed in fp64 and
// rounded once on the host.
struct AdamConsts {
  float lr, b1, b2, eps, wd, c1, c2, bc1, bc2;
};
hipError_t launch_adamw8(uint16_t *p, const uint16_t *g, int64_t n, int8_t *mq, float *ms, uint8_t *uq, float *us,
                         const AdamConsts &c, hipStream_t s);
// The same step over up to QN_ADAMW_MULTI tensors in one launch: tensor i owns
// spans (of 256 parameters) [first[i], first[i + 1]).
struct AdamTensor {
  uint16_t *p;
  const uint16_t *g;
  int64_t n;
  int8_t *mq;
  float *ms;
  uint8_t *uq;
  float *us;
};
struct AdamMulti {
  AdamTensor t[QN_ADAMW_MULTI];
  int64_t first[QN_ADAMW_MULTI + 1];
  int n;
};
hipError_t launch_adamw8_multi(const AdamMulti &mt, const AdamConsts &c, hipStream_t s);

// Adapter merged into the dequantised base (k_merge.hip).  W.K % 64 == 0, 1 <= r <= 64.
hipError_t launch_merge(const qn_nf4_weight &W, const uint16_t *A, const uint16_t *B, int64_t r, float alpha,
                        void *out, int out_bf16, hipStream_t s);

// Scale of block b: fl32(k_b * step_g) with double quantisation, else
// absmax[b]; qtype names the table the codes index.
struct ScaleSrc {
  const float *absmax;
  const uint8_t *absmax_q;
  const float *scale2;
  int qtype;
};

// The 16 values of a 4-bit table, passed by value to kernels that build LDS
// tables from them.
struct Code16 {
  float v[16];
};
Code16 code16(int qtype = QN_NF4);

// Counter-based dropout (qn_philox.h): thr = 0 means none.
struct DropArgs {
  uint32_t thr;
  float c;                     // 1 / (1 - thr / 65536); 1 without dropout
  uint64_t seed, offset;
  const uint64_t *offset_dev;  // added to offset on the device, or null
};
constexpr DropArgs kNoDrop{0u, 1.0f, 0u, 0u, nullptr};
hipError_t launch_dropout(const void *x, int is_bf16, int64_t n, const DropArgs &d, void *y, hipStream_t s);

// Dequant-GEMM (k_qgemm.hip).  out[M, Nout] (bf16) =
//   sum_k L[m, k] * W_hat(k, n)  +  sum_{j<r} L2[m, j] * R2(j, n)
// where W_hat(k, n) = bf16(fl32(table[q] * scale)) of weight element
//   (n, k) of codes [Nout, Kc]   (forward, "NK"), or
//   (k, n) of codes [Kc, Nout]   (dX, "KN"),
// and R2(j, n) = R2[n*ldr2 + j] (forward) or R2[j*ldr2 + n] (dX).
// Requires Kc % 64 == 0 and Nout % 64 == 0.
struct QGemmArgs {
  const uint16_t *L;
  int64_t ldl;
  int64_t M, Nout, Kc;
  const uint8_t *codes;
  const float *absmax;
  const uint8_t *absmax_q;
  const float *scale2;
  int qtype;
  const uint16_t *L2;
  int64_t ldl2;
  const uint16_t *R2;
  int64_t ldr2;
  int64_t r;
  uint16_t *out;
  int64_t ldo;
  int tiles_m, tiles_n, group_m;
  DropArgs drop;   // dX only: thr > 0 adds c keep(m, n) * (adapter term), keep over [M, Nout]
  float *part;     // launch_qgemm_split: fp32 [splits][M, Nout] partial products, instead of out
  int splits;
};
// The calls with dropout, whose sums no earlier result pins, cut the contraction
// into ranges where the tiles alone leave most CUs idle.  qgemm_splits: how
// many (1: none; part takes qgemm_part_bytes); launch_qgemm_split: the partial
// products of a.splits > 1 ranges, for launch_split_sum.
int qgemm_splits(int64_t M, int64_t Nout, int64_t Kc);
size_t qgemm_part_bytes(int64_t M, int64_t Nout, int64_t Kc);
hipError_t launch_qgemm_split(const QGemmArgs &a, bool dx, hipStream_t s);
hipError_t launch_qgemm_fwd(const QGemmArgs &a, hipStream_t s);
hipError_t launch_qgemm_dx(const QGemmArgs &a, hipStream_t s);
// Several independent forward products in one launch (n <= QN_MAX_GROUP); the
// problems must agree on the scale source (all double-quantised or none) and
// on the 4-bit type.
hipError_t launch_qgemm_fwd_group(const QGemmArgs *a, int n, hipStream_t s);
// Tiling choice of the dequant-GEMMs (forward and dX) for all later launches: 0 automatic, 1 256 x 128, 2 256 x 256.
void set_gemm_variant(int v);

// Problems of one grouped launch, passed by value in the kernel arguments.
// Workgroups [start[g], start[g+1]) run problem g; each range is a multiple of
// 8 workgroups (the XCD count), the tail ones past the problem's tiles exit.
struct QGemmGroup {
  QGemmArgs p[QN_MAX_GROUP];
  int start[QN_MAX_GROUP + 1];
  int n;
};

// Low-rank product (k_lowrank.hip): C[M, R] = L[M, Kc] * P[R, Kc]^T, R <= 64,
// Kc % 64 == 0.  Writes any of: out_f32 [M, R] (unscaled), out_b [M, ldb] =
// bf16(scale * C) zero beyond R, out_t [ldt_rows, Mp] = bf16(scale * C)^T zero
// beyond R and beyond M (Mp >= M).  The contraction is cut into
// lowrank_splits(M, Kc) ranges whose fp32 partial products go to `part`
// (lowrank_part_bytes(M, Kc, R) bytes of workspace) and are then added in
// range order, so the result depends on the shape alone.
struct LowRankArgs {
  const uint16_t *L;
  int64_t ldl, M, Kc;
  const uint16_t *P;
  int64_t ldp, R;
  float scale;
  float *out_f32;
  uint16_t *out_b;
  int64_t ldb;
  uint16_t *out_t;
  int64_t ldt_rows, Mp;
  float *part;
  int splits;   // set by the launcher
  DropArgs drop = kNoDrop;   // thr > 0: L is read as keep * L and C scaled by c
  uint8_t *qc = nullptr;     // non-null (a launch of one product): MXFP4 of L (before dropout) is written
  uint8_t *qs = nullptr;     // too, codes [M, 128 C] and scales [C][M][8]
  int t_pieces = 1;          // 2: out_t is [2][ldt_rows, Mp], the rounded value and the rounded rest
  bool p_transposed = false; // P is [Kc, R] (ldp not used)
  const float *given = nullptr;   // C itself, fp32 [M, R], scaled by drop.c already: the outputs only
};
int lowrank_splits(int64_t M, int64_t Kc);
size_t lowrank_part_bytes(int64_t M, int64_t Kc, int64_t R);
hipError_t launch_lowrank(const LowRankArgs &a, hipStream_t s);
// Two independent products with the same rank bucket in one launch (b may be null).
hipError_t launch_lowrank2(const LowRankArgs &a, const LowRankArgs *b, hipStream_t s);
// Up to QN_MAX_GROUP independent products in one launch (blockIdx.y picks one).
hipError_t launch_lowrank_n(const LowRankArgs *a, int n, hipStream_t s);

// Column-streaming reduction over rows (k_lowrank.hip): out = bf16(sum_m
// Lt[j][m] * Q[m][c]) for j < R <= 64, as [R][Ncols] or transposed [Ncols][R].
// Lt is [>= R rows, Mp] bf16 zero beyond M; Q is [M, Ncols] bf16, leading dim
// ldq.  `part` holds colred_splits(M) * R * Ncols floats.
struct ColRedArgs {
  const uint16_t *Lt;
  int64_t Mp;
  const uint16_t *Q;
  int64_t ldq, M, Ncols, R;
  float *part;
  uint16_t *out;
  bool transpose;
};
int colred_splits(int64_t M);
hipError_t launch_colred(const ColRedArgs &a, hipStream_t s, int trace_kind);
// Two independent reductions over the same M in one launch (b may be null);
// each needs its own `part`.
hipError_t launch_colred2(const ColRedArgs &a, const ColRedArgs *b, hipStream_t s, int trace_kind);

// The same sums on the matrix cores (k_colsum.hip), for the MXFP4 linear and for
// dropout: `part` holds splits * R * Ncols floats, Ncols % 64 == 0.
struct ColSumArgs {
  const uint16_t *Lt;  // [2][R, Mp]: two bf16 pieces
  int64_t Mp;
  const uint16_t *Q;   // [M, Ncols]
  int64_t M, Ncols, R;
  float *part;
  int splits;
  uint16_t *out;
  bool transpose;
  DropArgs drop;       // thr > 0: Q is read as keep * Q and the sum scaled by c; kNoDrop for none
};
int colsum_splits(int64_t M, int64_t cols);
hipError_t launch_colsum2(const ColSumArgs &a, const ColSumArgs &b, hipStream_t s, int trace_kind);
// Their reduction over the splits, a launch of its own (the MXFP4 dX's finishing
// pass, when there is one, takes it along: launch_mx_dx).
hipError_t launch_colsum_reduce(const ColSumArgs &a, const ColSumArgs &b, hipStream_t s);

// out (bf16, n elements, n % 8 == 0) = the sum of the fp32 partial products [splits][n]; with sums non-null also
// the reduction of those two column sums.
hipError_t launch_split_sum(const float *part, int splits, int64_t n, uint16_t *out, const ColSumArgs *sums,
                            hipStream_t s);

// Forward pieces.
struct FwdArgs {
  const uint16_t *X;     // bf16 [M,K]
  int64_t M, N, K, r;
  const uint8_t *codes;
  ScaleSrc sc;
  const uint16_t *A;     // bf16 [r,K]
  const uint16_t *B;     // bf16 [N,r]
  float s;               // alpha / r
  uint16_t *Y;           // bf16 [M,N]
  float *H_out;          // fp32 [M,r] or null
  void *ws;
  size_t ws_bytes;
  DropArgs drop = kNoDrop;   // run_fwd_dropout only
};
size_t fwd_workspace(int64_t M, int64_t N, int64_t K, int64_t r);
hipError_t run_fwd(const FwdArgs &a, hipStream_t s);
// The forward with dropout on the adapter's input: the MFMA path for every M.
size_t fwd_dropout_workspace(int64_t M, int64_t N, int64_t K, int64_t r);
hipError_t run_fwd_dropout(const FwdArgs &a, hipStream_t s);
// Several forwards: decode-path problems (M <= 8) as in run_fwd, the others
// with one low-rank launch and one dequant-GEMM launch per scale source.  Each
// problem's workspace is a[g].ws (carved by the caller).
hipError_t run_fwd_group(const FwdArgs *a, int n, hipStream_t s);
// Device address of the current device's static scratch array (k_linear.hip),
// looked up once per device.
hipError_t noalloc_scratch(void **ptr);

struct BwdArgs {
  const uint16_t *dY;    // bf16 [M,N]
  const uint16_t *X;     // bf16 [M,K]
  const float *H;        // fp32 [M,r] = X A^T from the forward, or null (recomputed)
  int64_t M, N, K, r;
  const uint8_t *codes;
  ScaleSrc sc;
  const uint16_t *A;     // bf16 [r,K]
  const uint16_t *B;     // bf16 [N,r]
  float s;
  uint16_t *dX;          // bf16 [M,K] or null
  uint16_t *dA;          // bf16 [r,K]
  uint16_t *dB;          // bf16 [N,r]
  void *ws;
  size_t ws_bytes;
  DropArgs drop = kNoDrop;
  bool dropout = false;                 // a call with dropout (whose p may be 0)
  const uint8_t *mx_scales = nullptr;   // non-null: the base is MXFP4 (codes, mx_scales)
};
// Without dX's partial products; fused: the MXFP4 base and the calls with dropout.
size_t bwd_workspace(int64_t M, int64_t N, int64_t K, int64_t r, bool fused);
hipError_t run_bwd(const BwdArgs &a, hipStream_t s);

// ---- MXFP4 (k_mx.hip, k_mxdx.hip).  Layouts as qn_mx_matrix.
inline int64_t mx_chunks(int64_t cols) { return (cols + QN_MX_CHUNK - 1) / QN_MX_CHUNK; }
hipError_t launch_mx_quantize(const void *x, int is_bf16, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                              hipStream_t s);
hipError_t launch_mx_dequant(const qn_mx_matrix &W, void *out, int out_bf16, hipStream_t s);
struct MxFwdArgs {
  const uint16_t *X;       // bf16 [M, K]
  int64_t M, N, K, r;      // r = 0: no adapter
  const uint8_t *codes, *scales;
  const uint16_t *A, *B;
  float s;
  uint16_t *Y;
  float *H_out;
  void *ws;
  DropArgs drop;
};
size_t mx_fwd_workspace(int64_t M, int64_t N, int64_t K, int64_t r);
hipError_t run_mx_fwd(const MxFwdArgs &a, hipStream_t s);
// dX[M, K] = G[M, N] bf16(W[N, K]) + c keep * (dHb[M, ldh] A[r, K]); r = 0: no adapter term.
struct MxDxArgs {
  const uint16_t *G;
  int64_t M, N, K;
  const uint8_t *codes, *scales;
  const uint16_t *dHb;
  int64_t ldh;
  const uint16_t *A;
  int64_t r;
  DropArgs drop;
  uint16_t *dX;
  float *part;             // mx_dx_part_bytes(M, N, K) of workspace
  int splits;              // set by the launcher
};
size_t mx_dx_part_bytes(int64_t M, int64_t N, int64_t K);
// With sums non-null (two ColSumArgs, already launched), also their reduction.
hipError_t launch_mx_dx(const MxDxArgs &a, const ColSumArgs *sums, hipStream_t s);

}  // namespace qn
