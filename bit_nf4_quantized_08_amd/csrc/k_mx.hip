// MXFP4 on gfx950: quantisation, dequantisation and the QLoRA linear's forward
// over an MXFP4 base.
//
// The format (32 elements of E2M1 under one power of two) is what
// v_mfma_scale_f32_*_f8f6f4 multiplies: lane operands are 32 consecutive
// elements of one row, 16 bytes, with the block's scale byte beside them, so
// codes go from memory to the matrix cores without any expansion.  A product
// of two codes is exact and every sum is fp32.
//
// Kernels, with times on their own (a traced launch) where the bound shows:
//   mx_quantize_kernel   fp32 or bf16 rows -> codes and scales; bound by memory
//                        (4096 x 8192 bf16: 85 MB, 15.3 us, 5.5 TB/s)
//   mx_dequant_kernel    codes and scales -> fp32 or bf16; bound by memory (the
//                        same to bf16: 15.7 us, 5.4 TB/s)
//   mx_gemm_kernel       tiles of mx(X) W^T with the adapter term, optionally over
//                        a part of K with fp32 partial sums (4096 x 8192 x 8192, r =
//                        64: 134 to 138 us, 4.1 PFLOP/s at 1.75 GHz).  A step's 3700
//                        cycles are near the sum of the MFMAs' 2048 (57 % busy) and
//                        LDS' 196 KB of reads and 68 KB of writes (2080 at 128 bytes a
//                        cycle; the LDS-active counter, which leaves the direct loads
//                        out, shows 1070): the two overlap little
//   mx_prep_kernel       few rows: X^ and the adapter's H partials; bound by its
//                        launch and one memory latency (M = 1, K = 8192, r = 64: 4.0 us)
//   mx_decode_kernel     M <= 32: streams the weights; bound by memory (M = 13, 28672
//                        x 8192: 125 MB, 22 us, 5.7 TB/s; M = 1, 8192 x 8192: 36 MB,
//                        9.0 us, 4.0 TB/s, a third of it start and end)
//   mx_finish_kernel     adds partial products and the adapter term; bound by its
//                        launch at the sizes that cut K (about 5 us)

#include <algorithm>

#include "qn_mx.h"
#include "qn_mx_scales.h"
#include "qn_philox.h"
#include "qn_tile.h"

namespace qn {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

#define QN_TRY(x)                      \
  do {                                 \
    hipError_t e_ = (x);               \
    if (e_ != hipSuccess) return e_;   \
  } while (0)

// n / d for n < 2^31 by one multiply: q = (mulhi(n, m) + n) >> s.
struct FastDiv {
  uint32_t m, s, d;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{(uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) { return (__umulhi(n, f.m) + n) >> f.s; }

// ------------------------------------------------------------------ codec
// Unit u of a matrix: 8 consecutive columns of one row, 32 units per 256-column
// chunk, chunks of a row together.  A lane owns one unit, a quad of lanes one
// block (qn_mx.h).  Each thread takes kUnits units a workgroup apart, loads
// first.
constexpr int kThreads = 256;
constexpr int kUnits = 4;

// A grid dimension holds less than 2^32 threads; 2^31 chunks need 2^34.
constexpr int64_t kMaxGridX = 1 << 22;
__device__ __forceinline__ uint32_t codec_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

// VEC: cols is a multiple of 8, so that a unit is aligned and whole.  T threads
// take chunks `first` .. of the matrix, U units each.
template <bool BF16, bool VEC, int T, int U>
__device__ __forceinline__ void quantize_units(const uint8_t *__restrict__ x, uint32_t rows, int64_t cols, FastDiv cd,
                                               uint32_t chunks, uint32_t first, uint8_t *__restrict__ codes,
                                               uint8_t *__restrict__ scales) {
  constexpr int V = BF16 ? 1 : 2, ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x;
  u32x4 v[U][V];
  uint32_t ch[U], row[U];
  const uint32_t c0 = first + (tid >> 5);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t c = c0 + i * (T / 32);
    row[i] = div_by(c, cd);
    ch[i] = c - row[i] * cd.d;
    const int64_t col = (int64_t)ch[i] * 256 + 8 * (tid & 31);
    const uint8_t *p = x + ((int64_t)row[i] * cols + col) * ES;
#pragma unroll
    for (int q = 0; q < V; ++q) v[i][q] = u32x4{0, 0, 0, 0};
    if (c < chunks) {
      if constexpr (VEC) {
        if (col < cols)
#pragma unroll
          for (int q = 0; q < V; ++q) v[i][q] = reinterpret_cast<const u32x4 *>(p)[q];
      } else {
        uint32_t e[4 * V] = {};
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (col + t >= cols) break;
          if constexpr (BF16) e[t >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[t] << (16 * (t & 1));
          else e[t] = reinterpret_cast<const uint32_t *>(p)[t];
        }
#pragma unroll
        for (int q = 0; q < V; ++q) v[i][q] = u32x4{e[4 * q], e[4 * q + 1], e[4 * q + 2], e[4 * q + 3]};
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t b = scale_byte<BF16>(quad_max(unit_amax<BF16>(v[i])));
    const uint32_t c = c0 + i * (T / 32);
    if (c < chunks) {
      reinterpret_cast<uint32_t *>(codes)[(int64_t)c * 32 + (tid & 31)] = unit_codes<BF16>(v[i], b);
      if ((tid & 3) == 0) scales[((int64_t)ch[i] * rows + row[i]) * 8 + ((tid & 31) >> 2)] = (uint8_t)b;
    }
  }
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const uint8_t *__restrict__ x, uint32_t rows,
                                                               int64_t cols, FastDiv cd, uint32_t chunks,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scales) {
  quantize_units<BF16, VEC, kThreads, kUnits>(x, rows, cols, cd, chunks, codec_block() * (kThreads / 32 * kUnits), codes,
                                              scales);
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, uint32_t rows,
                                                              int64_t cols, FastDiv cd, uint32_t chunks,
                                                              uint8_t *__restrict__ out) {
  constexpr int ES = BF16 ? 2 : 4;
  const int tid = threadIdx.x;
  uint32_t cw[kUnits], sb[kUnits], ch[kUnits], row[kUnits];
  const uint32_t c0 = codec_block() * (kThreads / 32 * kUnits) + (tid >> 5);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t c = c0 + i * (kThreads / 32);
    row[i] = div_by(c, cd);
    ch[i] = c - row[i] * cd.d;
    cw[i] = sb[i] = 0;
    if (c < chunks) {
      cw[i] = reinterpret_cast<const uint32_t *>(codes)[(int64_t)c * 32 + (tid & 31)];
      sb[i] = scales[((int64_t)ch[i] * rows + row[i]) * 8 + ((tid & 31) >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t c = c0 + i * (kThreads / 32);
    const int64_t col = (int64_t)ch[i] * 256 + 8 * (tid & 31);
    if (c >= chunks || col >= cols) continue;
    const float sc = as_f32(sb[i] << 23);
    uint8_t *p = out + ((int64_t)row[i] * cols + col) * ES;
    uint32_t o[BF16 ? 4 : 8];
    if constexpr (BF16) {
      o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[i], sc, 0));
      o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[i], sc, 1));
      o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[i], sc, 2));
      o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[i], sc, 3));
      if (sb[i] == 255u) o[0] = o[1] = o[2] = o[3] = 0x7FC07FC0u;
    } else {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], sc, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], sc, 1);
      const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], sc, 2);
      const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw[i], sc, 3);
      const float w[8] = {a.x, a.y, b.x, b.y, e.x, e.y, f.x, f.y};
#pragma unroll
      for (int t = 0; t < 8; ++t) o[t] = sb[i] == 255u ? 0x7FC00000u : as_u32(w[t]);
    }
    if constexpr (VEC) {
      reinterpret_cast<u32x4 *>(p)[0] = u32x4{o[0], o[1], o[2], o[3]};
      if constexpr (!BF16) reinterpret_cast<u32x4 *>(p)[1] = u32x4{o[4], o[5], o[6], o[7]};
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (col + t >= cols) break;
        if constexpr (BF16) reinterpret_cast<uint16_t *>(p)[t] = (uint16_t)(o[t >> 1] >> (16 * (t & 1)));
        else reinterpret_cast<uint32_t *>(p)[t] = o[t];
      }
    }
  }
}

// ------------------------------------------------------------------ tiles
// out[M, N] = X^ W^T over steps of one 256-column chunk (128 bytes of codes per
// row).  A workgroup of WR x WC waves computes a 32 TM WR x 32 TN WC tile; a
// wave multiplies TM x TN tiles of 32 x 32 with v_mfma_scale_f32_32x32x64: in
// sub-step j (0..3) lane half h of a row supplies block 4h + j of the chunk for
// both operands, so that one dword per row half (blocks 4h .. 4h + 3) holds
// the scale bytes of all four sub-steps, picked by the instruction's byte
// select.
// Codes reach LDS by direct loads, one step ahead in the other of two stages,
// 16-byte piece k of row r at slot k ^ ((r >> 1) & 7): a fragment read takes
// one piece of 16 consecutive rows, which then fall on 16 distinct groups of
// four banks (rows are 128 bytes apart, two rows to a turn of the 64 banks).
// The scale bytes come with them (8 BM and 8 BN contiguous bytes, 16 a lane).
// The adapter term bf16(s H) B^T (r <= 64) follows as bf16 MFMAs into the same
// accumulators, its fragments read from global memory (H is small, B is read
// once per tile column).  One piece of s H rounds each product by 2^-8 at most, as
// Y's own rounding does Y: it shows where the adapter's part is most of Y (error
// against 64 bits at 4096 x 8192 x 8192: 0.0017 of Y's norm, that of a bf16 result
// formed in fp32); two pieces would double these MFMAs and s H's memory.  (Reading them a sub-step ahead, or leaving out the
// loads past the last step, changes nothing at 4096 x 8192 x 8192: 136.5 us at
// best in each form, the clock falls by what the schedule gains.)
struct MxGemmArgs {
  const uint8_t *xc, *xs;    // X^: codes [M, 128 C], scales [C][M][8]
  const uint8_t *wc, *ws;    // W: [N, 128 C], [C][N][8]
  int64_t M, N, C;           // N: columns of this launch
  int64_t ldn;               // columns of Y and rows of the scale array
  const uint16_t *sH;        // bf16 [M, 64], zero beyond r, or null
  const uint16_t *B;         // bf16 [N, r]
  int64_t r;
  uint16_t *out;             // bf16 [M, N] (splits == 1)
  float *part;               // fp32 [splits][M][N]
  int tiles_m, tiles_n, group_m, splits;
};

template <int TM, int TN, int WR, int WC, bool PART>
__global__ __launch_bounds__(64 * WR * WC) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx_gemm_kernel(MxGemmArgs a) {
  constexpr int NW = WR * WC, BM = 32 * TM * WR, BN = 32 * TN * WC;
  constexpr int XL = BM / 8 / NW, WL = BN / 8 / NW;   // direct loads (8 rows each) per wave and step
  static_assert(XL * 8 * NW == BM && WL * 8 * NW == BN, "stage loads");
  constexpr int EP = (BM + BN) / 128;                 // direct loads of scales (128 rows each)
  static_assert(NW % EP == 0 && BM % 128 == 0, "scale loads");
  constexpr int kPitch = 32 * TN + 8;                 // bf16 per row of a store block
  __shared__ __attribute__((aligned(16))) uint8_t xs0[BM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t xs1[BM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ws0[BN * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ws1[BN * 128];
  __shared__ __attribute__((aligned(16))) uint8_t es0[(BM + BN) * 8];   // scales: X^'s rows, then W's
  __shared__ __attribute__((aligned(16))) uint8_t es1[(BM + BN) * 8];
  static_assert(NW * 32 * kPitch * 2 <= 2 * BM * 128 + 2 * BN * 128, "store blocks fit the stages");

  int tm, tn;
  xcd_tile((int)blockIdx.x, a.tiles_m, a.tiles_n, a.group_m, tm, tn);
  const int split = (int)blockIdx.y;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave % WR, wc = wave / WR;
  const int C = (int)a.C, s0 = C * split / a.splits, s1 = C * (split + 1) / a.splits;
  const int64_t pitch = 128 * a.C;

  const rsrc_t rx = make_rsrc_u(a.xc + m0 * pitch, (a.M - m0) * pitch);
  const rsrc_t rw = make_rsrc_u(a.wc + n0 * pitch, (a.N - n0) * pitch);
  // Direct load g covers rows 8g .. 8g + 7: lane l fills slot l & 7 of row
  // 8g + l / 8 with piece (l & 7) ^ ((row >> 1) & 7) of that row.
  auto load_off = [&](int g) {
    const int row = 8 * g + (lane >> 3);
    return (uint32_t)(row * pitch + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
  };
  uint32_t xo[XL], wo[WL];
#pragma unroll
  for (int i = 0; i < XL; ++i) xo[i] = load_off(wave * XL + i);
#pragma unroll
  for (int i = 0; i < WL; ++i) wo[i] = load_off(wave * WL + i);
  const int64_t xrow = m0 + wr * 32 * TM, wrow = n0 + wc * 32 * TN;
  // Scales: load p covers rows 128 p .. of X^'s BM rows and then W's.  Every wave
  // makes one load, so some are made twice, with the same bytes to the same
  // place: a branch here would split the step's block, and the compiler would
  // move the MFMAs past it.  Rows past the matrix get the last rows' scales: their
  // products are not stored.
  const int erow = 128 * (wave % EP);
  const bool of_x = erow < BM;
  const rsrc_t re = of_x ? make_rsrc_u(a.xs, a.C * a.M * 8) : make_rsrc_u(a.ws, (a.C - 1) * a.ldn * 8 + a.N * 8);
  const uint32_t eo = mx_scale_pair((of_x ? m0 + erow : n0 + erow - BM) + 2 * lane, of_x ? a.M : a.N);
  const int estep = (int)((of_x ? a.M : a.ldn) * 8);
  // Load i of step s into a stage.
  constexpr int LOADS = XL + WL + 1;
  const uint32_t xl = (uint32_t)(wave * XL * 1024), wl = (uint32_t)(wave * WL * 1024);
  auto issue = [&](uint8_t *xd, uint8_t *wd, uint8_t *ed, int s, int i) {
    if (i < XL) load_lds16(rx, (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(xd)) + xl + i * 1024, xo[i], s * 128);
    else if (i < XL + WL)
      load_lds16(rw, (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(wd)) + wl + (i - XL) * 1024, wo[i - XL], s * 128);
    else
      load_lds16(re, (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(ed)) + 8 * erow, eo, s * estep);
  };
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  uint32_t fo[4];   // LDS offset of sub-step j's piece in row lr of a tile
#pragma unroll
  for (int j = 0; j < 4; ++j) fo[j] = (uint32_t)(lr * 128 + 16 * ((4 * lh + j) ^ ((lr >> 1) & 7)));
  // A fragment is four registers; the instruction's eight-register operand type
  // is formed at its use (carried over the loop, its unused half would be too).
  auto frag = [&](const uint8_t *p) { return *reinterpret_cast<const u32x4 *>(p); };
  auto wide = [&](u32x4 v) { return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; };
  // Sub-step j: blocks 4 lh + j; byte j of the rows' scale dwords.
  struct Frag {
    u32x4 a[TM], b[TN];
  };
  struct Scales {
    uint32_t a[TM], b[TN];
  };
  const int xp = wr * 32 * TM * 128, wp = wc * 32 * TN * 128;
  const int ex = (wr * 32 * TM + lr) * 8 + 4 * lh, ew = (BM + wc * 32 * TN + lr) * 8 + 4 * lh;
  auto read_f = [&](Frag &f, const uint8_t *xc, const uint8_t *wc_, int j) {
#pragma unroll
    for (int i = 0; i < TM; ++i) f.a[i] = frag(xc + xp + i * 32 * 128 + fo[j]);
#pragma unroll
    for (int i = 0; i < TN; ++i) f.b[i] = frag(wc_ + wp + i * 32 * 128 + fo[j]);
  };
  auto read_e = [&](Scales &t, const uint8_t *ec) {
#pragma unroll
    for (int i = 0; i < TM; ++i) t.a[i] = *reinterpret_cast<const uint32_t *>(ec + ex + 32 * 8 * i);
#pragma unroll
    for (int i = 0; i < TN; ++i) t.b[i] = *reinterpret_cast<const uint32_t *>(ec + ew + 32 * 8 * i);
  };
  // Sub-step J's MFMAs, with hook(0) .. hook(3) spread between them.
  auto mma = [&](const Frag &f, const Scales &t, auto J, auto &&hook) {
    constexpr int j = decltype(J)::value, per = TM * TN / 4;
#pragma unroll
    for (int m = 0; m < TM * TN; ++m) {
      const int i = m / TN, k = m % TN;
      acc[i][k] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(f.a[i]), wide(f.b[k]), acc[i][k], 4, 4, j,
                                                                  (int)t.a[i], j, (int)t.b[k]);
      if (m % per == per - 1) {
        __builtin_amdgcn_sched_barrier(0);
        hook(m / per);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // One step: stage `c` now, stage `n` next.  On entry f0 and tc hold sub-step 0's
  // fragments and the scales, and the first four loads of step s + 1 are on
  // their way.  Fragments are read a sub-step ahead; the barrier comes when the
  // last of them are in registers, so that the next stage's first fragments are
  // read under the last sub-step's MFMAs.  The direct loads are spread over the
  // MFMAs, the other loads of step s + 1 over sub-steps 0 and 1, the first four
  // of step s + 2 over sub-step 3: issued together they fill the CU's vector
  // memory path, and each wave would stand at its next load with its MFMAs
  // behind it.  (Touching the lines of later steps to bring them into L2 costs
  // more of that path than it saves: 139 -> 152 us.)
  const int last = s1 - 1;
  auto none = [](int) {};
  auto step = [&](int s, uint8_t *xc, uint8_t *wc_, uint8_t *ec, uint8_t *xn, uint8_t *wn, uint8_t *en, Frag &f0, Frag &f1,
                  const Scales &tc, Scales &tn_) {
    const int sn = min(s + 1, last), sm = min(s + 2, last);
    read_f(f1, xc, wc_, 1);
    __builtin_amdgcn_sched_barrier(0);
    mma(f0, tc, std::integral_constant<int, 0>{}, [&](int q) {
      if (4 + q < LOADS) issue(xn, wn, en, sn, 4 + q);
    });
    read_f(f0, xc, wc_, 2);
    __builtin_amdgcn_sched_barrier(0);
    mma(f1, tc, std::integral_constant<int, 1>{}, [&](int q) {
      if (8 + q < LOADS) issue(xn, wn, en, sn, 8 + q);
    });
    read_f(f1, xc, wc_, 3);
    __builtin_amdgcn_sched_barrier(0);
    mma(f0, tc, std::integral_constant<int, 2>{}, none);
    stage_barrier();
    read_e(tn_, en);
    read_f(f0, xn, wn, 0);
    __builtin_amdgcn_sched_barrier(0);
    mma(f1, tc, std::integral_constant<int, 3>{}, [&](int q) { issue(xc, wc_, ec, sm, q); });
  };
  // Stage (s - s0) & 1 holds step s; past the end the last step is loaded again.
  static_assert(LOADS > 4 && LOADS <= 12, "load schedule");
#pragma unroll
  for (int i = 0; i < LOADS; ++i) issue(xs0, ws0, es0, s0, i);
  stage_barrier();
  Frag f0, f1;
  Scales t0, t1;
#pragma unroll
  for (int i = 0; i < 4; ++i) issue(xs1, ws1, es1, min(s0 + 1, last), i);
  read_e(t0, es0);
  read_f(f0, xs0, ws0, 0);
  for (int s = s0; s < s1; s += 2) {
    step(s, xs0, ws0, es0, xs1, ws1, es1, f0, f1, t0, t1);
    if (s + 1 >= s1) break;
    step(s + 1, xs1, ws1, es1, xs0, ws0, es0, f0, f1, t1, t0);
  }
  // The loads past the end must land before the stages are written again.
  stage_barrier();

  if constexpr (PART) {
    float *part = a.part + (int64_t)split * a.M * a.N;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int64_t n = wrow + 32 * j + lr;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int64_t m = xrow + 32 * i + 8 * (e >> 2) + 4 * lh + (e & 3);
          if (m < a.M && n < a.N) part[m * a.N + n] = acc[i][j][e];
        }
      }
    return;
  }

  if (a.sH) {
    // Sub-step c: lane half h supplies ranks 16 c + 8 h .. + 7 of its row.
    const rsrc_t rh = make_rsrc_u(a.sH + xrow * 64, (a.M - xrow) * 128);
    const rsrc_t rb = make_rsrc_u(a.B + wrow * a.r, (a.N - wrow) * a.r * 2);
    const int steps = (int)(a.r + 15) / 16;
    const bool vec = (a.r & 7) == 0;
    for (int c = 0; c < steps; ++c) {
      u32x4 ha[TM], hb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        ha[i] = __builtin_amdgcn_raw_buffer_load_b128(rh, (uint32_t)((32 * i + lr) * 128 + 32 * c + 16 * lh), 0, 0);
      const int j0 = 16 * c + 8 * lh;
      if (vec) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
          hb[i] = __builtin_amdgcn_raw_buffer_load_b128(
              rb, j0 < a.r ? (uint32_t)(((32 * i + lr) * a.r + j0) * 2) : kOutOfRange, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t o = (uint32_t)(((32 * i + lr) * a.r + j0 + 2 * q) * 2);
            const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(rb, j0 + 2 * q < a.r ? o : kOutOfRange, 0, 0);
            const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(rb, j0 + 2 * q + 1 < a.r ? o + 2 : kOutOfRange, 0, 0);
            w[q] = (lo & 0xFFFFu) | hi << 16;
          }
          hb[i] = u32x4{w[0], w[1], w[2], w[3]};
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int k = 0; k < TN; ++k)
          acc[i][k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, ha[i]),
                                                              __builtin_bit_cast(bf16x8, hb[k]), acc[i][k], 0, 0, 0);
    }
  }

  // Store through LDS (the stages are no longer read): each wave turns its
  // 32 x 32 TN blocks into whole 16-byte pieces of rows.  Rows at or beyond M
  // fall outside the buffer; N is a multiple of 64, so pieces are whole.
  constexpr int kBlock = 32 * kPitch;   // bf16
  constexpr int kPerStage = BM * 64 / kBlock;
  static_assert(kPerStage >= 1, "a store block fits a stage");
  uint16_t *blk;
  {
    // Blocks are laid over xs0, xs1, ws0, ws1 in turn.
    constexpr int wper = BN * 64 / kBlock;
    uint8_t *p = wave < kPerStage ? xs0 + wave * kBlock * 2
                 : wave < 2 * kPerStage ? xs1 + (wave - kPerStage) * kBlock * 2
                 : wave < 2 * kPerStage + wper ? ws0 + (wave - 2 * kPerStage) * kBlock * 2
                                               : ws1 + (wave - 2 * kPerStage - wper) * kBlock * 2;
    static_assert(2 * kPerStage + 2 * wper >= NW, "store blocks");
    blk = reinterpret_cast<uint16_t *>(p);
  }
  const rsrc_t rout = make_rsrc_u(a.out + m0 * a.ldn, (a.M - m0) * a.ldn * 2);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        blk[(8 * (e >> 2) + 4 * lh + (e & 3)) * kPitch + j * 32 + lr] = f32_to_bf16(acc[i][j][e]);
    constexpr int kPieces = 4 * TN, kRows = 64 / kPieces;   // pieces per row, rows per store
#pragma unroll
    for (int q = 0; q < 32 / kRows; ++q) {
      const int row = kRows * q + lane / kPieces, c8 = 8 * (lane % kPieces);
      const u32x4 v = *reinterpret_cast<const u32x4 *>(&blk[row * kPitch + c8]);
      const int64_t lrow = wr * 32 * TM + 32 * i + row, n = wrow + c8;
      __builtin_amdgcn_raw_buffer_store_b128(v, rout, n < a.N ? (uint32_t)((lrow * a.ldn + n) * 2) : kOutOfRange, 0, 0);
    }
  }
}

// ------------------------------------------------------------------ few rows
// M <= 32, two launches.  The first quantises X and forms partial sums of H = X
// A^T (with both repeated in every workgroup of the streaming kernel 11.4 + 9.8 us
// against 5.2 + 8.9 at M = 1, 8192 x 8192, r = 64; H is what costs there: a wave needs
// only its own columns of X^, and quantising those alone in the streaming kernel is
// not built); the second streams the weights
// and, when a workgroup's waves cover all of K (up to 8192 columns), finishes Y.
//
// Streaming: a wave owns 16 weight rows x 1024 columns at a time, eight
// sub-steps of v_mfma_scale_f32_16x16x128 with the weights as the first operand
// (lane: row lane % 16, block lane / 16 of the sub-step's four) and X^ in groups
// of 16 rows, held in registers, as the second.  The codes come through LDS by
// direct loads of two rows x 512 contiguous bytes each: read straight into the
// fragments they would come as 64-byte pieces of 16 rows (8192 x 8192, M = 1, when
// this was measured: 10.4 against 12.1 us).  The wave reads a group's eight
// fragments into registers and asks for the next group before it multiplies, so
// its 8 KB of LDS are always on their way.  16-byte piece p of row r sits at slot
// p ^ r, which spreads a fragment read's 16 rows over the banks.
// A workgroup's 8 waves cover nk (a power of two) column segments of 8 / nk
// sets of row groups; partial sums meet in LDS.
constexpr int DW = 8;                 // waves
constexpr int DSEG = 1024;            // columns per wave
constexpr int DSUB = DSEG / 128;      // sub-steps

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }

struct MxPrepArgs {
  const uint16_t *X;
  int64_t M, K;
  FastDiv cd;          // by the chunks of a row
  uint32_t chunks;     // of X
  uint8_t *xc, *xs;
  int qblocks;         // workgroups that quantise; the rest form H partials
  const uint16_t *A;
  int64_t r;
  DropArgs drop;
  float *h_part;       // [hsplits][M][64]
  int hsplits, mgroups;   // mgroups: 16-row groups of X
};

// H partials: workgroup b of them takes 16 rows of X, 16 ranks of A and 8 x HSEG
// columns.
template <int HSEG>
__device__ __forceinline__ void prep_h(const MxPrepArgs &a, int b, float (*red)[256]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, kb = lane >> 4;
  const int mg = b % a.mgroups, jt = b / a.mgroups / a.hsplits, hs = b / a.mgroups % a.hsplits, j = 16 * jt + l16;
  const int64_t m = 16 * mg + l16;
  const int64_t k0 = (int64_t)hs * (DW * HSEG) + wave * HSEG + 8 * kb;
  const rsrc_t ra = make_rsrc_u(a.A, a.r * a.K * 2), rx = make_rsrc_u(a.X, a.M * a.K * 2);
  u32x4 av[HSEG / 32], xv[HSEG / 32];
#pragma unroll
  for (int i = 0; i < HSEG / 32; ++i) {
    const int64_t k = k0 + 32 * i;
    av[i] = __builtin_amdgcn_raw_buffer_load_b128(ra, j < a.r && k < a.K ? (uint32_t)((j * a.K + k) * 2) : kOutOfRange, 0, 0);
    xv[i] = __builtin_amdgcn_raw_buffer_load_b128(rx, m < a.M && k < a.K ? (uint32_t)((m * a.K + k) * 2) : kOutOfRange, 0, 0);
  }
  if (a.drop.thr) {
    const DropKey dk = drop_key(a.drop);
#pragma unroll
    for (int i = 0; i < HSEG / 32; ++i) {
      uint32_t w[4];
      philox7((uint64_t)m * (uint64_t)(a.K / 8) + (uint64_t)((k0 + 32 * i) >> 3), dk, w);
      xv[i] &= u32x4{keep_mask2(w[0], dk.thr2), keep_mask2(w[1], dk.thr2), keep_mask2(w[2], dk.thr2),
                     keep_mask2(w[3], dk.thr2)};
    }
  }
  f32x4 acc = zero4();
#pragma unroll
  for (int i = 0; i < HSEG / 32; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[i]), __builtin_bit_cast(bf16x8, xv[i]),
                                                  acc, 0, 0, 0);
  // acc[e]: rank 16 jt + 4 kb + e, row l16.
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][l16 * 16 + 4 * kb + e] = acc[e];
  __syncthreads();
  if (tid < 256) {
    const int mo = 16 * mg + (tid >> 4), jj = tid & 15;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < DW; ++w) v += red[w][tid];
    if (mo < a.M) a.h_part[((int64_t)hs * a.M + mo) * 64 + 16 * jt + jj] = v;
  }
}

template <int HSEG>
__global__ __launch_bounds__(64 * DW) void mx_prep_kernel(MxPrepArgs a) {
  __shared__ float red[DW][256];
  if ((int)blockIdx.x < a.qblocks)
    quantize_units<true, true, 64 * DW, 1>(reinterpret_cast<const uint8_t *>(a.X), (uint32_t)a.M, a.K, a.cd, a.chunks,
                                           blockIdx.x * (64 * DW / 32), a.xc, a.xs);
  else
    prep_h<HSEG>(a, (int)blockIdx.x - a.qblocks, red);
}

// Adapter operands of a 16 x 16 block of Y (v_mfma_f32_16x16x32_bf16, B's rows
// first): H's row m from its partial sums, ranks 8 kb .. + 7 of group jg of 32,
// scaled by c, then s H in two bf16 pieces (high and the rest, 2^-17 of it left
// over, so H counts as in fp32).
struct HPieces {
  bf16x8 hi, lo;
};
struct AdapterArgs {
  const uint16_t *sH;  // bf16 s H [M, 64], zero beyond r (one piece, as in the tiles): used when non-null, else
  const float *hp;     // [hsplits][M][64] unscaled (columns at or beyond r undefined), or null
  int hsplits;
  const uint16_t *B;   // bf16 [N, r]
  int64_t r;
  float s, c;
  float *H_out;        // or null
};

// c * the sum of H's partial sums first .. end - 1, ranks j0 .. + 7 of row m.
__device__ __forceinline__ void sum_h(const AdapterArgs &a, int64_t M, int64_t m, int j0, int first, int end, float (&h)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) h[t] = 0.0f;
  // Batches of four partial sums, loaded without a condition (past the last
  // one it is read again and dropped), so that a batch waits once.
  for (int q0 = first; q0 < end; q0 += 4) {
    f32x4 v[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 *p = reinterpret_cast<const f32x4 *>(a.hp + ((int64_t)min(q0 + q, end - 1) * M + m) * 64 + j0);
      v[q][0] = p[0];
      v[q][1] = p[1];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q0 + q < end)
#pragma unroll
        for (int t = 0; t < 8; ++t) h[t] += v[q][t >> 2][t & 3];
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) h[t] = j0 + t < a.r ? h[t] * a.c : 0.0f;
}

__device__ __forceinline__ void store_h(const AdapterArgs &a, int64_t m, int j0, const float (&h)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if (j0 + t < a.r) a.H_out[m * a.r + j0 + t] = h[t];
}

__device__ __forceinline__ HPieces pieces_of(const AdapterArgs &a, const float (&h)[8]) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float x = a.s * h[2 * t], y = a.s * h[2 * t + 1];
    hi[t] = pack_bf16x2(x, y);
    lo[t] = pack_bf16x2(x - bf16_lo(hi[t]), y - bf16_hi(hi[t]));
  }
  return HPieces{__builtin_bit_cast(bf16x8, (u32x4{hi[0], hi[1], hi[2], hi[3]})),
                 __builtin_bit_cast(bf16x8, (u32x4{lo[0], lo[1], lo[2], lo[3]}))};
}

// B[n][j0 .. j0 + 7], zero beyond r.
__device__ __forceinline__ bf16x8 load_b(const AdapterArgs &a, int64_t n, int j0) {
  uint32_t w[4];
  if ((a.r & 7) == 0) {
    const u32x4 v = j0 < a.r ? *reinterpret_cast<const u32x4 *>(a.B + n * a.r + j0) : u32x4{0, 0, 0, 0};
    return __builtin_bit_cast(bf16x8, v);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t x = j0 + 2 * t < a.r ? a.B[n * a.r + j0 + 2 * t] : 0u;
    const uint32_t y = j0 + 2 * t + 1 < a.r ? a.B[n * a.r + j0 + 2 * t + 1] : 0u;
    w[t] = x | y << 16;
  }
  return __builtin_bit_cast(bf16x8, (u32x4{w[0], w[1], w[2], w[3]}));
}

// The same from bf16 s H.
__device__ __forceinline__ bf16x8 load_sh(const AdapterArgs &a, int64_t m, int j0) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(a.sH + m * 64 + j0));
}

// The rest's sum is kept apart and added where it is finite: an infinite s H (or
// one that rounds to an infinite bf16) leaves the rest an opposite infinity or NaN,
// and an infinite element of B an infinity of either sign, while the high pieces
// alone give the infinity that the product has.
__device__ __forceinline__ f32x4 add_adapter(f32x4 acc, bf16x8 b, const HPieces &h) {
  const f32x4 rest = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, h.lo, zero4(), 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, h.hi, acc, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] += __builtin_isfinite(rest[e]) ? rest[e] : 0.0f;
  return acc;
}

struct MxDecodeArgs {
  const uint8_t *xc, *xs;   // X^: codes [M, 128 C], scales [C][M][8]
  int64_t M, N, C;
  const uint8_t *wc, *ws;
  AdapterArgs ad;           // used when out is written
  uint16_t *out;            // Y, when one workgroup covers K; else null and
  float *y_part;            // [ksplits][M][N]
  int nk, row_blocks;
};

// G, MB: 16-row groups of W per wave and of X.  At most 128 registers: two
// workgroups to a CU.
template <int G, int MB>
__global__ __launch_bounds__(64 * DW) __attribute__((amdgpu_waves_per_eu(4, 4))) void mx_decode_kernel(MxDecodeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t stage[DW][16 * DSEG / 2];   // a wave's weights
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kb = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rb = (int)blockIdx.x % a.row_blocks, ks = (int)blockIdx.x / a.row_blocks;
  const int seg = wave & (a.nk - 1), rg = wave / a.nk, ng = DW / a.nk;
  const int64_t k0 = ((int64_t)ks * a.nk + seg) * DSEG;
  const int64_t pitch = 128 * a.C;
  const int64_t n0 = ((int64_t)rb * ng + rg) * (16 * G);     // first row of the wave
  const int bytes = (int)min((int64_t)DSEG / 2, max((int64_t)0, pitch - k0 / 2));   // of the segment that exist

  // Scale bytes of a lane's block in the eight sub-steps (byte kb of the sub-step's
  // dword), four to a register: the instruction's byte select takes them there.
  const uint32_t pick = 0x0C0C0000u | (uint32_t)(kb + 4) << 8 | (uint32_t)kb;
  auto pack_scales = [&](const u32x2 (&e)[DSUB / 2], uint32_t (&out)[DSUB / 4]) {
#pragma unroll
    for (int h = 0; h < DSUB / 4; ++h)
      out[h] = __builtin_amdgcn_perm(e[2 * h].y, e[2 * h].x, pick) |
               __builtin_amdgcn_perm(e[2 * h + 1].y, e[2 * h + 1].x, pick) << 16;
  };
  // X^: rows 16 b + l16, piece 4 i + kb of the segment; zero past the row or the
  // rows.
  const rsrc_t rx = make_rsrc_u(a.xc, a.M * pitch);
  const rsrc_t rxs = make_rsrc_u(a.xs, a.C * a.M * 8);
  u32x4 xv[MB][DSUB];
  uint32_t xe[MB][DSUB / 4];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int m = 16 * b + l16;
    u32x2 e[DSUB / 2];
#pragma unroll
    for (int i = 0; i < DSUB; ++i)
      xv[b][i] = __builtin_amdgcn_raw_buffer_load_b128(
          rx, m < a.M && 64 * i < bytes ? (uint32_t)(m * pitch + k0 / 2 + 64 * i + 16 * kb) : kOutOfRange, 0, 0);
#pragma unroll
    for (int i = 0; i < DSUB / 2; ++i)
      e[i] = __builtin_amdgcn_raw_buffer_load_b64(
          rxs, m < a.M && 128 * i < bytes ? (uint32_t)(((k0 / 256 + i) * a.M + m) * 8) : kOutOfRange, 0, 0);
    pack_scales(e, xe[b]);
  }

  // Weights: direct load t of a group brings rows 2 t and 2 t + 1 (slot lane % 32
  // of row 2 t + lane / 32: piece slot ^ row).  Out-of-range lanes bring zeros.
  const rsrc_t rw = make_rsrc_u(a.wc + n0 * pitch + k0 / 2, (a.N - n0) * pitch - k0 / 2);
  const rsrc_t rs = make_rsrc_u(a.ws, a.C * a.N * 8);
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(stage[wave]));
  u32x2 we[DSUB / 2];
  auto load_w = [&](int g) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int row = 2 * t + (lane >> 5), piece = (lane & 31) ^ row;
      const bool in = n0 + 16 * g + row < a.N && 16 * piece < bytes;
      load_lds16(rw, lds + 1024 * t, in ? (uint32_t)((16 * g + row) * pitch + 16 * piece) : kOutOfRange, 0);
    }
#pragma unroll
    for (int i = 0; i < DSUB / 2; ++i)
      we[i] = __builtin_amdgcn_raw_buffer_load_b64(
          rs, n0 + 16 * g + l16 < a.N && 128 * i < bytes ? (uint32_t)(((k0 / 256 + i) * a.N + n0 + 16 * g + l16) * 8) : kOutOfRange,
          0, 0);
  };
  load_w(0);
  // With one group of each, the adapter's operands are requested here too, behind
  // the weights.
  constexpr bool PRE = G == 1 && MB == 1;
  f32x4 ph[2][2] = {};
  bf16x8 pb[2] = {};
  if (PRE && a.out && a.ad.hp && seg < a.ad.hsplits) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (32 * q >= a.ad.r) break;
      const f32x4 *p = reinterpret_cast<const f32x4 *>(a.ad.hp + ((int64_t)seg * a.M + min((int64_t)l16, a.M - 1)) * 64 + 32 * q + 8 * kb);
      ph[q][0] = p[0];
      ph[q][1] = p[1];
      pb[q] = load_b(a.ad, min(n0 + l16, a.N - 1), 32 * q + 8 * kb);
    }
  }

  f32x4 acc[G][MB];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's direct loads have landed
    asm volatile("" ::: "memory");
    i32x8 wf[DSUB];
#pragma unroll
    for (int i = 0; i < DSUB; ++i) {
      const u32x4 v = *reinterpret_cast<const u32x4 *>(&stage[wave][l16 * 512 + 16 * ((4 * i + kb) ^ l16)]);
      wf[i] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
    }
    uint32_t sw[DSUB / 4];
    pack_scales(we, sw);
    if (g + 1 < G) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the fragments are read before LDS is refilled
      load_w(g + 1);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      acc[g][b] = zero4();
      auto sub = [&](auto I) {
        constexpr int i = decltype(I)::value;
        const i32x8 xf = {(int)xv[b][i].x, (int)xv[b][i].y, (int)xv[b][i].z, (int)xv[b][i].w, 0, 0, 0, 0};
        acc[g][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[i], xf, acc[g][b], 4, 4, i & 3, (int)sw[i >> 2],
                                                                     i & 3, (int)xe[b][i >> 2]);
      };
      sub(std::integral_constant<int, 0>{}); sub(std::integral_constant<int, 1>{});
      sub(std::integral_constant<int, 2>{}); sub(std::integral_constant<int, 3>{});
      sub(std::integral_constant<int, 4>{}); sub(std::integral_constant<int, 5>{});
      sub(std::integral_constant<int, 6>{}); sub(std::integral_constant<int, 7>{});
    }
  }
  // acc[g][b][e]: weight row 16 g + 4 kb + e, row 16 b + l16 of X.
  // The adapter term is linear in H, so each wave adds that of the partial sums
  // its segment index selects (with one workgroup over K there is one per
  // segment), and none stands at all of them.  Under an infinite element of B the
  // parts' signs would meet as inf - inf: the first segment's wave then adds the
  // term of all of H, the others none (every wave of the rows sees the same B).
  if (a.out && a.ad.hp && seg < a.ad.hsplits) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int j0 = 32 * q + 8 * kb;
      if (32 * q >= a.ad.r) break;
      bf16x8 bv[G];
      float h[MB][8];
      uint32_t top = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) bv[g] = PRE ? pb[q] : load_b(a.ad, min(n0 + 16 * g + l16, a.N - 1), j0);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const u32x4 u[1] = {__builtin_bit_cast(u32x4, bv[g])};
        top = max(top, unit_amax<true>(u));
      }
      // Expected false, so that its code lies out of the way too.
      const bool whole = __builtin_expect(__any(top >= 0x7F80u), 0);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        if (PRE) {
#pragma unroll
          for (int t = 0; t < 8; ++t) h[b][t] = j0 + t < a.ad.r ? ph[q][t >> 2][t & 3] * a.ad.c : 0.0f;
        } else {
          sum_h(a.ad, a.M, min((int64_t)(16 * b + l16), a.M - 1), j0, seg, seg + 1, h[b]);
        }
      }
      if (__builtin_expect(whole, 0)) {
#pragma unroll
        for (int b = 0; b < MB; ++b) sum_h(a.ad, a.M, min((int64_t)(16 * b + l16), a.M - 1), j0, 0, a.ad.hsplits, h[b]);
      }
      if (!whole || seg == 0) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const HPieces p = pieces_of(a.ad, h[b]);
#pragma unroll
          for (int g = 0; g < G; ++g) acc[g][b] = add_adapter(acc[g][b], bv[g], p);
        }
      }
    }
  }
  // Partial sums [G * MB * 256] in place of the wave's own stage.
  static_assert(G * MB * 1024 <= 16 * DSEG / 2, "partial sums fit");
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<float *>(stage[wave])[(g * MB + b) * 256 + l16 * 16 + 4 * kb + e] = acc[g][b][e];
  __syncthreads();
  // Element idx of a row group set: (set q, group g, group b, row of X in 16, row in 16).
  constexpr int per = G * MB * 256;
  for (int idx = tid; idx < ng * per; idx += 64 * DW) {
    const int q = idx / per, in = idx % per, g = in / (MB * 256), b = in / 256 % MB;
    float v = 0.0f;
    for (int w = 0; w < a.nk; ++w) v += reinterpret_cast<const float *>(stage[q * a.nk + w])[in];
    const int64_t n = ((int64_t)rb * ng + q) * (16 * G) + 16 * g + (in & 15);
    const int m = 16 * b + ((in >> 4) & 15);
    if (m < a.M && n < a.N) {
      if (a.out) a.out[m * a.N + n] = f32_to_bf16(v);
      else a.y_part[((int64_t)ks * a.M + m) * a.N + n] = v;
    }
  }
  // H itself, written by one wave, comes last: its code among the above, skipped by
  // the others, costs them 0.3 us of fetching (one token, 8192 x 8192).
  if (a.out && a.ad.hp && a.ad.H_out && rb == 0 && wave == 0)
#pragma unroll
    for (int b = 0; b < MB; ++b)
      for (int j0 = 8 * kb; j0 < a.ad.r; j0 += 32) {
        const int64_t m = 16 * b + l16;
        float h[8];
        sum_h(a.ad, a.M, min(m, a.M - 1), j0, 0, a.ad.hsplits, h);
        if (m < a.M) store_h(a.ad, m, j0, h);
      }
}

// Y = sum of the partial products + s H B^T; also writes H.  A wave owns 16
// columns x 16 rows of Y and needs no LDS; a lane ends with four consecutive
// columns of one row: 16-byte reads of the partial products, one 8-byte store.
struct MxFinishArgs {
  const float *part;   // [splits][M][N]
  int splits;
  AdapterArgs ad;
  int64_t M, N;
  uint16_t *out;
};

__global__ __launch_bounds__(256) void mx_finish_kernel(MxFinishArgs a) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, kb = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * 16, m = (int64_t)blockIdx.y * 16 + l16;
  const bool in = m < a.M;
  const int64_t mc = in ? m : a.M - 1;   // lanes past the rows read the last one
  f32x4 acc = zero4();
  for (int q0 = 0; q0 < a.splits; q0 += 4) {
    f32x4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = *reinterpret_cast<const f32x4 *>(a.part + ((int64_t)min(q0 + q, a.splits - 1) * a.M + mc) * a.N + n0 + 4 * kb);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q0 + q < a.splits) acc += v[q];
  }
  if (a.ad.sH) {
    for (int j0 = 8 * kb; j0 - 8 * kb < a.ad.r; j0 += 32)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(load_b(a.ad, n0 + l16, j0), load_sh(a.ad, mc, j0), acc, 0, 0, 0);
  } else if (a.ad.hp) {
    for (int j0 = 8 * kb; j0 - 8 * kb < a.ad.r; j0 += 32) {
      const bf16x8 b = load_b(a.ad, n0 + l16, j0);
      float h[8];
      sum_h(a.ad, a.M, mc, j0, 0, a.ad.hsplits, h);
      if (a.ad.H_out && blockIdx.x == 0 && wave == 0 && in) store_h(a.ad, m, j0, h);
      acc = add_adapter(acc, b, pieces_of(a.ad, h));
    }
  }
  // acc[e]: column n0 + 4 kb + e, row m.
  if (in)
    *reinterpret_cast<u32x2 *>(a.out + m * a.N + n0 + 4 * kb) =
        u32x2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
}

// ------------------------------------------------------------------ plans
struct Carve {
  char *base;
  size_t off = 0;
  explicit Carve(void *p) : base(static_cast<char *>(p)) {}
  template <typename T>
  T *take(int64_t count) {
    T *p = reinterpret_cast<T *>(base ? base + off : nullptr);
    off += (size_t)align_up(count * (int64_t)sizeof(T), 256);
    return p;
  }
};

constexpr int64_t kDecodeRows = 32;

struct DecodePlan {
  int nk, ksplits, row_blocks, groups;
};
DecodePlan decode_plan(int64_t M, int64_t N, int64_t K) {
  DecodePlan p;
  const int64_t segs = cdiv(K, DSEG);
  p.nk = 1;
  while (p.nk < DW && p.nk < segs) p.nk *= 2;
  p.ksplits = (int)cdiv(segs, p.nk);
  // Row groups per wave: one while the workgroups are resident at once (two to
  // a CU), then two or four, which keeps them resident for longer weights and
  // lets a wave ask for its next rows before it is done with these (four with 32
  // rows of X would spill).
  const int64_t wgs = cdiv(N, 16 * (DW / p.nk)) * p.ksplits;
  p.groups = wgs <= 2 * device_cus() ? 1 : (wgs <= 4 * device_cus() || M > 16 ? 2 : 4);
  p.row_blocks = (int)cdiv(N, (int64_t)16 * p.groups * (DW / p.nk));
  return p;
}

// Tiles of a forward.  256 x 256 ones (a workgroup fills a CU) move half the
// bytes per product of 128 x 128 ones (two fit a CU), so they are taken when they
// fill at least half the CUs.  A round of them costs about 2.0 us per chunk of K,
// a round of 128 x 128 tiles 1.3 us with two on a CU, 0.8 us with one (8192 x
// 8192 weights); a last round that is mostly empty is cut off as whole columns of
// tiles and given to 128 x 128 tiles in a second launch (about 3 us) where that
// is cheaper.  128 x 128 tiles may be cut over K, for which the partial sums are
// written and read once more.
struct GemmPlan {
  int64_t wide;   // columns on 256 x 256 tiles
  int splits;     // of the others, over K
};
GemmPlan gemm_plan(int64_t M, int64_t N, int64_t C) {
  const int64_t cus = device_cus(), tm = cdiv(M, 256), T = tm * cdiv(N, 256);
  if (2 * T > cus) {
    const int64_t rounds = T / cus, full = rounds * cus / tm * 256;   // columns of whole rounds
    if (rounds == 0 || T % cus == 0 || full >= N) return GemmPlan{N, 1};
    const int64_t rest = cdiv(M, 128) * cdiv(N - full, 128);
    const double narrow = rest <= cus ? 0.8 : 1.3 * (double)cdiv(rest, 2 * cus);
    return GemmPlan{narrow * (double)C + 3.0 < 2.0 * (double)C ? full : N, 1};
  }
  const int64_t mid = cdiv(M, 128) * cdiv(N, 128);
  int splits = 1;
  double best = 1e300;
  for (int k = 1; k <= 8 && (k == 1 || C / k >= 2); k *= 2) {
    const double rounds = mid * k <= cus ? 0.8 : 1.3 * (double)cdiv(mid * k, 2 * cus);
    const double sums = k == 1 ? 0.0 : 3.0 + (double)(k * M * N) * 8.0 / 4.5e6;   // written and read at 4.5 TB/s
    const double us = rounds * (double)cdiv(C, k) + sums;
    if (us < best) { best = us; splits = k; }
  }
  return GemmPlan{0, splits};
}

struct FwdPieces {
  uint8_t *xc, *xs;        // X^
  float *y_part;           // partial products (decode beyond one workgroup's columns, split tiles)
  float *h_part;           // partial sums of H (decode: [hsplits][M][64]; tiles: the low-rank kernel's)
  uint16_t *sH;            // bf16 s H (tiles that finish Y themselves)
  size_t bytes;
};
// Columns per wave of a partial sum of H: 128 where the streaming kernel finishes
// Y, so that there is one sum per segment and each wave adds its own (M = 1, 8192 x
// 8192, r = 64: 4.0 + 8.7 us against 5.1 + 9.0 with 256 columns and one wave adding
// them all); 256, half the sums to add, where another kernel finishes it.
int prep_hseg(int64_t M, int64_t N, int64_t K) { return M <= kDecodeRows && decode_plan(M, N, K).ksplits == 1 ? 128 : 256; }
int prep_hsplits(int64_t M, int64_t N, int64_t K) { return (int)cdiv(K, DW * prep_hseg(M, N, K)); }
// Rows up to which split tiles take X^ and H from the few-row path's first launch
// and leave H's partial sums to their finishing kernel (each of its waves reads
// them for its rows): the low-rank kernel has one workgroup per 128 rows and
// range, too few for so little.
constexpr int64_t kPrepRows = 128;

FwdPieces fwd_pieces(void *ws, int64_t M, int64_t N, int64_t K, int64_t r) {
  FwdPieces p{};
  Carve c(ws);
  const int64_t C = mx_chunks(K);
  p.xs = c.take<uint8_t>(M * 8 * C);   // the codes come after it: mx_scale_pair
  p.xc = c.take<uint8_t>(M * 128 * C);
  const int splits = M <= kDecodeRows ? decode_plan(M, N, K).ksplits : gemm_plan(M, N, C).splits;
  if (splits > 1) p.y_part = c.take<float>((int64_t)splits * M * N);
  if (r && (M <= kDecodeRows || (M <= kPrepRows && splits > 1))) {
    p.h_part = c.take<float>((int64_t)prep_hsplits(M, N, K) * M * 64);
  } else if (r) {
    p.h_part = reinterpret_cast<float *>(c.take<char>((int64_t)lowrank_part_bytes(M, K, r)));
    p.sH = c.take<uint16_t>(M * 64);
  }
  p.bytes = c.off;
  return p;
}

template <int TM, int TN, int WR, int WC, bool PART>
hipError_t launch_tiles(MxGemmArgs g, hipStream_t st) {
  constexpr int BM = 32 * TM * WR, BN = 32 * TN * WC;
  g.tiles_m = (int)cdiv(g.M, BM);
  g.tiles_n = (int)cdiv(g.N, BN);
  // An XCD runs about 1/8 of the tiles, at most a 32-CU round at a time: a
  // square-ish patch of them shares the most.
  g.group_m = std::max(1, std::min(g.tiles_m, 4));
  const int64_t T = (int64_t)g.tiles_m * g.tiles_n;
  if (T > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)T, (unsigned)g.splits), block(64 * WR * WC);
  TraceScope tr(QN_TRACE_MX_GEMM, st);
  hipLaunchKernelGGL((mx_gemm_kernel<TM, TN, WR, WC, PART>), grid, block, 0, st, g);
  return hipGetLastError();
}

hipError_t launch_finish(const MxFinishArgs &f, hipStream_t st) {
  const dim3 grid((unsigned)(f.N / 64), (unsigned)cdiv(f.M, 16));   // N % 64 == 0
  hipLaunchKernelGGL(mx_finish_kernel, grid, dim3(256), 0, st, f);
  return hipGetLastError();
}

// X^ and H's partial sums (h_part [prep_hsplits][M][64]).
hipError_t launch_prep(const MxFwdArgs &a, const FwdPieces &w, hipStream_t st) {
  const int64_t C = mx_chunks(a.K);
  const uint32_t chunks = (uint32_t)(a.M * C);
  const int qblocks = (int)cdiv(chunks, 64 * DW / 32), mgroups = (int)cdiv(a.M, 16), hsplits = prep_hsplits(a.M, a.N, a.K);
  const int hblocks = a.r ? (int)cdiv(a.r, 16) * hsplits * mgroups : 0;
  const MxPrepArgs q{a.X, a.M, a.K, fast_div((uint32_t)C), chunks, w.xc, w.xs, qblocks, a.A, a.r, a.drop,
                     w.h_part, hsplits, mgroups};
  const dim3 grid((unsigned)(qblocks + hblocks)), block(64 * DW);
  if (prep_hseg(a.M, a.N, a.K) == 128) hipLaunchKernelGGL(mx_prep_kernel<128>, grid, block, 0, st, q);
  else hipLaunchKernelGGL(mx_prep_kernel<256>, grid, block, 0, st, q);
  return hipGetLastError();
}

hipError_t run_decode(const MxFwdArgs &a, const FwdPieces &w, hipStream_t st) {
  const DecodePlan p = decode_plan(a.M, a.N, a.K);
  const int64_t C = mx_chunks(a.K);
  const dim3 block(64 * DW);
  QN_TRY(launch_prep(a, w, st));
  const AdapterArgs ad{nullptr, a.r ? w.h_part : nullptr, prep_hsplits(a.M, a.N, a.K), a.B, a.r, a.s, a.drop.c, a.H_out};
  const MxDecodeArgs d{w.xc, w.xs, a.M, a.N, C, a.codes, a.scales, ad, p.ksplits == 1 ? a.Y : nullptr, w.y_part,
                       p.nk, p.row_blocks};
  const dim3 grid((unsigned)(p.row_blocks * p.ksplits));
  {
    TraceScope tr(QN_TRACE_MX_GEMV, st);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, d); };
    if (a.M <= 16) p.groups == 1 ? go(mx_decode_kernel<1, 1>) : p.groups == 2 ? go(mx_decode_kernel<2, 1>) : go(mx_decode_kernel<4, 1>);
    else p.groups == 1 ? go(mx_decode_kernel<1, 2>) : go(mx_decode_kernel<2, 2>);
  }
  QN_TRY(hipGetLastError());
  if (p.ksplits == 1) return hipSuccess;
  return launch_finish(MxFinishArgs{w.y_part, p.ksplits, ad, a.M, a.N, a.Y}, st);
}

template <bool Q>
hipError_t launch_codec(const void *x, int bf16, int64_t rows, int64_t cols, const uint8_t *ci, const uint8_t *si,
                        uint8_t *co, uint8_t *so, void *out, hipStream_t st) {
  const int64_t C = mx_chunks(cols), chunks = rows * C;
  const FastDiv cd = fast_div((uint32_t)C);
  const int64_t blocks = cdiv(chunks, kThreads / 32 * kUnits), wide = std::min(blocks, kMaxGridX);
  const dim3 grid((unsigned)wide, (unsigned)cdiv(blocks, wide)), block(kThreads);
  const bool vec = cols % 8 == 0;
  const auto *xb = static_cast<const uint8_t *>(x);
  auto *ob = static_cast<uint8_t *>(out);
  const uint32_t R = (uint32_t)rows, n = (uint32_t)chunks;
#define QN_CODEC(B, V)                                                                                          \
  do {                                                                                                          \
    if constexpr (Q) hipLaunchKernelGGL((mx_quantize_kernel<B, V>), grid, block, 0, st, xb, R, cols, cd, n, co, so); \
    else hipLaunchKernelGGL((mx_dequant_kernel<B, V>), grid, block, 0, st, ci, si, R, cols, cd, n, ob);         \
  } while (0)
  if (bf16) {
    if (vec) QN_CODEC(true, true);
    else QN_CODEC(true, false);
  } else {
    if (vec) QN_CODEC(false, true);
    else QN_CODEC(false, false);
  }
#undef QN_CODEC
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int is_bf16, int64_t rows, int64_t cols, uint8_t *codes, uint8_t *scales,
                              hipStream_t st) {
  TraceScope tr(QN_TRACE_MX_QUANTIZE, st);
  return launch_codec<true>(x, is_bf16, rows, cols, nullptr, nullptr, codes, scales, nullptr, st);
}

hipError_t launch_mx_dequant(const qn_mx_matrix &W, void *out, int out_bf16, hipStream_t st) {
  TraceScope tr(QN_TRACE_MX_DEQUANT, st);
  return launch_codec<false>(nullptr, out_bf16, W.rows, W.cols, W.codes, W.scales, nullptr, nullptr, out, st);
}

size_t mx_fwd_workspace(int64_t M, int64_t N, int64_t K, int64_t r) { return fwd_pieces(nullptr, M, N, K, r).bytes; }

hipError_t run_mx_fwd(const MxFwdArgs &a, hipStream_t st) {
  const FwdPieces w = fwd_pieces(a.ws, a.M, a.N, a.K, a.r);
  if (a.M <= kDecodeRows) return run_decode(a, w, st);
  const int64_t C = mx_chunks(a.K);
  const GemmPlan p = gemm_plan(a.M, a.N, C);
  if (a.r == 0) {
    QN_TRY(launch_mx_quantize(a.X, 1, a.M, a.K, w.xc, w.xs, st));
  } else if (!w.sH) {
    QN_TRY(launch_prep(a, w, st));
  } else {   // one pass over X: its low-rank product and its quantisation
    LowRankArgs l{};
    l.L = a.X; l.ldl = a.K; l.M = a.M; l.Kc = a.K;
    l.P = a.A; l.ldp = a.K; l.R = a.r; l.scale = a.s; l.drop = a.drop;
    l.Mp = a.M; l.part = w.h_part;
    l.qc = w.xc; l.qs = w.xs;
    l.out_f32 = a.H_out;
    l.out_b = w.sH;
    l.ldb = 64;
    QN_TRY(launch_lowrank(l, st));
  }
  MxGemmArgs g{w.xc, w.xs, a.codes, a.scales, a.M, a.N, C, a.N, a.r ? w.sH : nullptr, a.B, a.r, a.Y, w.y_part,
               0, 0, 0, p.splits};
  if (p.wide) {
    g.N = p.wide;
    QN_TRY((launch_tiles<2, 4, 4, 2, false>(g, st)));
    if (p.wide == a.N) return hipSuccess;
    g.wc += p.wide * 128 * C;
    g.ws += p.wide * 8;
    if (g.sH) g.B += p.wide * a.r;
    g.out += p.wide;
    g.N = a.N - p.wide;
  }
  if (p.splits == 1) return launch_tiles<2, 2, 2, 2, false>(g, st);
  QN_TRY((launch_tiles<2, 2, 2, 2, true>(g, st)));
  const AdapterArgs ad{w.sH, a.r ? w.h_part : nullptr, prep_hsplits(a.M, a.N, a.K), a.B, a.r, a.s, a.drop.c, a.H_out};
  return launch_finish(MxFinishArgs{w.y_part, p.splits, ad, a.M, a.N, a.Y}, st);
}

}  // namespace qn
