// Column sums over rows on the matrix cores (gfx950): out[j][c] = sum_m L[j][m] *
// Q[m][c] for j < R <= 64, the contraction of dA = dH^T (keep * X) and dB^T = (s
// H)^T dY, which runs down the rows of row-major activations.  L is fp32 given as
// two bf16 pieces, the rounded value and the rounded rest (2^-17 of it is left
// over), [2][R, Mp], zero beyond M: with one piece the rounding of L would be as
// large as that of the bf16 result.
//
// Bound by reading Q once (both sums of 4096 rows of 8192, r = 64, with dropout:
// 134 MB in 37 us, 3.6 TB/s, then 8 us for the reduction); the products are 128 MACs
// per element of Q at R = 64, too many for vector dot products (the v_dot2
// kernel of k_lowrank.hip, with one piece, takes 150 us for the two sums of 4096
// rows of 8192) and little for the matrix cores.  The MFMA wants eight
// consecutive rows of one column, so a 64-row x 256-column stage of Q goes
// through LDS as it lies and comes back by the transposing read
// (ds_read_b64_tr_b16), as in k_mxdx.hip.  The stage is filled through registers,
// not by direct loads: a 16-byte piece there is one call of the dropout
// generator, so the mask is applied on the way.
//
// A workgroup (8 waves) owns 256 columns and a range of rows; wave w multiplies
// columns 32 w .. + 31 with all ranks.  Stage of Q: row m (512 bytes), piece u of
// 8 columns at slot u ^ 4 (m & 3), so that a transposing read's four rows fall
// on different banks.  Stage of L: rank j (128 bytes), direct loads, piece k at
// slot k ^ ((j >> 1) & 7), two stages.  Q has one stage, refilled between two
// barriers from registers that were loaded a step earlier: with two, 64 ranks
// would leave room for one workgroup on a CU, and half the loads in flight.
// The partial sums of the row ranges go to `part` and are added in order by
// the reduce kernel, so results depend on the shape and, through the number of
// ranges, on the device's CU count.

#include <algorithm>

#include "qn_colsum.h"
#include "qn_philox.h"
#include "qn_tile.h"

namespace qn {
namespace {

constexpr int CS_THREADS = 512;
constexpr int CS_COLS = 256;

// Two bf16 values a dword with infinities and NaN as zero: (0x7F80 - exponent bits),
// 0 for those only, at most 1, times the value.  In asm for what keep_mask2 says.
__device__ __forceinline__ uint32_t finite_or_zero2(uint32_t w) {
  uint32_t d = w & 0x7F807F80u;
  asm("v_pk_sub_u16 %0, %1, %0" : "+v"(d) : "s"(0x7F807F80u));
  asm("v_pk_min_u16 %0, %0, %1" : "+v"(d) : "s"(0x00010001u));
  asm("v_pk_mul_lo_u16 %0, %0, %1" : "+v"(d) : "v"(w));
  return d;
}

// What the second piece of L multiplies: an infinite element of Q times the first
// piece gives the sum its infinity or NaN, times a rest of either sign it would
// make every such sum NaN.
__device__ __forceinline__ bf16x8 finite_or_zero(bf16x8 q) {
  const u32x4 w = __builtin_bit_cast(u32x4, q);
  return __builtin_bit_cast(bf16x8, (u32x4{finite_or_zero2(w.x), finite_or_zero2(w.y), finite_or_zero2(w.z),
                                           finite_or_zero2(w.w)}));
}

template <int RT, bool DROP>   // 32-rank tiles
__global__ __launch_bounds__(CS_THREADS) __attribute__((amdgpu_waves_per_eu(4, 4)))
void colsum_kernel(ColSumArgs a0, ColSumArgs a1) {
  __shared__ __attribute__((aligned(16))) uint8_t qs[64 * 512];
  __shared__ __attribute__((aligned(16))) uint8_t ls0[64 * RT * 128];   // both pieces
  __shared__ __attribute__((aligned(16))) uint8_t ls1[64 * RT * 128];
  const ColSumArgs a = blockIdx.z ? a1 : a0;
  const int64_t c0 = (int64_t)blockIdx.x * CS_COLS;
  if (c0 >= a.Ncols) return;   // the other sum is wider
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = (int)blockIdx.y;
  const int steps = (int)((a.M + 63) / 64);
  const int s0 = (int)((int64_t)steps * split / a.splits), s1 = (int)((int64_t)steps * (split + 1) / a.splits);

  // Q: thread t loads pieces (t & 31) of rows t / 32 + 16 i of a stage, i < 4.
  const int qu = tid & 31, qr = tid >> 5;
  const uint32_t qo = c0 + 8 * qu < a.Ncols ? (uint32_t)((qr * a.Ncols + c0 + 8 * qu) * 2) : kOutOfRange;
  const uint32_t qst = (uint32_t)(qr * 512 + 16 * (qu ^ (4 * (qr & 3))));   // row qr + 16 i: + 8192 i
  u32x4 qv[4];
  auto load_q = [&](int s) {
    // The resource starts at the stage's first row: offsets within 64 rows.
    const rsrc_t rq = make_rsrc_u(a.Q + (int64_t)s * 64 * a.Ncols, (a.M - (int64_t)s * 64) * a.Ncols * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      qv[i] = __builtin_amdgcn_raw_buffer_load_b128(
          rq, qo == kOutOfRange ? kOutOfRange : qo + (uint32_t)(i * 32 * a.Ncols), 0, 0);
  };
  DropKey dk{};
  const bool dropping = DROP && a.drop.thr != 0;
  if constexpr (DROP)
    if (dropping) dk = drop_key(a.drop);
  const uint64_t call0 = (uint64_t)qr * (uint64_t)(a.Ncols / 8) + (uint64_t)(c0 / 8 + qu);
  auto store_q = [&](int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DROP) {
        if (dropping) {
          uint32_t w[4];
          philox7(call0 + (uint64_t)((int64_t)s * 64 + 16 * i) * (uint64_t)(a.Ncols / 8), dk, w);
          qv[i] &= u32x4{keep_mask2(w[0], dk.thr2), keep_mask2(w[1], dk.thr2), keep_mask2(w[2], dk.thr2),
                         keep_mask2(w[3], dk.thr2)};
        }
      }
      *reinterpret_cast<u32x4 *>(qs + qst + 8192 * i) = qv[i];
    }
  };
  // L: direct load g covers stage rows 8 g .. + 7, 64 rows of Q (128 bytes); RT per
  // wave.  Stage rows 0 .. 32 RT - 1 are the first piece's ranks, the others the
  // second's; ranks from R on are out of range and come as zeros.
  const int lj = 8 * RT * wave + (lane >> 3);
  uint32_t lo[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int j = lj + 8 * i, rank = j & (32 * RT - 1), piece = j / (32 * RT);
    lo[i] = rank < a.R ? (uint32_t)((piece * a.R + rank) * a.Mp * 2 + 16 * ((lane & 7) ^ ((j >> 1) & 7))) : kOutOfRange;
  }
  auto issue_l = [&](uint8_t *dst, int s) {
    const rsrc_t rl = make_rsrc_u(a.Lt + (int64_t)s * 64, (2 * a.R * a.Mp - (int64_t)s * 64) * 2);
#pragma unroll
    for (int i = 0; i < RT; ++i)
      load_lds16(rl, (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(dst)) + (wave * RT + i) * 1024, lo[i], 0);
  };

  f32x16 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[t][e] = 0.0f;
  // Fragments of sub-step c: lane half h takes rows 32 h + 8 c .. + 7.
  // A lane of a transposing read points at row (lane % 16) / 4 of four, columns
  // 4 (lane % 4) of its group's 16; rows 8 c + 4 p on add whole rows.
  uint32_t fl[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) fl[c] = (uint32_t)(lr * 128 + 16 * ((4 * lh + c) ^ ((lr >> 1) & 7)));
  const int tr = (lane & 15) >> 2, tc = 32 * wave + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const uint32_t fq = (uint32_t)((32 * lh + tr) * 512 + 16 * ((tc >> 3) ^ (4 * tr)) + 2 * (tc & 7));
  auto multiply = [&](const uint8_t *l) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bf16x8 b = read_transposed(qs + fq + c * 4096, qs + fq + c * 4096 + 2048);
      const bf16x8 bf = finite_or_zero(b);
#pragma unroll
      for (int t = 0; t < 2 * RT; ++t)
        acc[t % RT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            *reinterpret_cast<const bf16x8 *>(l + t * 32 * 128 + fl[c]), t < RT ? b : bf, acc[t % RT], 0, 0, 0);
    }
  };

  // Step s: L's stage of step s + 1 is asked for; Q's stage is multiplied; between
  // the barriers it is refilled with step s + 1 from registers, and step s + 2 is
  // requested.  Those four loads stay in flight across the second barrier,
  // which waits for L's direct loads, issued before them.
  const int last = s1 - 1;
  auto step = [&](int s, const uint8_t *l, uint8_t *ln) {
    issue_l(ln, min(s + 1, last));
    __builtin_amdgcn_sched_barrier(0);
    multiply(l);
    stage_barrier<15>();   // reads of the stage are done; any number of loads in flight
    store_q(min(s + 1, last));
    __builtin_amdgcn_sched_barrier(0);
    load_q(min(s + 2, last));
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier<4>();
  };
  if (s0 < s1) {
    load_q(s0);
    issue_l(ls0, s0);
    store_q(s0);
    __builtin_amdgcn_sched_barrier(0);
    load_q(min(s0 + 1, last));
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier<4>();
    for (int s = s0; s < s1; s += 2) {
      step(s, ls0, ls1);
      if (s + 1 >= s1) break;
      step(s + 1, ls1, ls0);
    }
  }
  // The direct loads past the end have landed (the last barrier waited for
  // them); the four of Q still on their way write registers that no one reads.
  // acc[t][e]: rank 32 t + 8 (e / 4) + 4 lh + e % 4, column c0 + 32 wave + lr.
  const int64_t col = c0 + 32 * wave + lr;
  float *part = a.part + (int64_t)split * a.R * a.Ncols;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int j = 32 * t + 8 * (e >> 2) + 4 * lh + (e & 3);
      if (j < a.R && col < a.Ncols) part[(int64_t)j * a.Ncols + col] = acc[t][e];
    }
}

__global__ __launch_bounds__(256) void colsum_reduce_kernel(ColSumArgs a0, ColSumArgs a1) {
  __shared__ float tile[64 * 17];
  colsum_reduce(blockIdx.y ? a1 : a0, (int)blockIdx.x, tile);
}

}  // namespace

// Enough ranges for about two workgroups per CU over the call's two sums
// (`cols` columns between them), at least 128 rows each and at most 16.
int colsum_splits(int64_t M, int64_t cols) {
  const int64_t tiles = (cols + CS_COLS - 1) / CS_COLS;
  const int64_t want = (2 * device_cus() + tiles - 1) / tiles;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, 16), (M + 127) / 128));
}

hipError_t launch_colsum2(const ColSumArgs &a, const ColSumArgs &b, hipStream_t st, int trace_kind) {
  const int64_t ncols = std::max(a.Ncols, b.Ncols), R = std::max(a.R, b.R);
  const dim3 grid((unsigned)((ncols + CS_COLS - 1) / CS_COLS), (unsigned)a.splits, 2u), block(CS_THREADS);
  {
    TraceScope tr(trace_kind, st);
    const bool drop = a.drop.thr || b.drop.thr;
    if (R <= 32) {
      if (drop) hipLaunchKernelGGL((colsum_kernel<1, true>), grid, block, 0, st, a, b);
      else hipLaunchKernelGGL((colsum_kernel<1, false>), grid, block, 0, st, a, b);
    } else {
      if (drop) hipLaunchKernelGGL((colsum_kernel<2, true>), grid, block, 0, st, a, b);
      else hipLaunchKernelGGL((colsum_kernel<2, false>), grid, block, 0, st, a, b);
    }
  }
  return hipGetLastError();
}

hipError_t launch_colsum_reduce(const ColSumArgs &a, const ColSumArgs &b, hipStream_t st) {
  const dim3 grid((unsigned)std::max(colsum_reduce_blocks(a), colsum_reduce_blocks(b)), 2u);
  hipLaunchKernelGGL(colsum_reduce_kernel, grid, dim3(256), 0, st, a, b);
  return hipGetLastError();
}

}  // namespace qn
