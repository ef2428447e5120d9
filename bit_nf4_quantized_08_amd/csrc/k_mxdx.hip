// dX of the MXFP4 linear on gfx950: dX[M, K] = G[M, N] bf16(W[N, K]) + c keep *
// (dH[M, r] A[r, K]).
//
// The contraction runs down the weight's rows, across its blocks, so the
// block scales cannot ride on the matrix instruction: each 64-row step
// expands a 64 x 256 patch of codes to bf16 (exact, v_cvt_scalef32_pk_bf16_fp4)
// into LDS as it lies, and the fragments, which need eight consecutive
// contraction rows of one column, come back through the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes point at 4 rows x 16 columns and receive 16
// columns x 4 rows).  Bound by the bf16 matrix rate at the clock it sustains:
// 4096 x 8192 x 8192, r = 64, p = 0.05: 420 to 465 us as the card's clock has it, 1.2
// to 1.3 PFLOP/s, matrix pipes busy 63 % of the cycles at about 1.9 GHz, LDS a third;
// a dense bf16 library product of that shape, weights ready in bf16, takes 408 us.
//
// A workgroup of 8 waves owns a (32 TM WR) x 256 tile of dX: one chunk of the
// weight's columns, so a step's scale bytes are 512 contiguous bytes.  Step s
// multiplies stage s & 1 while G of step s + 1 goes to the other stage by
// direct-to-LDS loads and the codes of step s + 1, loaded during step s - 1, are
// expanded into it.
//
// Expanded stage: row n (pitch 544 bytes, 32 past the banks' turn of 256: the eight
// 32-byte pieces of 32 lanes' transposing reads, four rows at two places 128
// bytes apart, fall on different banks; with 576 two of the rows met, 18 M
// conflict cycles against 0.7 M), 16-byte units of 8 columns.  Thread (n, ch)
// expands one block, columns 32 ch .. +31, as four units q = 0..3; unit (ch, q)
// sits at slot 8 q + ch, so that the eight lanes of a write cycle store 128
// contiguous bytes.  A wave's columns are the units ch = UW wc .. + UW - 1 for all q (UW =
// 8 / WC): 32 UW consecutive columns of dX.  "Tile column" x of a wave is unit
// (q, u) = (x / 8 / UW, x / 8 % UW).
//
// dH enters in one bf16 piece: its rounding is 2^-8 of each product of the adapter
// term at most, as the result's is of dX (error against 64 bits at 4096 x 8192 x 8192:
// 0.0017 of dX's norm, that of a bf16 result formed in fp32).
//
// G's stage is swizzled in 16-byte pieces as in the forward: piece k of row r
// at slot k ^ ((r >> 1) & 7).  Contraction order: in sub-step c of a step, lane
// half h supplies rows 32 h + 8 c .. + 7 of both operands.

#include <algorithm>

#include "qn_colsum.h"
#include "qn_philox.h"
#include "qn_tile.h"

namespace qn {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kRowPitch = 544;           // bytes per expanded row
constexpr int kWStage = 64 * kRowPitch;  // bytes per expanded stage

template <int TM, int TN, int WR, int WC, bool DROP, bool PART>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void mx_dx_kernel(MxDxArgs a, int tiles_m, int tiles_n, int group_m) {
  static_assert(WR * WC == 8 && TN * WC == 8, "8 waves over 256 columns");
  constexpr int BM = 32 * TM * WR, UW = 8 / WC;
  constexpr int GL = BM / 64;   // direct loads (8 rows each) per wave and step
  static_assert(GL >= 1 && GL <= 4, "stage loads");
  constexpr int kPitch = 32 * TN + 8;   // bf16 per row of a store block
  __shared__ __attribute__((aligned(16))) uint8_t gs0[BM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t gs1[BM * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ws0[kWStage];
  __shared__ __attribute__((aligned(16))) uint8_t ws1[kWStage];
  __shared__ uint32_t keep[DROP ? BM * 8 : 1];   // the tile's mask (make_mask)

  int tm, tn;
  xcd_tile((int)blockIdx.x, tiles_m, tiles_n, group_m, tm, tn);
  const int split = (int)blockIdx.y;
  const int64_t m0 = (int64_t)tm * BM, k0 = (int64_t)tn * 256;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave % WR, wc = wave / WR;
  const int steps = (int)(a.N / 64), s0 = (int)((int64_t)steps * split / a.splits),
            s1 = (int)((int64_t)steps * (split + 1) / a.splits);

  // G: load g covers rows 8g .. 8g + 7, 64 columns (128 bytes).
  const rsrc_t rg = make_rsrc_u(a.G + m0 * a.N, (a.M - m0) * a.N * 2);
  uint32_t go[GL];
#pragma unroll
  for (int i = 0; i < GL; ++i) {
    const int row = 8 * (wave * GL + i) + (lane >> 3);
    go[i] = (uint32_t)(row * a.N * 2 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
  }
  auto issue_g = [&](uint8_t *dst, int s, int i) {
    load_lds16(rg, (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_offset(dst)) + wave * GL * 1024 + i * 1024, go[i], s * 128);
  };
  // W: thread (n, ch) of a step.
  const int64_t C = (a.K + 255) / 256, pitch = 128 * C;
  const int wn = tid >> 3, ch = tid & 7;
  const rsrc_t rw = make_rsrc_u(a.codes + tn * 128, a.N * pitch - tn * 128);
  const rsrc_t rs = make_rsrc_u(a.scales + (int64_t)tn * a.N * 8, a.N * 8);
  const uint32_t wo = (uint32_t)(wn * pitch + 16 * ch);
  struct Set {
    u32x4 code;
    uint32_t sb;
  };
  auto load_w = [&](Set &t, int s) {
    t.code = __builtin_amdgcn_raw_buffer_load_b128(rw, wo, (int)(s * 64 * pitch), 0);
    t.sb = __builtin_amdgcn_raw_buffer_load_b8(rs, (uint32_t)tid, s * 512, 0);
  };
  uint32_t wst = (uint32_t)(wn * kRowPitch + 16 * ch);
  auto expand = [&](const Set &t, int q, uint8_t *dst) {
    const float sc = as_f32(t.sb << 23);
    const uint32_t cw[4] = {t.code.x, t.code.y, t.code.z, t.code.w};
    u32x4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[q], sc, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[q], sc, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[q], sc, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[q], sc, 3));
    if (t.sb == 255u) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    *reinterpret_cast<u32x4 *>(dst + wst + 128 * q) = o;
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // Fragments.  G: row lr of a tile, piece 4 lh + c.  W: 16 tile columns per
  // group of 16 lanes; a lane points at row (lane % 16) / 4, columns 4 (lane % 4).
  uint32_t fg[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) fg[c] = (uint32_t)((wr * 32 * TM + lr) * 128 + 16 * ((4 * lh + c) ^ ((lr >> 1) & 7)));
  uint32_t fw[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int g16 = 2 * j + ((lane >> 4) & 1), q = 2 * g16 / UW, u = 2 * g16 % UW;
    const int scol = 64 * q + 8 * (UW * wc + u);
    fw[j] = (uint32_t)((32 * lh + ((lane & 15) >> 2)) * kRowPitch + (scol + 4 * (lane & 3)) * 2);
  }
  auto read_g = [&](const uint8_t *gst, int i, int c) {
    return *reinterpret_cast<const bf16x8 *>(gst + fg[c] + i * 32 * 128);
  };
  auto read_w = [&](const uint8_t *wst_, int j, int c) {
    const uint8_t *b = wst_ + fw[j] + c * 8 * kRowPitch;
    return read_transposed(b, b + 4 * kRowPitch);
  };
  // Step s: stage (s - s0) & 1; past the end the last step is loaded again.  On
  // entry f0 holds sub-step 0's fragments.  Fragments are read a sub-step ahead,
  // the next stage's codes are expanded with the first three sub-steps' MFMAs,
  // and the barrier comes when the last fragments are in registers: the next
  // stage's first fragments are read, and G of the step after asked for, under
  // the last sub-step's MFMAs.  The two loads of W are the last issued before
  // the barrier and stay in flight across it.
  const int last = s1 - 1;
  struct Frag {
    bf16x8 a[TM], b[TN];
  };
  auto read_f = [&](Frag &f, const uint8_t *gst, const uint8_t *wst_, int c) {
#pragma unroll
    for (int i = 0; i < TM; ++i) f.a[i] = read_g(gst, i, c);
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = read_w(wst_, j, c);
  };
  // The mask of the tile, BM x 256 bits, one generator call to a byte: row R's byte
  // 8 w + n holds tile columns 8 n .. + 7 of the waves wc = w.  Call c of the
  // workgroup, thread t's k-th (c = 512 k + t, k < kCalls), is byte c % 32 of row
  // c / 32.  The calls run under the main loop, one a step while they last, in
  // four parts between the third sub-step's MFMAs; run after it, before the
  // masked add, they cost what the matrix cores then wait (4096 rows: N = 512, K =
  // 8192 61 against 55 us, N = 3584, K = 18944 493 against 478; nothing at 8192 x 8192,
  // where the clock takes the gain back).
  constexpr int kCalls = BM / 16;
  DropKey dk{};
  if constexpr (DROP) dk = drop_key(a.drop);
  const int byte = tid & 31, unit = byte & 7;
  const uint64_t call0 = (uint64_t)(m0 + (tid >> 5)) * (uint64_t)(a.K / 8) +
                         (uint64_t)(k0 / 8 + 4 * (UW * (byte >> 3) + unit % UW) + unit / UW);
  Philox ph;
  int calls = 0;
  auto make_mask = [&](int q) {
    if (q == 0) ph.start(call0 + (uint64_t)(16 * calls) * (uint64_t)(a.K / 8), dk);
    ph.rounds<2>(dk, 2 * q);   // 2, 2, 2 and 1 of the seven
    if (q == 3) {
      reinterpret_cast<uint8_t *>(keep)[512 * calls + tid] = (uint8_t)keep_bits8(ph.c, dk.thr2);
      ++calls;
    }
  };
  // A sub-step's MFMAs, with hook(0) .. hook(3) spread between them.
  auto mma = [&](const Frag &f, auto &&hook) {
    constexpr int n = TM * TN, per = n >= 4 ? n / 4 : 1;
#pragma unroll
    for (int m = 0; m < n; ++m) {
      const int i = m / TN, j = m % TN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
      if (m % per == per - 1) {
        __builtin_amdgcn_sched_barrier(0);
        hook(n < 4 ? 2 * m : m / per);
        if (n < 4) hook(2 * m + 1);   // two MFMAs: two hooks after each
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto step = [&](int s, uint8_t *gc, const uint8_t *wc_, const uint8_t *gn, uint8_t *wn_, Frag &f0, Frag &f1,
                  const Set &t, Set &t2, auto &&third) {
    Set nt;
    read_f(f1, gc, wc_, 1);
    __builtin_amdgcn_sched_barrier(0);
    mma(f0, [&](int q) {
      if (q == 0) load_w(nt, min(s + 2, last));
      if (q == 1) expand(t, 0, wn_);
      if (q == 3) expand(t, 1, wn_);
    });
    read_f(f0, gc, wc_, 2);
    __builtin_amdgcn_sched_barrier(0);
    mma(f1, [&](int q) {
      if (q == 1) expand(t, 2, wn_);
      if (q == 3) expand(t, 3, wn_);
    });
    read_f(f1, gc, wc_, 3);
    __builtin_amdgcn_sched_barrier(0);
    mma(f0, third);
    t2 = nt;
    stage_barrier<2>();
    read_f(f0, gn, wn_, 0);
    __builtin_amdgcn_sched_barrier(0);
    mma(f1, [&](int q) {
      if (q < GL) issue_g(gc, min(s + 2, last), q);
    });
  };
  Set t0, t1;
  load_w(t0, s0);
#pragma unroll
  for (int i = 0; i < GL; ++i) issue_g(gs0, s0, i);
  __builtin_amdgcn_sched_barrier(0);
  load_w(t1, min(s0 + 1, last));
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int q = 0; q < 4; ++q) expand(t0, q, ws0);
  stage_barrier<2>();
  Frag f0, f1;
#pragma unroll
  for (int i = 0; i < GL; ++i) issue_g(gs1, min(s0 + 1, last), i);
  __builtin_amdgcn_sched_barrier(0);
  read_f(f0, gs0, ws0, 0);
  int s = s0;
  const bool masked = DROP && a.r && (!PART || split == 0);   // of split products, the first carries the adapter
  if constexpr (DROP)
    if (masked)
      for (; s + 1 < s1 && calls < kCalls; s += 2) {
        step(s, gs0, ws0, gs1, ws1, f0, f1, t1, t0, make_mask);
        step(s + 1, gs1, ws1, gs0, ws0, f0, f1, t0, t1, make_mask);
      }
  auto none = [](int) {};
  for (; s < s1; s += 2) {
    step(s, gs0, ws0, gs1, ws1, f0, f1, t1, t0, none);
    if (s + 1 >= s1) break;
    step(s + 1, gs1, ws1, gs0, ws0, f0, f1, t0, t1, none);
  }
  if constexpr (DROP)
    if (masked)
      while (calls < kCalls)   // short contractions leave some
#pragma unroll
        for (int q = 0; q < 4; ++q) make_mask(q);
  // The loads past the end must land, and the last reads past it end, before the
  // stages are written again.
  stage_barrier();

  const int64_t row0 = m0 + wr * 32 * TM, colw = k0 + 32 * UW * wc;   // the wave's first row and column
  // dX column (from k0) of the wave's tile column x.
  auto col_of = [&](int x) {
    const int un = x >> 3, q = un / UW, u = un % UW;
    return 32 * (UW * wc + u) + 8 * q + (x & 7);
  };
  // Adapter term: A as an expanded stage (rows j < r, zero beyond), dH's
  // fragments from global memory.  Every wave has passed the last barrier, so
  // ws0 is free.
  if (a.r && (!PART || split == 0)) {   // of split products, the first carries it
    {
      const rsrc_t ra = make_rsrc_u(a.A, a.r * a.K * 2);
      const int64_t col = k0 + 32 * ch;
      u32x4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = __builtin_amdgcn_raw_buffer_load_b128(
            ra, wn < a.r && col < a.K ? (uint32_t)((wn * a.K + col + 8 * q) * 2) : kOutOfRange, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<u32x4 *>(ws0 + wst + 128 * q) = v[q];
    }
    const rsrc_t rh = make_rsrc_u(a.dHb + row0 * a.ldh, (a.M - row0) * a.ldh * 2);
    bf16x8 fa[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = 32 * lh + 8 * c;
        fa[i][c] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rh, j < a.ldh ? (uint32_t)(((32 * i + lr) * a.ldh + j) * 2) : kOutOfRange, 0, 0));
      }
    __syncthreads();
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const uint32_t row = keep[(wr * 32 * TM + 32 * i + lr) * 8 + wc * TN + j];   // of lane lr and lr + 32
          f32x16 t;
#pragma unroll
          for (int e = 0; e < 16; ++e) t[e] = 0.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c) t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i][c], read_w(ws0, j, c), t, 0, 0, 0);
          add_kept(acc[i][j], t, a.drop.c, row);
        }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const bf16x8 fb = read_w(ws0, j, c);
#pragma unroll
          for (int i = 0; i < TM; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i][c], fb, acc[i][j], 0, 0, 0);
        }
    }
  }

  if constexpr (PART) {
    float *part = a.part + (int64_t)split * a.M * a.K;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int64_t k = k0 + col_of(32 * j + lr);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int64_t m = row0 + 32 * i + 8 * (e >> 2) + 4 * lh + (e & 3);
          if (m < a.M && k < a.K) part[m * a.K + k] = acc[i][j][e];
        }
      }
    return;
  }

  // Store through LDS: each wave turns its 32-row blocks into whole 16-byte
  // pieces of dX's rows.  ws1 (the stages of G too) is no longer read; ws0 may
  // still be (adapter), so the blocks lie in ws1, gs0 and gs1.
  constexpr int kBlock = 32 * kPitch * 2;   // bytes
  constexpr int kInW = kWStage / kBlock, kInG = BM * 128 / kBlock;
  static_assert(kInW + 2 * kInG >= 8, "store blocks fit");
  uint16_t *blk = reinterpret_cast<uint16_t *>(wave < kInW ? ws1 + wave * kBlock
                                               : wave < kInW + kInG ? gs0 + (wave - kInW) * kBlock
                                                                    : gs1 + (wave - kInW - kInG) * kBlock);
  const rsrc_t rout = make_rsrc_u(a.dX + m0 * a.K, (a.M - m0) * a.K * 2);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        blk[(8 * (e >> 2) + 4 * lh + (e & 3)) * kPitch + j * 32 + lr] = f32_to_bf16(acc[i][j][e]);
    constexpr int kPieces = 4 * TN, kRows = 64 / kPieces;   // pieces per row, rows per store
#pragma unroll
    for (int p = 0; p < 32 / kRows; ++p) {
      const int row = kRows * p + lane / kPieces, t = lane % kPieces, q = t & 3, u = t >> 2;
      const u32x4 v = *reinterpret_cast<const u32x4 *>(&blk[row * kPitch + 8 * (UW * q + u)]);
      const int64_t lrow = wr * 32 * TM + 32 * i + row, k = colw + 8 * t;
      __builtin_amdgcn_raw_buffer_store_b128(v, rout, k < a.K ? (uint32_t)((lrow * a.K + k) * 2) : kOutOfRange, 0, 0);
    }
  }
}

// out = bf16(sum of the splits' partial products), one thread per 8 of its n
// elements (dX, and the NF4 linear's split products).  The workgroups past
// out's (`blocks`) reduce the call's two column sums: launches are what a small
// call costs.
__global__ __launch_bounds__(256) void split_sum_kernel(const float *part, int splits, int64_t n, uint16_t *out,
                                                        ColSumArgs c0, ColSumArgs c1, int blocks) {
  __shared__ float tile[64 * 17];
  if ((int)blockIdx.x >= blocks) {
    const int b = (int)blockIdx.x - blocks, n0 = (int)colsum_reduce_blocks(c0);
    colsum_reduce(b < n0 ? c0 : c1, b < n0 ? b : b - n0, tile);
    return;
  }
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= n) return;
  f32x4 v0 = {0.0f, 0.0f, 0.0f, 0.0f}, v1 = v0;
  for (int q0 = 0; q0 < splits; q0 += 4) {   // four loads at a time, past the last one again
    f32x4 x[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 *p = reinterpret_cast<const f32x4 *>(part + (int64_t)min(q0 + q, splits - 1) * n + i);
      x[q][0] = p[0];
      x[q][1] = p[1];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q0 + q < splits) {
        v0 += x[q][0];
        v1 += x[q][1];
      }
  }
  *reinterpret_cast<u32x4 *>(out + i) = u32x4{pack_bf16x2(v0[0], v0[1]), pack_bf16x2(v0[2], v0[3]),
                                             pack_bf16x2(v1[0], v1[1]), pack_bf16x2(v1[2], v1[3])};
}

// Rows of the tiles and cuts of the contraction, by the time of a launch: rounds
// of workgroups over the CUs (one fits each) times a step's time (64 rows of W,
// measured at 8192 x 8192) times the steps, and for cuts the partial products'
// way to memory and back at 4.5 TB/s (their launch is there anyway: it reduces
// the column sums too).
struct DxPlan {
  int rows, splits;
};
DxPlan dx_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t cus = device_cus(), cols = cdiv(K, 256), steps = N / 64;
  const struct { int rows; double us; } tile[3] = {{256, 1.62}, {128, 0.95}, {64, 0.62}};
  DxPlan p{256, 1};
  double best = 1e300;
  for (const auto &t : tile)
    for (int s = 1; s <= 8 && (s == 1 || steps / s >= 4); ++s) {
      const double us = t.us * (double)cdiv(cdiv(M, t.rows) * cols * s, cus) * (double)cdiv(steps, s) +
                        (s == 1 ? 0.0 : 0.5 + (double)(s * M * K) * 8.0 / 4.5e6);
      if (us < best) { best = us; p = DxPlan{t.rows, s}; }
    }
  return p;
}

template <int TM, int TN, int WR, int WC>
hipError_t launch_tiles(const MxDxArgs &a, hipStream_t st) {
  const int tiles_m = (int)cdiv(a.M, 32 * TM * WR), tiles_n = (int)cdiv(a.K, 256);
  const int64_t T = (int64_t)tiles_m * tiles_n;
  if (T > INT32_MAX) return hipErrorInvalidValue;
  const int gm = std::max(1, std::min(tiles_m, 4));
  const dim3 grid((unsigned)T, (unsigned)a.splits), block(512);
  TraceScope tr(QN_TRACE_MX_DX, st);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a, tiles_m, tiles_n, gm); };
  if (a.splits > 1) {
    if (a.drop.thr) go(mx_dx_kernel<TM, TN, WR, WC, true, true>);
    else go(mx_dx_kernel<TM, TN, WR, WC, false, true>);
  } else {
    if (a.drop.thr) go(mx_dx_kernel<TM, TN, WR, WC, true, false>);
    else go(mx_dx_kernel<TM, TN, WR, WC, false, false>);
  }
  return hipGetLastError();
}

}  // namespace

size_t mx_dx_part_bytes(int64_t M, int64_t N, int64_t K) {
  const DxPlan p = dx_plan(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)K * sizeof(float) : 0;
}

hipError_t launch_mx_dx(const MxDxArgs &in, const ColSumArgs *sums, hipStream_t st) {
  MxDxArgs a = in;
  const DxPlan p = dx_plan(a.M, a.N, a.K);
  a.splits = p.splits;
  const hipError_t e = p.rows == 256   ? launch_tiles<4, 2, 2, 4>(a, st)
                       : p.rows == 128 ? launch_tiles<2, 2, 2, 4>(a, st)
                                       : launch_tiles<1, 2, 2, 4>(a, st);
  if (e != hipSuccess) return e;
  if (p.splits == 1) return sums ? launch_colsum_reduce(sums[0], sums[1], st) : hipSuccess;
  return launch_split_sum(a.part, p.splits, a.M * a.K, a.dX, sums, st);
}

hipError_t launch_split_sum(const float *part, int splits, int64_t n, uint16_t *out, const ColSumArgs *sums,
                            hipStream_t st) {
  const int blocks = (int)cdiv(n / 8, 256);
  const ColSumArgs none{};
  const int64_t more = sums ? colsum_reduce_blocks(sums[0]) + colsum_reduce_blocks(sums[1]) : 0;
  hipLaunchKernelGGL(split_sum_kernel, dim3((unsigned)(blocks + more)), dim3(256), 0, st, part, splits, n, out,
                     sums ? sums[0] : none, sums ? sums[1] : none, blocks);
  return hipGetLastError();
}

}  // namespace qn
