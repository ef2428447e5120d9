// Reduction of the column sums over their row ranges (gfx950), shared by its own
// kernel and the finishing pass of the MXFP4 dX.
#pragma once

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {

// Workgroups (256 threads) of one reduction: 64 columns x 16 ranks each.
__host__ __device__ inline int64_t colsum_reduce_blocks(const ColSumArgs &a) {
  return a.Ncols / 64 * ((a.R + 15) / 16);   // Ncols % 64 == 0
}

// out = bf16(c * sum of the ranges, in order), as [R][Ncols] or transposed
// [Ncols][R]: read along the columns, stored along whichever is contiguous,
// through LDS (64 * 17 floats).
__device__ __forceinline__ void colsum_reduce(const ColSumArgs &a, int block, float *tile) {
  if (block >= colsum_reduce_blocks(a)) return;
  const int jb = (int)((a.R + 15) / 16);
  const int64_t c0 = (int64_t)(block / jb) * 64;
  const int tid = threadIdx.x, cl = tid & 63, j0 = block % jb * 16, j1 = min((int)a.R, j0 + 16), w = j1 - j0;
  const int64_t stride = a.R * a.Ncols;
  // A thread's four ranks (every fourth of the workgroup's, past the last one
  // that again) and eight ranges at a time: 32 loads on their way, not eight.
  const int jw = j0 + (tid >> 6);
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int q0 = 0; q0 < a.splits; q0 += 8) {
    float x[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float *p = a.part + (int64_t)min(jw + 4 * i, j1 - 1) * a.Ncols + c0 + cl;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[i][q] = p[(int64_t)min(q0 + q, a.splits - 1) * stride];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q0 + q < a.splits) v[i] += x[i][q];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = jw + 4 * i;
    if (j >= j1) continue;
    if (a.transpose) tile[cl * 17 + j - j0] = v[i] * a.drop.c;
    else a.out[(int64_t)j * a.Ncols + c0 + cl] = f32_to_bf16(v[i] * a.drop.c);
  }
  if (!a.transpose) return;
  __syncthreads();
  for (int i = tid; i < 64 * w; i += 256) a.out[(c0 + i / w) * a.R + j0 + i % w] = f32_to_bf16(tile[i / w * 17 + i % w]);
}

}  // namespace qn
