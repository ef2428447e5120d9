// Element-wise counter-based dropout on gfx950:
//   y[i] = keep(i) ? round(x[i] * c) : 0,  c = fl32(1 / (1 - thr / 65536)).
// The mask comes from the generator of qn_philox.h and is not stored; the
// same call on a gradient is the backward.
//
// Eight elements (one generator call) per thread: a 16-byte load and store for
// bf16, two for fp32.  Memory bound with a second limit close by: one generator
// call is 14 quarter-rate multiplies and about 50 other vector instructions.  4096 x
// 8192 bf16 (134 MB, part of it in the 256 MB cache): 19.7 us, 6.8 TB/s; a plain copy
// takes 17 to 19.  Two or four groups per thread, loads first, take 20.7 and 21.2;
// fp32 in one 16-byte piece per lane, each call made by two neighbours, 48 against
// 42 at 33.5 M elements; stores marked as not read again gain here (134 M
// elements: 89 -> 74) what the reader of y then loses.

#include "qn_philox.h"

namespace qn {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGridX = 1 << 22;

template <bool BF16, bool DROP>
__device__ __forceinline__ void drop8(const DropArgs &d, const DropKey &k, uint64_t g, const u32x4 (&x)[BF16 ? 1 : 2],
                                      u32x4 (&y)[BF16 ? 1 : 2]) {
  uint32_t m[4] = {~0u, ~0u, ~0u, ~0u};
  if constexpr (DROP) {
    uint32_t w[4];
    philox7(g, k, w);
#pragma unroll
    for (int t = 0; t < 4; ++t) m[t] = keep_mask2(w[t], k.thr2);
  }
  if constexpr (BF16) {
    const uint32_t v[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
    uint32_t o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = pack_bf16x2(bf16_lo(v[t]) * d.c, bf16_hi(v[t]) * d.c) & m[t];
    y[0] = u32x4{o[0], o[1], o[2], o[3]};
  } else {
    const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t o[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t r = as_u32(as_f32(v[t]) * d.c);
      o[t] = (m[t >> 1] >> (16 * (t & 1))) & 1u ? r : 0u;
    }
    y[0] = u32x4{o[0], o[1], o[2], o[3]};
    y[1] = u32x4{o[4], o[5], o[6], o[7]};
  }
}

template <bool BF16, bool DROP>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const uint8_t *x, uint8_t *y, int64_t n, DropArgs d) {
  constexpr int V = BF16 ? 1 : 2;
  constexpr int ES = BF16 ? 2 : 4;
  const DropKey k = drop_key(d);
  const int64_t full = n >> 3, g = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  u32x4 xv[V], yv[V];
  if (g < full) {
#pragma unroll
    for (int v = 0; v < V; ++v) xv[v] = *reinterpret_cast<const u32x4 *>(x + g * 8 * ES + 16 * v);
    drop8<BF16, DROP>(d, k, (uint64_t)g, xv, yv);
#pragma unroll
    for (int v = 0; v < V; ++v) *reinterpret_cast<u32x4 *>(y + g * 8 * ES + 16 * v) = yv[v];
  } else if (g == full && (n & 7)) {   // the last, partial group
    const int left = (int)(n & 7);
    uint32_t e[4 * V] = {};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= left) break;
      if constexpr (BF16) e[t >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(x)[g * 8 + t] << (16 * (t & 1));
      else e[t] = reinterpret_cast<const uint32_t *>(x)[g * 8 + t];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) xv[v] = u32x4{e[4 * v], e[4 * v + 1], e[4 * v + 2], e[4 * v + 3]};
    drop8<BF16, DROP>(d, k, (uint64_t)g, xv, yv);
    uint32_t o[4 * V];
#pragma unroll
    for (int v = 0; v < V; ++v) { o[4 * v] = yv[v].x; o[4 * v + 1] = yv[v].y; o[4 * v + 2] = yv[v].z; o[4 * v + 3] = yv[v].w; }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t >= left) break;
      if constexpr (BF16) reinterpret_cast<uint16_t *>(y)[g * 8 + t] = (uint16_t)(o[t >> 1] >> (16 * (t & 1)));
      else reinterpret_cast<uint32_t *>(y)[g * 8 + t] = o[t];
    }
  }
}

}  // namespace

hipError_t launch_dropout(const void *x, int is_bf16, int64_t n, const DropArgs &d, void *y, hipStream_t st) {
  // A grid dimension holds less than 2^32 threads (n <= 2^40 needs up to 2^37).
  const int64_t blocks = ((n + 7) / 8 + kThreads - 1) / kThreads, wide = blocks < kMaxGridX ? blocks : kMaxGridX;
  const dim3 grid((unsigned)wide, (unsigned)((blocks + wide - 1) / wide));
  const auto *xs = static_cast<const uint8_t *>(x);
  auto *ys = static_cast<uint8_t *>(y);
  TraceScope tr(QN_TRACE_DROPOUT, st);
  if (is_bf16) {
    if (d.thr) hipLaunchKernelGGL((dropout_kernel<true, true>), grid, dim3(kThreads), 0, st, xs, ys, n, d);
    else hipLaunchKernelGGL((dropout_kernel<true, false>), grid, dim3(kThreads), 0, st, xs, ys, n, d);
  } else {
    if (d.thr) hipLaunchKernelGGL((dropout_kernel<false, true>), grid, dim3(kThreads), 0, st, xs, ys, n, d);
    else hipLaunchKernelGGL((dropout_kernel<false, false>), grid, dim3(kThreads), 0, st, xs, ys, n, d);
  }
  return hipGetLastError();
}

}  // namespace qn
