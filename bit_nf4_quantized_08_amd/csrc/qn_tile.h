// Pieces shared by the MXFP4 tile kernels (gfx950).
#pragma once

#include "qn_device.h"

namespace qn {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef int i32x8 __attribute__((ext_vector_type(8)));
constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;  // a per-lane offset that always reads zero

// Wave-uniform buffer resource over [base, base + bytes); accesses whose per-lane
// offset lies beyond `bytes` read zero and store nothing.  A scalar offset is not
// counted on to take part in that check: where one is used, every lane's offset is
// out of range by itself or inside together with it.
__device__ __forceinline__ rsrc_t make_rsrc_u(const void *base, int64_t bytes) {
  const int64_t cap = 0xFFFFFFF0LL;
  const uint64_t p = (uint64_t)base;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)(uint32_t)(bytes < 0 ? 0 : (bytes > cap ? cap : bytes)));
  return __builtin_amdgcn_make_buffer_rsrc((void *)(((uint64_t)hi << 32) | lo), (short)0, n, 0x00020000);
}

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// 16 bytes per lane from global memory straight to LDS: lane l's bytes land at
// lds + 16 l (lds wave-uniform).
__device__ __forceinline__ void load_lds16(rsrc_t r, uint32_t lds, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(size_t)lds, 16, voff, soff,
                                           0, 0);
}

// Barrier that publishes a stage: before it arrives, the wave's LDS accesses are
// done and all but the last IN_FLIGHT of its global loads (direct-to-LDS loads
// among them) have landed.  The loads that may stay in flight must be the last
// ones issued (fenced from the scheduler); asm, because a compiler's own
// workgroup fence would wait for them too.
template <int IN_FLIGHT = 0>
__device__ __forceinline__ void stage_barrier() {
  static_assert(IN_FLIGHT < 16, "low bits of vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | IN_FLIGHT);   // vmcnt(IN_FLIGHT), lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// Transposing LDS read: 16 lanes point at 4 rows x 16 columns of 16-bit values (8
// bytes each) and receive 16 columns x 4 rows.  The pointer keeps its array, so
// that the compiler does not take the read for one of another stage's bytes
// and wait for the loads on their way there.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8 read_transposed(const uint8_t *lo, const uint8_t *hi) {
  typedef __attribute__((address_space(3))) s16x4 *lds4;
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(__attribute__((address_space(3))) uint8_t *)lo);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(__attribute__((address_space(3))) uint8_t *)hi);
  return __builtin_bit_cast(bf16x8, (s16x8){x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w});
}

// Tile of workgroup h: workgroups are dealt round-robin to the 8 XCDs, so XCD x
// gets the contiguous run of logical tiles x T/8 .. of an order that walks
// groups of gm row tiles column by column; the workgroups that share an L2 then
// share row and column panels.  (T not a multiple of 8: the remainder goes to
// the first XCDs.)
__device__ __forceinline__ void xcd_tile(int h, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
  const int T = tiles_m * tiles_n, q = T >> 3, rem = T & 7, x = h & 7;
  const int L = x * q + min(x, rem) + (h >> 3);
  const int span = group_m * tiles_n, g = L / span, first = g * group_m;
  const int gm = min(tiles_m - first, group_m), in = L - g * span;
  tm = first + in % gm;
  tn = in / gm;
}

}  // namespace qn
