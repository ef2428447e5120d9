// Counter-based dropout, device side (gfx950).
//
// Element i of a tensor (row-major) is field i % 8 of generator call i / 8:
// Philox4x32 with 7 rounds (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011: the smallest round count that
// passed all their tests; the usual 10 leave a margin that a dropout mask does
// not use), counter (call index, offset) and key (seed), gives four 32-bit
// words, read as eight 16-bit fields, low half first.  The element is kept
// when its field is at least thr = round(65536 p).  One call serves the eight
// elements of a 16-byte bf16 load, so the mask costs 14 32 x 32 -> 64 bit
// multiplies for eight elements and is never stored: the backward forms it
// again from the same (seed, offset).
#pragma once

#include "qn_device.h"
#include "qn_internal.h"

namespace qn {

struct DropKey {
  uint32_t k0, k1, o0, o1;
  uint32_t thr2;   // thr - 1 in both halves (thr >= 1)
};

// Wave-uniform; reads the caller's device-side offset, if any.
__device__ __forceinline__ DropKey drop_key(const DropArgs &d) {
  uint64_t off = d.offset;
  if (d.offset_dev) off += *d.offset_dev;
  DropKey k;
  k.k0 = (uint32_t)d.seed;
  k.k1 = (uint32_t)(d.seed >> 32);
  k.o0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)off);
  k.o1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(off >> 32));
  k.thr2 = (d.thr - 1u) * 0x10001u;
  return k;
}

// A generator call in parts: start, then the seven rounds in order.
struct Philox {
  uint32_t c[4];
  __device__ __forceinline__ void start(uint64_t g, const DropKey &k) {
    c[0] = (uint32_t)g; c[1] = (uint32_t)(g >> 32); c[2] = k.o0; c[3] = k.o1;
  }
  // Rounds `first` .. first + N - 1 of the seven.
  template <int N>
  __device__ __forceinline__ void rounds(const DropKey &k, int first) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (first + i >= 7) break;
      const uint32_t n = (uint32_t)(first + i);
      const uint64_t p0 = (uint64_t)0xD2511F53u * c[0], p1 = (uint64_t)0xCD9E8D57u * c[2];
      c[0] = (uint32_t)(p1 >> 32) ^ c[1] ^ (k.k0 + n * 0x9E3779B9u);
      c[1] = (uint32_t)p1;
      c[2] = (uint32_t)(p0 >> 32) ^ c[3] ^ (k.k1 + n * 0xBB67AE85u);
      c[3] = (uint32_t)p0;
    }
  }
};

// The four words of generator call g.
__device__ __forceinline__ void philox7(uint64_t g, const DropKey &k, uint32_t (&w)[4]) {
  Philox p;
  p.start(g, k);
  p.rounds<7>(k, 0);
  w[0] = p.c[0]; w[1] = p.c[1]; w[2] = p.c[2]; w[3] = p.c[3];
}

// Two fields -> 0xFFFF in the half of each kept element, 0 in the other's: field -
// (thr - 1) saturating at 0, at most 1, negated.  In asm because the compiler
// turns the same three packed operations into compares, selects and a permute
// per pair.
__device__ __forceinline__ uint32_t keep_mask2(uint32_t w, uint32_t thr2) {
  uint32_t d;
  asm("v_pk_sub_u16 %0, %1, %2 clamp" : "=v"(d) : "v"(w), "s"(thr2));
  asm("v_pk_min_u16 %0, %0, %1" : "+v"(d) : "s"(0x00010001u));
  asm("v_pk_sub_i16 %0, 0, %0" : "+v"(d));
  return d;
}

// Bit t set when element t of the call's eight is kept.
__device__ __forceinline__ uint32_t keep_bits8(const uint32_t (&w)[4], uint32_t thr2) {
  uint32_t b = 0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t m = keep_mask2(w[t], thr2);
    b |= (m & 1u) << (2 * t) | ((m >> 16) & 1u) << (2 * t + 1);
  }
  return b;
}

// acc += c keep * t for one 32 x 32 tile of dX's adapter term (a lane's element
// e is row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32), with row lr's 32
// mask bits in lanes lr and lr + 32: an element's lane mask is two rows' words,
// read out of their lanes into a scalar pair.  Elements that are not kept add
// nothing, whatever t holds.  The tiles are fenced from each other: run ahead, they
// would spill the accumulators.
__device__ __forceinline__ void add_kept(f32x16 &acc, const f32x16 &t, float c, uint32_t row) {
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int ra = 8 * (e >> 2) + (e & 3);
    const uint64_t mask = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)row, ra + 4) << 32 |
                          (uint32_t)__builtin_amdgcn_readlane((int)row, ra);
    const float v = __builtin_fmaf(c, t[e], acc[e]);
    acc[e] = __builtin_amdgcn_inverse_ballot_w64(mask) ? v : acc[e];
  }
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace qn
