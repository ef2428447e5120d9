// Address of a lane's scale load in the MXFP4 forward tiles; plain C++, for the
// kernel and for a host check of its bounds.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define QN_HOST_DEVICE __host__ __device__
#else
#define QN_HOST_DEVICE
#endif

namespace qn {

// A lane loads the scale bytes of rows `row` (even) and row + 1 of a chunk, 16
// bytes at this offset from the chunk's first.  Rows past a matrix of `rows` rows
// give the last pair: the chunk is added outside the buffer's range check (a
// scalar offset), so the offset itself must stay inside.  With an odd row count
// the last pair of the last chunk ends 8 bytes past the scales; weights have even
// counts, and behind the scales of X^ lie its codes.
QN_HOST_DEVICE inline uint32_t mx_scale_pair(int64_t row, int64_t rows) {
  const int64_t last = (rows - 1) & ~(int64_t)1;
  return (uint32_t)((row < last ? row : last) * 8);
}

}  // namespace qn
