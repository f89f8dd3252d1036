// Limits, strides and overlaps as the layer operators' entry points check them.
#pragma once

#include "host_checks.h"
#include "selective.h"

namespace ssd {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 31;  // tokens, sequences, batch rows, slots
constexpr int64_t kMaxChannels = int64_t(1) << 20;
// a token stride in elements: fewer than 2^24 bytes of either type (a factor of
// the kernels' 24-bit products for offsets inside a tile)
constexpr int64_t kMaxTokenStride = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxGridZ = 65535;

inline bool io_of(int32_t dtype, int* io) {
  if (dtype == SSD_DTYPE_F32) *io = kF32;
  else if (dtype == SSD_DTYPE_BF16) *io = kBF16;
  else return false;
  return true;
}
inline size_t bytes_of(int io) { return io == kBF16 ? 2 : 4; }

// Strides of [batch, rows, width]: dense where they are given as 0. False
// where rows overlap their neighbours, or the extent or the dense size (an
// output's) leaves the limits.
inline bool resolve(const ssd_stride_t& s, int64_t batch, int64_t rows, int64_t width, Stride* out, int64_t* extent) {
  if (rows > kMaxElems / width || batch > kMaxElems / (rows * width)) return false;
  Stride r{s.token, s.batch};
  if (r.token == 0) r.token = width;
  if (r.token < width || r.token > kMaxTokenStride) return false;
  if (r.batch == 0) r.batch = rows * r.token;  // below 2^53
  if (r.batch < width || r.batch > kMaxElems) return false;
  if (rows - 1 > kMaxElems / r.token || batch - 1 > kMaxElems / r.batch) return false;
  *extent = (batch - 1) * r.batch + (rows - 1) * r.token + width;
  if (*extent > kMaxElems) return false;
  *out = r;
  return true;
}

template <size_t N>
bool overlaps_any(const Range& r, const Range (&with)[N]) {
  for (const Range& w : with)
    if (overlap(r, w)) return true;
  return false;
}

}  // namespace ssd
