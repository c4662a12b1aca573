// Grids whose size grows with tokens times weight rows (plain C++, no device code).  A launch
// takes fewer than 2^32 threads along x and 65535 workgroups along y and z.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace mx {

constexpr int STREAM_MAX_T = 32;  // tokens of a workgroup of the weight-streaming kernel

// A workgroup to `cols` weight rows along x and STREAM_MAX_T tokens along y and z; the last z may
// reach past the tokens.
struct StreamGrid {
  uint32_t items, y, z;
};
inline StreamGrid stream_grid(int64_t T, int64_t rows, int64_t cols) {
  const int64_t groups = (T + STREAM_MAX_T - 1) / STREAM_MAX_T, y = std::min<int64_t>(groups, 1 << 15);
  return {(uint32_t)((rows + cols - 1) / cols), (uint32_t)y, (uint32_t)((groups + y - 1) / y)};
}

}  // namespace mx
