// Checks of arguments that the entry points of the dense operators share (host code).
#pragma once
#include "mx_internal.hpp"

namespace mx {

constexpr int64_t MAX_T = (int64_t)1 << 24, MAX_K = (int64_t)1 << 20, MAX_N = (int64_t)1 << 22;
constexpr int64_t MAX_VALUES = (int64_t)1 << 38;  // values of one activation tensor

// Reduction length K (a multiple of 32), `rows` weight rows.
inline bool sizes_ok(int64_t T, int64_t K, int64_t rows) {
  return T >= 1 && T <= MAX_T && K >= 32 && K <= MAX_K && K % 32 == 0 && rows >= 1 && rows <= MAX_N &&
         T <= MAX_VALUES / K && T <= MAX_VALUES / rows;
}
inline bool gated_ok(int64_t T, int64_t H, int64_t I) { return I >= 1 && I <= MAX_N / 2 && sizes_ok(T, H, 2 * I); }
inline bool block_ok(int64_t T, int64_t H, int64_t I) { return gated_ok(T, H, I) && sizes_ok(T, I, H); }
inline bool act_ok(int act) { return act >= MX_ACT_NONE && act <= MX_ACT_SIGMOID; }
inline bool opt_aligned(const void* p, size_t a) { return !p || aligned(p, a); }
// 8-byte scale loads where a row's scales are a multiple of 8 bytes, 4-byte copies of 4
inline bool scales_aligned(const uint8_t* s, int64_t K) {
  return K % 256 == 0 ? aligned(s, 8) : K % 128 != 0 || aligned(s, 4);
}
inline int workspace_ok(const void* ws, size_t have, size_t need) {
  if (need == 0) return MX_OK;
  return (!ws || !aligned(ws, 256) || have < need) ? MX_ERR_WORKSPACE : MX_OK;
}
inline bool norm_sizes_ok(int64_t T, int64_t H) {
  return T >= 1 && T <= MAX_T && H >= 8 && H <= MX_NORM_MAX_H && H % 8 == 0;
}

}  // namespace mx
