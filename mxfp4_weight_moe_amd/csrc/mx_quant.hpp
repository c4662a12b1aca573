// Rows of fp32 values to MXFP8 or MXFP4 (OCP MX: 32 consecutive values of a row share one E8M0
// scale), 8 values a lane, 4 lanes a block.
//
//   scale = 2^(floor(log2 amax) - EMAX), at least 2^-127;  EMAX = 8 for E4M3, 2 for E2M1: the block's
//   largest value lands in the last binade of its type.
//   element = value / scale to the nearest, halves to the even code, saturating at 448 or 6.
//   All zeros: scale byte 0.  An Inf or NaN: scale byte 0xFF (NaN), elements 0x7F (E4M3) or 0 (E2M1).
// floor(log2 amax) is fp32's exponent field, so the scale is integer work.  The conversion
// instructions divide by the power of two in an fp32's exponent field (0 stands for 2^-127) and
// round to nearest even; that to E2M1 saturates, that to E4M3 gives NaN from 464 on, hence the clamp.
#pragma once
#include "mx_act8.hpp"

namespace mx {

// FMT: bits of an element, 8 or 4 (0: none)
template <int FMT>
struct MxElement {
  static constexpr uint32_t EMAX = FMT == 8 ? 8 : 2;
  static constexpr uint32_t MAX_MANTISSA = 0x600000u;  // 448 = 1.75 * 2^8; 6 = 1.5 * 2^2 is not needed
};

// The largest |value| of a quad of lanes as bits (Inf and NaN sort above all else).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));  // quad_perm [2,3,0,1]
}

// Codes of a lane's 8 values (2 words of E4M3, 1 of E2M1) and its block's scale byte.  The 4 lanes of
// an aligned quad hold one block and are all active.
template <int FMT>
__device__ __forceinline__ void quantize8(const float (&v)[8], uint32_t (&codes)[FMT / 4], uint32_t& byte) {
  typedef MxElement<FMT> E;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = quad_max(m);
  const uint32_t e = m >> 23;
  const uint32_t b = e > E::EMAX ? e - E::EMAX : 0u;
  const float scale = e8m0_scale_operand(b);
  if constexpr (FMT == 8) {
    const float lim = __uint_as_float(((b + E::EMAX) << 23) | E::MAX_MANTISSA);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_fmed3f(v[4 * j + i], -lim, lim);
      s16x2 q = {0, 0};
      q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c[0], c[1], scale, false);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c[2], c[3], scale, true);
      codes[j] = __builtin_bit_cast(uint32_t, q);
    }
  } else {
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
    codes[0] = q;
  }
  byte = b;
  if (e == 0xFFu) {
    byte = 0xFFu;
#pragma unroll
    for (int j = 0; j < FMT / 4; ++j) codes[j] = FMT == 8 ? 0x7F7F7F7Fu : 0u;
  }
}

// Stores a lane's 8 codes (piece `p` of the tensor, 8 values each) and, once a block, the scale.
template <int FMT>
__device__ __forceinline__ void store_codes8(uint8_t* codes, uint8_t* scales, size_t p, const uint32_t (&c)[FMT / 4],
                                             uint32_t byte) {
  if constexpr (FMT == 8)
    *reinterpret_cast<u32x2*>(codes + p * 8) = u32x2{c[0], c[1]};
  else
    *reinterpret_cast<uint32_t*>(codes + p * 4) = c[0];
  if ((p & 3) == 0) scales[p >> 2] = (uint8_t)byte;
}

// The bf16 values that 8 codes stand for: every element times a power of two, exact down to bf16's last
// step of 2^-133 (an E4M3 element times the smallest scale may need 2^-136 and is rounded).
template <int FMT>
__device__ __forceinline__ u32x4 code_values8(const uint32_t (&c)[FMT / 4], uint32_t byte) {
  const float scale = e8m0_scale_operand(byte);
  if constexpr (FMT == 4) {
    return __builtin_bit_cast(u32x4, decode8(c[0], scale));
  } else {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[j], scale, false));
      r[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[j], scale, true));
    }
    return r;
  }
}

}  // namespace mx
