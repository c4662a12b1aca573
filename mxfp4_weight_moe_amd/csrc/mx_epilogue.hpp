// Activations of the dense feed-forward operators, their derivatives, and the epilogues that
// turn fp32 products into outputs.  Everything here is fp32; a value is rounded to bf16 once,
// when it is stored.
#pragma once
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace mx {

// p = 1 / (1 + e^-z).  e^-z overflows to Inf below z = -88, where p = 0 is right to fp32's
// smallest normal value; 1 ulp reciprocal and exponential, so p is within 2e-7 of exact
// relative to p for |z| <= 16.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// gelu_tanh(z) = z/2 (1 + tanh v) with v = sqrt(2/pi) (z + 0.044715 z^3); (1 + tanh v) / 2 is
// the logistic function of 2v.
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 1.5957691216057308f * __builtin_fmaf(0.044715f * z * z, z, z);
}

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case MX_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case MX_ACT_SILU: return z * logistic(z);
    case MX_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case MX_ACT_GELU_TANH: return z * logistic(gelu_tanh_arg(z));
    case MX_ACT_SIGMOID: return logistic(z);
    default: return z;
  }
}

// act(z) and act'(z)
__device__ __forceinline__ void act_value_slope(int act, float z, float& a, float& d) {
  switch (act) {
    case MX_ACT_RELU:
      a = z > 0.f ? z : (z != z ? z : 0.f);
      d = z > 0.f ? 1.f : 0.f;
      break;
    case MX_ACT_SILU: {
      const float p = logistic(z);
      a = z * p;
      d = __builtin_fmaf(a, 1.f - p, p);
      break;
    }
    case MX_ACT_GELU: {
      const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
      a = z * c;
      d = __builtin_fmaf(z, 0.39894228040143268f * __expf(-0.5f * z * z), c);
      break;
    }
    case MX_ACT_GELU_TANH: {
      const float p = logistic(gelu_tanh_arg(z));
      a = z * p;
      d = __builtin_fmaf(a * (1.f - p), 1.5957691216057308f * __builtin_fmaf(0.134145f * z, z, 1.f), p);
      break;
    }
    case MX_ACT_SIGMOID:
      a = logistic(z);
      d = a * (1.f - a);
      break;
    default:
      a = z;
      d = 1.f;
      break;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_to_bf16_rne(lo) | ((uint32_t)f32_to_bf16_rne(hi) << 16);
}

// V consecutive bf16 values from p (V = 4, 8 or 16), as whole pieces where `wide` says that p
// is aligned for them and all V exist, else one by one up to `n` values (the rest read as 0).
template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&v)[V], bool wide, int n) {
  if (wide) {
    constexpr int P = V < 8 ? V : 8;
#pragma unroll
    for (int b = 0; b < V; b += P) {
      uint32_t q[P / 2];
      if constexpr (P == 8) {
        const u32x4 t = ld16(p + b);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = t[i];
      } else {
        const u32x2 t = ld8(p + b);
        q[0] = t[0], q[1] = t[1];
      }
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        v[b + 2 * i] = __uint_as_float(q[i] << 16);
        v[b + 2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? bf16_bits_to_f32(p[i]) : 0.f;
  }
}

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[V], bool wide, int n) {
  if (wide) {
    if constexpr (V >= 8) {
#pragma unroll
      for (int b = 0; b < V; b += 8)
        *reinterpret_cast<u32x4*>(p + b) = u32x4{pack_bf16(v[b], v[b + 1]), pack_bf16(v[b + 2], v[b + 3]),
                                                 pack_bf16(v[b + 4], v[b + 5]), pack_bf16(v[b + 6], v[b + 7])};
    } else {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = f32_to_bf16_rne(v[i]);
  }
}

// y = residual + scale * act(z + bias) of V consecutive columns of row t; optionally the
// biased z itself.  y may be the residual: each element is read before it is written, by the
// same lane.
struct LinearEpilogue {
  const uint16_t* bias;      // [N] or null
  const uint16_t* residual;  // [T, N] or null
  uint16_t* y;               // [T, N]
  uint16_t* z;               // [T, N] or null
  int N;
  int act;
  float scale;

  template <int V>
  __device__ __forceinline__ void store(int t, int n, float (&v)[V]) const {
    if (n >= N) return;
    const bool wide = n + V <= N && (N & 7) == 0;
    const int left = N - n;
    const size_t at = (size_t)t * N + n;
    if (bias) {
      float b[V];
      load_bf16<V>(bias + n, b, wide, left);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b[i];
    }
    if (z) store_bf16<V>(z + at, v, wide, left);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = scale * act_value(act, v[i]);
    if (residual) {
      float r[V];
      load_bf16<V>(residual + at, r, wide, left);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += r[i];
    }
    store_bf16<V>(y + at, v, wide, left);
  }
};

// h = act(g + bg) * (u + bu) of V consecutive columns; optionally the biased g and u.
struct GatedEpilogue {
  const uint16_t* bias;  // [2I] or null
  uint16_t* h;           // [T, I]
  uint16_t* z;           // [T, 2I] or null
  int I;
  int act;

  template <int V>
  __device__ __forceinline__ void store(int t, int n, float (&g)[V], float (&u)[V]) const {
    if (n >= I) return;
    const bool wide = n + V <= I && (I & 7) == 0;
    const int left = I - n;
    if (bias) {
      float b[V];
      load_bf16<V>(bias + n, b, wide, left);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] += b[i];
      load_bf16<V>(bias + I + n, b, wide, left);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] += b[i];
    }
    if (z) {
      store_bf16<V>(z + (size_t)t * 2 * I + n, g, wide, left);
      store_bf16<V>(z + (size_t)t * 2 * I + I + n, u, wide, left);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = act_value(act, g[i]) * u[i];
    store_bf16<V>(h + (size_t)t * I + n, g, wide, left);
  }
};

}  // namespace mx
