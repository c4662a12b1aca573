// Activations of the dense feed-forward operators, their derivatives, and the epilogues that
// turn fp32 products into outputs.  Everything here is fp32; a value is rounded to bf16 once,
// when it is stored.
#pragma once
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace mx {

// Error bounds below count u = 2^-24, half a step of fp32.  exp(a) is 2^(a log2 e) with the
// argument and the constant rounded, so it is off by 1.3 |a| u beside its own 2 u, and 0 below
// fp32's smallest normal value.
//
// p = 1 / (1 + e^-z), off by at most (1.3 |z| (1 - p) + 6) u relative to p; 0 below z = -87.3,
// where p is less than 2^-126.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// gelu_tanh(z) = z/2 (1 + tanh v) with v = sqrt(2/pi) (z + 0.044715 z^3); (1 + tanh v) / 2 is
// the logistic function of 2v.
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 1.5957691216057308f * __builtin_fmaf(0.044715f * z * z, z, z);
}

// The normal distribution function, Phi(z) = erfc(-z / sqrt 2) / 2.  With a = |z| / sqrt 2 and
// t = 1 / (1 + 0.4 a), erfc(a) e^(a^2) = t P(t); P is a degree-8 least-squares fit of ours with
// the weights moved until the relative error was level, 6e-8 on 0 <= a <= 9.6 (beyond, the
// exponential is 0).  In fp32 the exponential's argument sets the error: the tail is within
// (z^2 + 16) u of exact, relative (1e-6 at z = -1, 2e-6 at -4, 7e-6 at -10), what is stored in
// bf16 is rounded by 65536 u.  13 instructions; the library's erff with its two branches took
// 30 us of a 240 us product.
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.282842712f, __builtin_fabsf(z), 1.f));
  float p = 2.023664985e-02f;
  p = __builtin_fmaf(p, t, -6.824308055e-02f);
  p = __builtin_fmaf(p, t, 3.798630310e-02f);
  p = __builtin_fmaf(p, t, 4.862525028e-02f);
  p = __builtin_fmaf(p, t, 3.662653230e-02f);
  p = __builtin_fmaf(p, t, 9.810225960e-02f);
  p = __builtin_fmaf(p, t, 1.005784959e-01f);
  p = __builtin_fmaf(p, t, 1.132736117e-01f);
  p = __builtin_fmaf(p, t, 1.128140070e-01f);
  const float tail = p * t * __expf(-0.5f * z * z);
  return z > 0.f ? 1.f - tail : tail;
}

// V values at once: the choice stands outside, so that the values' chains overlap.
template <int V>
__device__ __forceinline__ void act_values(int act, float (&z)[V]) {
  switch (act) {
    case MX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = z[i] > 0.f ? z[i] : (z[i] != z[i] ? z[i] : 0.f);
      break;
    case MX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = z[i] * logistic(z[i]);
      break;
    case MX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = z[i] * normal_cdf(z[i]);
      break;
    case MX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = z[i] * logistic(gelu_tanh_arg(z[i]));
      break;
    case MX_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = logistic(z[i]);
      break;
    default: break;
  }
}

// act(z) and act'(z)
template <int V>
__device__ __forceinline__ void act_values_slopes(int act, const float (&z)[V], float (&a)[V], float (&d)[V]) {
  switch (act) {
    case MX_ACT_RELU:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = z[i] > 0.f ? z[i] : (z[i] != z[i] ? z[i] : 0.f);
        d[i] = z[i] > 0.f ? 1.f : 0.f;
      }
      break;
    case MX_ACT_SILU:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = logistic(z[i]);
        a[i] = z[i] * p;
        d[i] = __builtin_fmaf(a[i], 1.f - p, p);
      }
      break;
    case MX_ACT_GELU:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float c = normal_cdf(z[i]);
        a[i] = z[i] * c;
        d[i] = __builtin_fmaf(z[i], 0.39894228040143268f * __expf(-0.5f * z[i] * z[i]), c);
      }
      break;
    case MX_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = logistic(gelu_tanh_arg(z[i]));
        a[i] = z[i] * p;
        // z^2 held below overflow: the factor before it is 0 from |z| = 10 on
        const float z2 = fminf(z[i] * z[i], 1e30f);
        d[i] = __builtin_fmaf(a[i] * (1.f - p), 1.5957691216057308f * __builtin_fmaf(0.134145f, z2, 1.f), p);
      }
      break;
    case MX_ACT_SIGMOID:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // a (1 - a) from e = exp(-|z|) <= 1: of 1 - a as a difference no digit is left at z = 17
        const float e = __expf(-__builtin_fabsf(z[i])), r = __builtin_amdgcn_rcpf(1.f + e);
        a[i] = z[i] < 0.f ? e * r : r;
        d[i] = e * r * r;
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = z[i];
        d[i] = 1.f;
      }
      break;
  }
}

// Two bf16 values in one instruction (round to nearest even, as f32_to_bf16_rne).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2_t;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2));
}

// V consecutive bf16 values from p (V = 4 or 8), as one piece where all V exist (`wide`), else
// one by one up to `n` values (the rest read as 0).  A piece need not be aligned beyond its
// values: rows of an odd length stay whole accesses (global memory takes them at any address;
// value by value a gate_up of 3332 tokens with H = 2240, I = 1466 took 65 us instead of 62).
template <int V>
struct Piece {
  uint32_t q[V / 2];
};
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <int V>
__device__ __forceinline__ Piece<V> load_piece(const uint16_t* p, bool wide, int n) {
  Piece<V> r;
  if (wide) {
    if constexpr (V == 8) {
      const u32x4 t = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.q[i] = t[i];
    } else {
      const u32x2 t = *reinterpret_cast<const u32x2_any*>(p);
      r.q[0] = t[0], r.q[1] = t[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      r.q[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
  }
  return r;
}
template <int V>
__device__ __forceinline__ void unpack(const Piece<V>& r, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    v[2 * i] = __uint_as_float(r.q[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.q[i] & 0xFFFF0000u);
  }
}
template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&v)[V], bool wide, int n) {
  unpack(load_piece<V>(p, wide, n), v);
}

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[V], bool wide, int n) {
  if (wide) {
    if constexpr (V == 8)
      *reinterpret_cast<u32x4_any*>(p) =
          u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    else
      *reinterpret_cast<u32x2_any*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = f32_to_bf16_rne(v[i]);
  }
}

// An epilogue takes V consecutive columns of a row.  columns() gives what it needs of its
// columns (the bias), once for all rows of a lane; fetch() what it reads for one row, ahead of
// its use; store() computes and writes.

// y = residual + scale * act(z + bias); optionally the biased z itself.  y may be the
// residual: each element is read before it is written, by the same lane.
struct LinearEpilogue {
  static constexpr bool WHOLE_BLOCKS = false;
  const uint16_t* bias;      // [N] or null
  const uint16_t* residual;  // [T, N] or null
  uint16_t* y;               // [T, N]
  uint16_t* z;               // [T, N] or null
  int N;
  int act;
  float scale;

  template <int V>
  struct Columns {
    Piece<V> bias;
  };
  template <int V>
  __device__ __forceinline__ bool wide(int n) const {
    return n + V <= N;
  }
  template <int V>
  __device__ __forceinline__ Columns<V> columns(int n) const {
    Columns<V> c{};
    if (bias && n < N) c.bias = load_piece<V>(bias + n, wide<V>(n), N - n);
    return c;
  }
  template <int V>
  __device__ __forceinline__ Piece<V> fetch(int t, int n) const {
    Piece<V> r{};
    if (residual && n < N) r = load_piece<V>(residual + (size_t)t * N + n, wide<V>(n), N - n);
    return r;
  }
  template <int V>
  __device__ __forceinline__ void store(int t, int n, float (&v)[V], const Columns<V>& c, const Piece<V>& res) const {
    if (n >= N) return;
    const size_t at = (size_t)t * N + n;
    float b[V], r[V];
    unpack(c.bias, b);
    if (bias)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b[i];
    if (z) store_bf16<V>(z + at, v, wide<V>(n), N - n);
    act_values(act, v);
    unpack(res, r);
    if (residual)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(scale, v[i], r[i]);
    else
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= scale;
    store_bf16<V>(y + at, v, wide<V>(n), N - n);
  }
};

// h = act(g + bg) * (u + bu); optionally the biased g and u.
struct GatedEpilogue {
  static constexpr bool WHOLE_BLOCKS = false;  // takes any piece of a row, not blocks of 32 alone
  const uint16_t* bias;  // [2I] or null
  uint16_t* h;           // [T, I]
  uint16_t* z;           // [T, 2I] or null
  int I;
  int act;

  template <int V>
  struct Columns {
    Piece<V> gate, up;
  };
  template <int V>
  __device__ __forceinline__ bool wide(int n) const {
    return n + V <= I;
  }
  template <int V>
  __device__ __forceinline__ Columns<V> columns(int n) const {
    Columns<V> c{};
    if (bias && n < I) {
      c.gate = load_piece<V>(bias + n, wide<V>(n), I - n);
      c.up = load_piece<V>(bias + I + n, wide<V>(n), I - n);
    }
    return c;
  }
  // g becomes h; z is stored
  template <int V>
  __device__ __forceinline__ void product(int t, int n, float (&g)[V], float (&u)[V], const Columns<V>& c) const {
    const bool w = wide<V>(n);
    const int left = I - n;
    if (bias) {
      float b[V];
      unpack(c.gate, b);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] += b[i];
      unpack(c.up, b);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] += b[i];
    }
    if (z) {
      store_bf16<V>(z + (size_t)t * 2 * I + n, g, w, left);
      store_bf16<V>(z + (size_t)t * 2 * I + I + n, u, w, left);
    }
    act_values(act, g);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] *= u[i];
  }
  template <int V>
  __device__ __forceinline__ void store(int t, int n, float (&g)[V], float (&u)[V], const Columns<V>& c) const {
    if (n >= I) return;
    product<V>(t, n, g, u, c);
    store_bf16<V>(h + (size_t)t * I + n, g, wide<V>(n), I - n);
  }
};

}  // namespace mx
