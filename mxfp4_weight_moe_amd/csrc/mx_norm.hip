// The norms before and after a block, fused with the block's gate, residual scale and residual:
//   n  = rms_norm(b) * w_post      (or b)          rms_norm(v) = v / sqrt(mean v^2 + eps)
//   y  = bf16( x + scale * gate * n )              the residual stream after the block
//   xn = bf16( rms_norm(y) * w_pre )               the next block's input, from y as stored
// and its backward, with D = dy + J_pre^T dxn the whole gradient into y:
//   dx = D;  e = scale * D;  dgate = e * n;  e *= gate;  dw_post = sum_t e * b * q;
//   db = J_post^T (e * w_post)                     J^T t = q (t - v q^2 mean(t v)),  q = 1 / rms
//
// One pass: a workgroup holds a row of every input in registers (16-byte pieces, packed bf16),
// so each is read once and each output written once; sums are fp32, two block reductions a row
// at most.  The inverse rms values are computed again in the backward pass, from rows that it
// reads anyway, instead of being stored.  Parameter gradients add up in registers over a
// workgroup's rows and are summed over the workgroups in a fixed order by a second launch.
#include "mx_epilogue.hpp"
#include "mx_internal.hpp"

namespace mx {

struct NormArgs {
  const uint16_t* x;       // forward: x; backward: y
  const uint16_t* b;       // block output
  const uint16_t* w_post;
  const uint16_t* w_pre;
  const uint16_t* gate;
  const uint16_t* dy;
  const uint16_t* dxn;
  uint16_t* y;             // forward: y; backward: dx
  uint16_t* xn;            // forward: xn; backward: db
  void* dgate;             // token: fp32 [T]; full: bf16 [T, H]
  float* parts;            // [workgroups][arrays][H]
  int gate_mode;
  int T, H;
  int arrays;              // parameter gradients kept in parts
  float scale, eps;
};

__device__ __forceinline__ void unpack8(u32x4 q, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(q[i] << 16);
    v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// Sums of S values over the workgroup, in every thread; a fixed order.  `red` is used once per
// parity, so that one barrier is enough.
template <int NT, int S>
__device__ __forceinline__ void block_sum(float (&v)[S], float (*red)[S]) {
#pragma unroll
  for (int k = 0; k < S; ++k)
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v[k] += __shfl_xor(v[k], o, 64);
  if constexpr (NT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < S; ++k) red[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < S; ++k) {
      v[k] = red[0][k];
#pragma unroll
      for (int i = 1; i < NT / 64; ++i) v[k] += red[i][k];
    }
  }
}

constexpr u32x4 ZERO4 = {0u, 0u, 0u, 0u};

// BLK: there is a block output; POST: it is normalized; PRE: y is normalized.
template <int NT, int V, bool BLK, bool POST, bool PRE>
__global__ void __launch_bounds__(NT) norm_kernel(NormArgs a) {
  __shared__ float red[2][NT / 64][1];
  const int vecs = a.H / 8;
  u32x4 wpost[V], wpre[V], gch[V];
  int at[V];
  bool ok[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = i * NT + threadIdx.x;
    ok[i] = at[i] < vecs;
    wpost[i] = (POST && ok[i]) ? ld16(a.w_post + at[i] * 8) : ZERO4;
    wpre[i] = (PRE && ok[i]) ? ld16(a.w_pre + at[i] * 8) : ZERO4;
    gch[i] = (BLK && ok[i] && a.gate_mode == MX_GATE_CHANNEL) ? ld16(a.gate + at[i] * 8) : ZERO4;
  }
  const float inv_h = 1.f / (float)a.H;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = (size_t)t * a.H;
    u32x4 xv[V], bv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      xv[i] = ok[i] ? ld16(a.x + row + at[i] * 8) : ZERO4;
      if constexpr (BLK) {
        bv[i] = ok[i] ? ld16(a.b + row + at[i] * 8) : ZERO4;
        if (a.gate_mode == MX_GATE_FULL) gch[i] = ok[i] ? ld16(a.gate + row + at[i] * 8) : ZERO4;
      }
    }
    if constexpr (BLK) {
      float q = 1.f;
      if constexpr (POST) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v[8];
          unpack8(bv[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(v[j], v[j], ss[0]);
        }
        block_sum<NT, 1>(ss, red[0]);
        q = rsqrtf(ss[0] * inv_h + a.eps);
      }
      float tok = a.scale;
      if (a.gate_mode == MX_GATE_TOKEN) tok *= bf16_bits_to_f32(a.gate[t]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float xf[8], bf[8], w[8], g[8];
        unpack8(xv[i], xf);
        unpack8(bv[i], bf);
        unpack8(wpost[i], w);
        unpack8(gch[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float n = POST ? bf[j] * q * w[j] : bf[j];
          if (a.gate_mode >= MX_GATE_CHANNEL) n *= g[j];
          xf[j] = __builtin_fmaf(tok, n, xf[j]);
        }
        xv[i] = pack8(xf);
        if (ok[i]) *reinterpret_cast<u32x4*>(a.y + row + at[i] * 8) = xv[i];
      }
    }
    if constexpr (PRE) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8];
        unpack8(xv[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = __builtin_fmaf(v[j], v[j], ss[0]);
      }
      block_sum<NT, 1>(ss, red[1]);
      const float q = rsqrtf(ss[0] * inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8], w[8];
        unpack8(xv[i], v);
        unpack8(wpre[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * q * w[j];
        if (ok[i]) *reinterpret_cast<u32x4*>(a.xn + row + at[i] * 8) = pack8(v);
      }
    }
    if constexpr (NT > 64) __syncthreads();  // the sums are read before the next row's are written
  }
}

template <int NT, int V, bool BLK, bool POST, bool PRE>
__global__ void __launch_bounds__(NT) norm_backward_kernel(NormArgs a) {
  __shared__ float red1[NT / 64][3];
  __shared__ float red2[NT / 64][2];
  const int vecs = a.H / 8;
  int at[V];
  bool ok[V];
  float gpre[PRE ? V : 1][8] = {}, gpost[POST ? V : 1][8] = {}, ggate[BLK ? V : 1][8] = {};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = i * NT + threadIdx.x;
    ok[i] = at[i] < vecs;
  }
  const float inv_h = 1.f / (float)a.H;
  const bool channel = BLK && a.gate_mode == MX_GATE_CHANNEL;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = (size_t)t * a.H;
    u32x4 dv[V], yv[V], nv[V], bv[V], gv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const size_t p = row + at[i] * 8;
      dv[i] = (a.dy && ok[i]) ? ld16(a.dy + p) : ZERO4;
      if constexpr (PRE) {
        yv[i] = ok[i] ? ld16(a.x + p) : ZERO4;
        nv[i] = ok[i] ? ld16(a.dxn + p) : ZERO4;
      }
      if constexpr (BLK) {
        bv[i] = ok[i] ? ld16(a.b + p) : ZERO4;
        gv[i] = !ok[i] ? ZERO4
                : channel ? ld16(a.gate + at[i] * 8)
                : a.gate_mode == MX_GATE_FULL ? ld16(a.gate + p) : ZERO4;
      }
    }
    // reduction 1: sum y^2, sum dxn w_pre y, sum b^2
    float s1[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (PRE) {
        float y[8], d[8], w[8];
        unpack8(yv[i], y);
        unpack8(nv[i], d);
        unpack8(ok[i] ? ld16(a.w_pre + at[i] * 8) : ZERO4, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s1[0] = __builtin_fmaf(y[j], y[j], s1[0]);
          s1[1] = __builtin_fmaf(d[j] * w[j], y[j], s1[1]);
        }
      }
      if constexpr (POST) {
        float b[8];
        unpack8(bv[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[2] = __builtin_fmaf(b[j], b[j], s1[2]);
      }
    }
    float r = 0.f, rc = 0.f, q = 1.f;
    if constexpr (PRE || POST) {
      block_sum<NT, 3>(s1, red1);
      r = rsqrtf(s1[0] * inv_h + a.eps);
      rc = r * r * s1[1] * inv_h;
      q = rsqrtf(s1[2] * inv_h + a.eps);
    }
    float tok = a.scale;
    if (BLK && a.gate_mode == MX_GATE_TOKEN) tok *= bf16_bits_to_f32(a.gate[t]);
    float e[V][8];  // D, then scale * gate * D (times w_post)
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack8(dv[i], e[i]);
      if constexpr (PRE) {
        float y[8], d[8], w[8];
        unpack8(yv[i], y);
        unpack8(nv[i], d);
        unpack8(ok[i] ? ld16(a.w_pre + at[i] * 8) : ZERO4, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          gpre[i][j] = __builtin_fmaf(d[j], y[j] * r, gpre[i][j]);
          e[i][j] += r * (d[j] * w[j] - y[j] * rc);
        }
      }
      if (ok[i]) *reinterpret_cast<u32x4*>(a.y + row + at[i] * 8) = pack8(e[i]);
      if constexpr (BLK) {
        float b[8], g[8], w[8];
        unpack8(bv[i], b);
        unpack8(gv[i], g);
        if constexpr (POST) unpack8(ok[i] ? ld16(a.w_post + at[i] * 8) : ZERO4, w);
        float dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float unit = POST ? b[j] * q : b[j];
          const float n = POST ? unit * w[j] : unit;
          dg[j] = a.scale * e[i][j] * n;
          s2[1] += dg[j];
          if (channel) ggate[i][j] += dg[j];
          e[i][j] *= tok;
          if (a.gate_mode >= MX_GATE_CHANNEL) e[i][j] *= g[j];
          if constexpr (POST) {
            gpost[i][j] = __builtin_fmaf(e[i][j], unit, gpost[i][j]);
            e[i][j] *= w[j];
            s2[0] = __builtin_fmaf(e[i][j], b[j], s2[0]);
          }
        }
        if (a.gate_mode == MX_GATE_FULL && a.dgate && ok[i])
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dgate) + row + at[i] * 8) = pack8(dg);
      }
    }
    if constexpr (BLK) {
      if (POST || a.gate_mode == MX_GATE_TOKEN) block_sum<NT, 2>(s2, red2);
      if (a.gate_mode == MX_GATE_TOKEN && a.dgate && threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = s2[1];
      const float qc = q * q * s2[0] * inv_h;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (POST) {
          float b[8];
          unpack8(bv[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) e[i][j] = q * (e[i][j] - b[j] * qc);
        }
        if (a.xn && ok[i]) *reinterpret_cast<u32x4*>(a.xn + row + at[i] * 8) = pack8(e[i]);
      }
    }
    if constexpr (NT > 64) __syncthreads();
  }
  if (!a.parts) return;
  float* p = a.parts + (size_t)blockIdx.x * a.arrays * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!ok[i]) continue;
    float* c = p + at[i] * 8;
    if constexpr (PRE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = gpre[i][j];
      c += a.H;
    }
    if constexpr (POST) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = gpost[i][j];
      c += a.H;
    }
    if constexpr (BLK)
      if (channel)
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = ggate[i][j];
  }
}

// ------------------------------------------------------------------ launches

// Threads and 16-byte pieces per thread for a row of H values.
#define MX_NORM_SIZES(CALL)    \
  const int vecs = a.H / 8;    \
  if (vecs <= 64)              \
    CALL(64, 1);               \
  else if (vecs <= 256)        \
    CALL(256, 1);              \
  else if (vecs <= 512)        \
    CALL(256, 2);              \
  else if (vecs <= 1024)       \
    CALL(512, 2);              \
  else                         \
    CALL(1024, 2)

template <bool BLK, bool POST, bool PRE>
static void norm_forward(const NormArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)std::min(a.T, 8 * GPU_CUS));
#define MX_CALL(NT, V) hipLaunchKernelGGL((norm_kernel<NT, V, BLK, POST, PRE>), grid, dim3(NT), 0, stream, a)
  MX_NORM_SIZES(MX_CALL);
#undef MX_CALL
}

template <bool BLK, bool POST, bool PRE>
static void norm_backward(const NormArgs& a, int groups, hipStream_t stream) {
#define MX_CALL(NT, V) \
  hipLaunchKernelGGL((norm_backward_kernel<NT, V, BLK, POST, PRE>), dim3(groups), dim3(NT), 0, stream, a)
  MX_NORM_SIZES(MX_CALL);
#undef MX_CALL
}

int launch_norm_residual(const uint16_t* x, const uint16_t* b, const uint16_t* w_post, const uint16_t* gate,
                         int gate_mode, float scale, const uint16_t* w_pre, float eps, uint16_t* y, uint16_t* xn, int T,
                         int H, hipStream_t stream) {
  NormArgs a{};
  a.x = x, a.b = b, a.w_post = w_post, a.w_pre = w_pre, a.gate = gate;
  a.y = y, a.xn = xn, a.gate_mode = gate_mode, a.T = T, a.H = H, a.scale = scale, a.eps = eps;
  if (!b)
    norm_forward<false, false, true>(a, stream);
  else if (w_post)
    w_pre ? norm_forward<true, true, true>(a, stream) : norm_forward<true, true, false>(a, stream);
  else
    w_pre ? norm_forward<true, false, true>(a, stream) : norm_forward<true, false, false>(a, stream);
  return hip_status(hipGetLastError());
}

// Workgroups of the backward launch: two per CU, each with T / groups rows.
int norm_backward_groups(int64_t T) { return (int)std::min<int64_t>(T, 2 * GPU_CUS); }

int launch_norm_residual_backward(const uint16_t* dy, const uint16_t* dxn, const uint16_t* y, const uint16_t* b,
                                  const uint16_t* w_post, const uint16_t* gate, int gate_mode, float scale,
                                  const uint16_t* w_pre, float eps, uint16_t* dx, uint16_t* db, void* dgate,
                                  float* dw_post, float* dw_pre, int T, int H, float* parts, hipStream_t stream) {
  NormArgs a{};
  a.x = y, a.b = b, a.w_post = w_post, a.w_pre = w_pre, a.gate = gate, a.dy = dy, a.dxn = dxn;
  a.y = dx, a.xn = db, a.gate_mode = gate_mode, a.T = T, a.H = H, a.scale = scale, a.eps = eps;
  a.dgate = dgate;
  const bool channel = b && gate_mode == MX_GATE_CHANNEL;
  a.arrays = (w_pre ? 1 : 0) + (w_post ? 1 : 0) + (channel ? 1 : 0);
  float* out[3];
  int n = 0;
  if (w_pre) out[n++] = dw_pre;
  if (w_post) out[n++] = dw_post;
  if (channel) out[n++] = static_cast<float*>(dgate);
  bool any = false;
  for (int i = 0; i < n; ++i) any = any || out[i];
  a.parts = any ? parts : nullptr;
  const int groups = norm_backward_groups(T);
  if (!b)
    norm_backward<false, false, true>(a, groups, stream);
  else if (w_post)
    w_pre ? norm_backward<true, true, true>(a, groups, stream) : norm_backward<true, true, false>(a, groups, stream);
  else
    w_pre ? norm_backward<true, false, true>(a, groups, stream) : norm_backward<true, false, false>(a, groups, stream);
  int st = hip_status(hipGetLastError());
  if (st == MX_OK && any) st = launch_strip_sum(parts, groups, H, n, out, stream);
  return st;
}

}  // namespace mx
