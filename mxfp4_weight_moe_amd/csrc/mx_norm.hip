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
#include "mx_quant.hpp"

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
  uint8_t* codes;          // xn in MXFP8 or MXFP4 (then xn itself is optional)
  uint8_t* scales;
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

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum over groups of N consecutive lanes (N = 2, 4, 8 or 16), in every lane, in a fixed order: the
// lanes exchange in the vector unit (a shuffle through the LDS takes some 60 cycles).
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<0xB1>(v);                          // lane ^ 1
  if constexpr (N >= 4) v += dpp<0x4E>(v);    // lane ^ 2
  if constexpr (N >= 8) v += dpp<0x141>(v);   // mirrored within 8: the other 4
  if constexpr (N >= 16) v += dpp<0x140>(v);  // mirrored within 16: the other 8
  return v;
}
// Sum over the L lanes of a row (16, 32 or the wave), in every lane; the wave's rows of 16 lanes
// are read as scalars.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  v = lanes_sum<16>(v);
  if constexpr (L == 32) v += __shfl_xor(v, 16, 64);
  if constexpr (L == 64) v = (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
  return v;
}

// Sums of S values over the threads of a row, in each of them; a fixed order.  The caller leaves
// a barrier between two uses of the same `red`.
template <int NT, int L, int S>
__device__ __forceinline__ void block_sum(float (&v)[S], float (*red)[NT / 64]) {
#pragma unroll
  for (int k = 0; k < S; ++k) v[k] = row_sum<L>(v[k]);
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < S; ++k) red[k][wave] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = lanes_sum<W>(red[k][threadIdx.x & (W - 1)]);
  }
}

constexpr u32x4 ZERO4 = {0u, 0u, 0u, 0u};

// BLK: there is a block output; POST: it is normalized; PRE: y is normalized.
// Bound by memory: 8192 x 7168 with both norms and a gate per channel, 470 MB, in 80 to 89 us,
// 5.3 TB/s or more; 32 rows take 4 us, launch and latency.
// L: lanes of a row.  Less than a wave, for short rows, and a wave has 64 / L rows at a time.
// FMT: xn leaves as MXFP8 (8) or MXFP4 (4) codes and scales, quantized from its fp32 value; H % 32 == 0
// then, so that a block is a quad of lanes of one row.
// The same bound: 8192 x 7168 with both norms, a gate per channel, MXFP8 and xn in bf16, 532 MB, in
// 103 us, 5.2 TB/s; 16 rows take 4.2.
template <int NT, int V, int L, bool BLK, bool POST, bool PRE, int FMT = 0>
__global__ void __launch_bounds__(NT) norm_kernel(NormArgs a) {
  static_assert(L == 64 || NT == 64, "short rows have no barriers");
  static_assert(FMT == 0 || PRE, "what is quantized is xn");
  __shared__ float red[2][NT / 64];
  const int vecs = a.H / 8;
  u32x4 wpost[V], wpre[V], gch[V];
  int at[V];
  bool ok[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = i * NT + (L < 64 ? threadIdx.x % L : threadIdx.x);
    ok[i] = at[i] < vecs;
    wpost[i] = (POST && ok[i]) ? ld16(a.w_post + at[i] * 8) : ZERO4;
    wpre[i] = (PRE && ok[i]) ? ld16(a.w_pre + at[i] * 8) : ZERO4;
    gch[i] = (BLK && ok[i] && a.gate_mode == MX_GATE_CHANNEL) ? ld16(a.gate + at[i] * 8) : ZERO4;
  }
  const float inv_h = 1.f / (float)a.H;
  constexpr int R = 64 / L;
  for (int t = blockIdx.x * R + (L < 64 ? threadIdx.x / L : 0); t < a.T; t += gridDim.x * R) {
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
        block_sum<NT, L, 1>(ss, &red[0]);
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
      block_sum<NT, L, 1>(ss, &red[1]);
      const float q = rsqrtf(ss[0] * inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8], w[8];
        unpack8(xv[i], v);
        unpack8(wpre[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * q * w[j];
        if constexpr (FMT == 0) {
          if (ok[i]) *reinterpret_cast<u32x4*>(a.xn + row + at[i] * 8) = pack8(v);
        } else if (ok[i]) {
          uint32_t c[FMT / 4], byte;
          quantize8<FMT>(v, c, byte);
          store_codes8<FMT>(a.codes, a.scales, row / 8 + at[i], c, byte);
          if (a.xn) *reinterpret_cast<u32x4*>(a.xn + row + at[i] * 8) = pack8(v);
        }
      }
    }
    if constexpr (NT > 64) __syncthreads();  // the sums are read before the next row's are written
  }
}

// The rows of the backward pass's inputs that one thread holds.
template <int V>
struct NormRow {
  u32x4 d[V], y[V], n[V], b[V];  // dy, y, dxn, b
};

// What was unpacked from p before is unpacked again: 4 packed registers live on, not 8 floats.
__device__ __forceinline__ void repack(u32x4& p) { asm volatile("" : "+v"(p)); }

// 8 sums, held as two vectors.
__device__ __forceinline__ void add_to(f32x4* s, const float (&v)[8]) {
  s[0] += f32x4{v[0], v[1], v[2], v[3]};
  s[1] += f32x4{v[4], v[5], v[6], v[7]};
}

// AHEAD: the next row is loaded while this one is worked on (a workgroup of 16 waves is alone on
// its CU with the registers this takes, and waited for memory at each row without it).
// Bound by memory: at T = 4096, H = 7168 with both norms and a gate per channel 352 MB move in
// 79 us, 4.5 TB/s, as fast as a plain copy; with two pieces a thread, lane sums through the LDS
// and no row ahead it was 119.
// With both norms and 16 waves the compiler spills 8 of 128 registers (36 bytes of scratch a thread).
// Beyond H = 8192 (V = 4, 8 waves) there are no registers for that, nor for all sums of parameter
// gradients: those of w_post and the gate then stay in the LDS, each thread's in places of its
// own, and the weights are loaded for each row.  Both norms' instance still spills 41 of 256
// registers (168 bytes of scratch a thread, 25 stores and 44 loads of it in the code), the others
// none.  8704 x 4096 with both norms and a gate per channel 206 us, 2.1 TB/s; how much of that is
// the spills and how much the wait at each row has not been told apart (16 waves of two pieces: 315,
// and 562 with all sums in registers, which spill more; the next row's lines brought to the L2
// ahead: 263).
template <int NT, int V, int L, bool BLK, bool POST, bool PRE>
__global__ void __launch_bounds__(NT) norm_backward_kernel(NormArgs a) {
  static_assert(L == 64 || NT == 64, "short rows have no barriers");
  constexpr bool AHEAD = V == 1, IN_LDS = V > 1 && BLK;
  constexpr int R = 64 / L;
  extern __shared__ float sums[];  // [2][H]: w_post's, the gate's
  __shared__ float red1[3][NT / 64];
  __shared__ float red2[2][NT / 64];
  const int vecs = a.H / 8;
  int at[V];
  bool ok[V];
  float gpre[PRE ? V : 1][8] = {}, gpost[POST && !IN_LDS ? V : 1][8] = {}, ggate[BLK && !IN_LDS ? V : 1][8] = {};
  u32x4 wpre[V], wpost[V], gch[V];
  const bool channel = BLK && a.gate_mode == MX_GATE_CHANNEL, full = BLK && a.gate_mode == MX_GATE_FULL;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = i * NT + (L < 64 ? threadIdx.x % L : threadIdx.x);
    ok[i] = at[i] < vecs;
  }
  auto load_pre = [&](int i) { wpre[i] = (PRE && ok[i]) ? ld16(a.w_pre + at[i] * 8) : ZERO4; };
  auto load_post = [&](int i) {
    wpost[i] = (POST && ok[i]) ? ld16(a.w_post + at[i] * 8) : ZERO4;
    if (!full) gch[i] = (channel && ok[i]) ? ld16(a.gate + at[i] * 8) : ZERO4;
  };
  if constexpr (V == 1) load_pre(0), load_post(0);
  // this thread's 8 sums of piece i
  auto sums_of = [&](int k, int i) { return reinterpret_cast<f32x4*>(sums + k * a.H + at[i] * 8); };
  if constexpr (IN_LDS) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i])
#pragma unroll
        for (int k = 0; k < 2; ++k) sums_of(k, i)[0] = sums_of(k, i)[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto load_row = [&](int t) {
    NormRow<V> r;
    const size_t row = (size_t)t * a.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const size_t p = row + at[i] * 8;
      r.d[i] = (a.dy && ok[i]) ? ld16(a.dy + p) : ZERO4;
      if constexpr (PRE) {
        r.y[i] = ok[i] ? ld16(a.x + p) : ZERO4;
        r.n[i] = ok[i] ? ld16(a.dxn + p) : ZERO4;
      }
      if constexpr (BLK) r.b[i] = ok[i] ? ld16(a.b + p) : ZERO4;
    }
    return r;
  };
  const float inv_h = 1.f / (float)a.H;
  NormRow<V> cur;
  const int t0 = blockIdx.x * R + (L < 64 ? threadIdx.x / L : 0);
  if (AHEAD) cur = load_row(min(t0, a.T - 1));
  for (int t = t0; t < a.T; t += gridDim.x * R) {
    const size_t row = (size_t)t * a.H;
    NormRow<V> next;
    if (full) {
#pragma unroll
      for (int i = 0; i < V; ++i) gch[i] = ok[i] ? ld16(a.gate + row + at[i] * 8) : ZERO4;
    }
    if constexpr (AHEAD)
      next = load_row(min(t + (int)gridDim.x * R, a.T - 1));
    else
      cur = load_row(t);
    // reduction 1: sum y^2, sum dxn w_pre y, sum b^2
    float s1[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (PRE) {
        if constexpr (V > 1) {
          __builtin_amdgcn_sched_barrier(0);
          load_pre(i);
        }
        float y[8], d[8], w[8];
        unpack8(cur.y[i], y);
        unpack8(cur.n[i], d);
        unpack8(wpre[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s1[0] = __builtin_fmaf(y[j], y[j], s1[0]);
          s1[1] = __builtin_fmaf(d[j] * w[j], y[j], s1[1]);
        }
      }
      if constexpr (POST) {
        float b[8];
        unpack8(cur.b[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[2] = __builtin_fmaf(b[j], b[j], s1[2]);
      }
    }
    float r = 0.f, rc = 0.f, q = 1.f;
    if constexpr (PRE || POST) {
      block_sum<NT, L, 3>(s1, red1);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (PRE) repack(cur.y[i]), repack(cur.n[i]), repack(wpre[i]);
        if constexpr (POST) repack(cur.b[i]);
      }
      r = rsqrtf(s1[0] * inv_h + a.eps);
      rc = r * (r * s1[1] * inv_h);  // r * r leaves fp32 for the smallest eps
      q = rsqrtf(s1[2] * inv_h + a.eps);
    }
    float tok = a.scale;
    if (BLK && a.gate_mode == MX_GATE_TOKEN) tok *= bf16_bits_to_f32(a.gate[t]);
    float e[V][8];  // D, then scale * gate * D (times w_post)
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (V > 1) {
        __builtin_amdgcn_sched_barrier(0);  // one piece after the other: the registers of one
        load_pre(i), load_post(i);
      }
      unpack8(cur.d[i], e[i]);
      if constexpr (PRE) {
        float y[8], d[8], w[8];
        unpack8(cur.y[i], y);
        unpack8(cur.n[i], d);
        unpack8(wpre[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          gpre[i][j] = __builtin_fmaf(d[j], y[j] * r, gpre[i][j]);
          e[i][j] += r * (d[j] * w[j] - y[j] * rc);
        }
      }
      if (ok[i]) *reinterpret_cast<u32x4*>(a.y + row + at[i] * 8) = pack8(e[i]);
      if constexpr (BLK) {
        float b[8], g[8], w[8];
        unpack8(cur.b[i], b);
        unpack8(gch[i], g);
        if constexpr (POST) unpack8(wpost[i], w);
        float dg[8], dp[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float unit = POST ? b[j] * q : b[j];
          const float n = POST ? unit * w[j] : unit;
          dg[j] = a.scale * e[i][j] * n;
          s2[1] += dg[j];
          if constexpr (!IN_LDS)
            if (channel) ggate[i][j] += dg[j];
          e[i][j] *= tok;
          if (a.gate_mode >= MX_GATE_CHANNEL) e[i][j] *= g[j];
          if constexpr (POST) {
            if constexpr (IN_LDS)
              dp[j] = e[i][j] * unit;
            else
              gpost[i][j] = __builtin_fmaf(e[i][j], unit, gpost[i][j]);
            e[i][j] *= w[j];
            s2[0] = __builtin_fmaf(e[i][j], b[j], s2[0]);
          }
        }
        if constexpr (IN_LDS) {
          if (ok[i]) {
            if (channel) add_to(sums_of(1, i), dg);
            if constexpr (POST) add_to(sums_of(0, i), dp);
          }
        }
        if (full && a.dgate && ok[i])
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dgate) + row + at[i] * 8) = pack8(dg);
      }
    }
    if constexpr (BLK) {
      if (POST || a.gate_mode == MX_GATE_TOKEN) block_sum<NT, L, 2>(s2, red2);
      if constexpr (POST) {
#pragma unroll
        for (int i = 0; i < V; ++i) repack(cur.b[i]);
      }
      if (a.gate_mode == MX_GATE_TOKEN && a.dgate && threadIdx.x % L == 0 && threadIdx.x < 64)
        static_cast<float*>(a.dgate)[t] = s2[1];
      const float qc = q * (q * s2[0] * inv_h);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (POST) {
          float b[8];
          unpack8(cur.b[i], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) e[i][j] = q * (e[i][j] - b[j] * qc);
        }
        if (a.xn && ok[i]) *reinterpret_cast<u32x4*>(a.xn + row + at[i] * 8) = pack8(e[i]);
      }
    }
    if constexpr (NT > 64) __syncthreads();
    if constexpr (AHEAD) cur = next;
  }
  if (!a.parts) return;
  if constexpr (R > 1) {  // the rows of this wave, in a fixed order
    auto over_rows = [&](float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (L == 16) v[j] += __shfl_xor(v[j], 16, 64);
        v[j] += __shfl_xor(v[j], 32, 64);
      }
    };
    if constexpr (PRE) over_rows(gpre[0]);
    if constexpr (POST) over_rows(gpost[0]);
    if constexpr (BLK) over_rows(ggate[0]);
    if (threadIdx.x >= L) return;
  }
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
      for (int j = 0; j < 8; ++j) c[j] = IN_LDS ? sums_of(0, i)[j >> 2][j & 3] : gpost[IN_LDS ? 0 : i][j];
      c += a.H;
    }
    if constexpr (BLK)
      if (channel)
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = IN_LDS ? sums_of(1, i)[j >> 2][j & 3] : ggate[IN_LDS ? 0 : i][j];
  }
}

// ------------------------------------------------------------------ launches

// Threads, 16-byte pieces per thread and lanes for a row of H values: a piece a thread where that
// leaves no more than half of them idle.  Backward of 262144 x 128: 94 us with four rows a wave,
// 301 with one; 65536 x 520: 116 with 128 threads, 212 with 256.
#define MX_NORM_SIZES(CALL) \
  if (a.H <= 128)           \
    CALL(64, 1, 16);        \
  else if (a.H <= 256)      \
    CALL(64, 1, 32);        \
  else if (a.H <= 512)      \
    CALL(64, 1, 64);        \
  else if (a.H <= 1024)     \
    CALL(128, 1, 64);       \
  else if (a.H <= 2048)     \
    CALL(256, 1, 64);       \
  else if (a.H <= 4096)     \
    CALL(512, 1, 64);       \
  else if (a.H <= 8192)     \
    CALL(1024, 1, 64);      \
  else                      \
    CALL(512, 4, 64)
// Rows of a workgroup at a time.
static int norm_rows(int64_t H) { return H <= 128 ? 4 : H <= 256 ? 2 : 1; }

template <bool BLK, bool POST, bool PRE, int FMT = 0>
static void norm_forward(const NormArgs& a, hipStream_t stream) {
  const int rows = norm_rows(a.H);
  const dim3 grid((unsigned)std::min((a.T + rows - 1) / rows, 8 * GPU_CUS));
#define MX_CALL(NT, V, L) hipLaunchKernelGGL((norm_kernel<NT, V, L, BLK, POST, PRE, FMT>), grid, dim3(NT), 0, stream, a)
  MX_NORM_SIZES(MX_CALL);
#undef MX_CALL
}

template <bool BLK, bool POST, bool PRE>
static void norm_backward(const NormArgs& a, int groups, hipStream_t stream) {
  const unsigned lds = BLK && a.H > 8192 ? 2u * (unsigned)a.H * 4u : 0u;
#define MX_CALL(NT, V, L) \
  hipLaunchKernelGGL((norm_backward_kernel<NT, V, L, BLK, POST, PRE>), dim3(groups), dim3(NT), lds, stream, a)
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

template <int FMT>
static void norm_forward_quantized(const NormArgs& a, hipStream_t stream) {
  if (!a.b)
    norm_forward<false, false, true, FMT>(a, stream);
  else if (a.w_post)
    norm_forward<true, true, true, FMT>(a, stream);
  else
    norm_forward<true, false, true, FMT>(a, stream);
}

int launch_norm_residual_quantize(const uint16_t* x, const uint16_t* b, const uint16_t* w_post, const uint16_t* gate,
                                  int gate_mode, float scale, const uint16_t* w_pre, float eps, uint16_t* y,
                                  uint16_t* xn, int format, uint8_t* codes, uint8_t* scales, int T, int H,
                                  hipStream_t stream) {
  NormArgs a{};
  a.x = x, a.b = b, a.w_post = w_post, a.w_pre = w_pre, a.gate = gate;
  a.y = y, a.xn = xn, a.gate_mode = gate_mode, a.T = T, a.H = H, a.scale = scale, a.eps = eps;
  a.codes = codes, a.scales = scales;
  format == MX_FORMAT_MXFP8 ? norm_forward_quantized<8>(a, stream) : norm_forward_quantized<4>(a, stream);
  return hip_status(hipGetLastError());
}

// Workgroups of the backward launch, each with T / groups rows: what the CUs hold at once.
int norm_backward_groups(int64_t T, int64_t H) {
  const int rows = norm_rows(H);
  return (int)std::min<int64_t>((T + rows - 1) / rows, (H <= 256 ? 8 : H <= 1024 ? 4 : H <= 4096 ? 2 : 1) * GPU_CUS);
}

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
  const int groups = norm_backward_groups(T, H);
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
