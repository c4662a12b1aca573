// Backward of the dense feed-forward operators (frozen MXFP4 weights):
//   linear   dz = scale * dy * act'(z);  dx = dz W;  dbias = sum over tokens of dz
//   gate_up  dz = [dh * u * act'(g) | dh * act(g)] with z = [g | u]; dx and dbias the same way
// First launch: dz in bf16 and per-strip column sums, which use the unrounded fp32 values.  Where
// there is an activation dz is rounded here, once, as the matrix instructions take bf16: dx is then
// 0.0024 from exact instead of 0.0017 (root mean square), and dz in two bf16 parts would double the
// product.  Without one it is dy itself, and the scale follows the product.  Then the product dz W
// in tiles (mx_tile.hpp), with the strips' sums beside it.
#include "mx_epilogue.hpp"
#include "mx_tile.hpp"

namespace mx {

// ------------------------------------------------------------------ dz and the bias gradient

// A workgroup takes 256 columns (32 threads of 8) and a strip of rows, 8 at a time.  Bound by
// memory: 2048 x 4096 with z 50 MB in 12 us, 4.1 TB/s; gated, 4096 x 2048, 84 MB in 14 us (inputs
// partly from the last-level cache).
constexpr int DZ_COLS = 256;

struct LinearSlope {
  const uint16_t* dy;  // [T, N]
  const uint16_t* z;   // [T, N] or null (act none)
  int N, act;
  float scale;
  __device__ __forceinline__ int cols() const { return N; }
  // dy * act'(z), before the scale
  __device__ __forceinline__ void unscaled(int64_t t, int n, float (&v)[8], bool wide, int left) const {
    load_bf16<8>(dy + (size_t)t * N + n, v, wide, left);
    if (z) {
      float zv[8], a[8], d[8];
      load_bf16<8>(z + (size_t)t * N + n, zv, wide, left);
      act_values_slopes(act, zv, a, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= d[i];
    }
  }
  // What the product multiplies its sums with.  Without an activation it reads dy, exact in bf16,
  // and the scale comes after it; scale * dy would be rounded once more.
  __device__ __host__ __forceinline__ float alpha() const { return z ? 1.f : scale; }
};

// dz / alpha (bf16 [T][ldz], zeros in columns N .. ldz) and, if parts is set, the fp32 column sums
// of dz in this strip in parts[strip][cols].
template <class Slope>
__global__ void __launch_bounds__(256) dz_kernel(Slope f, uint16_t* __restrict__ dz, int ldz, float* __restrict__ parts,
                                                 int64_t T, int strip_rows) {
  __shared__ float red[8][DZ_COLS];
  const int N = f.cols();
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = blockIdx.x * DZ_COLS + cx * 8;
  const int64_t t0 = (int64_t)blockIdx.y * strip_rows, t1 = min(t0 + strip_rows, T);
  const bool wide = n + 8 <= N;
  const int left = N - n;
  float sum[8] = {};
  if (n < (dz ? ldz : N)) {  // columns N .. ldz read as 0
    for (int64_t t = t0 + ry; t < t1; t += 8) {
      float v[8];
      f.unscaled(t, n, v, wide, left);
      if (dz && !f.z) store_bf16<8>(dz + (size_t)t * ldz + n, v, true, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f.scale;
      if (dz && f.z) store_bf16<8>(dz + (size_t)t * ldz + n, v, true, 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[i];
    }
  }
  if (!parts) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ry][cx * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * DZ_COLS + threadIdx.x;
  if (c < N) {
    float a = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) a += red[r][threadIdx.x];
    parts[(size_t)blockIdx.y * N + c] = a;
  }
}

// gate_up: 8 columns of both halves a thread, see above.
__global__ void __launch_bounds__(256) dz_gated_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ z,
                                                       int I, int act, uint16_t* __restrict__ dz, int ldz,
                                                       float* __restrict__ parts, int64_t T, int strip_rows) {
  __shared__ float red[2][8][DZ_COLS];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = blockIdx.x * DZ_COLS + cx * 8;
  const int64_t t0 = (int64_t)blockIdx.y * strip_rows, t1 = min(t0 + strip_rows, T);
  const bool wide = n + 8 <= I;
  const int left = I - n;
  float sg[8] = {}, su[8] = {};
  if (n < I) {
    for (int64_t t = t0 + ry; t < t1; t += 8) {
      float d[8], g[8], u[8];
      load_bf16<8>(dh + (size_t)t * I + n, d, wide, left);
      load_bf16<8>(z + (size_t)t * 2 * I + n, g, wide, left);
      load_bf16<8>(z + (size_t)t * 2 * I + I + n, u, wide, left);
      float a[8], slope[8];
      act_values_slopes(act, g, a, slope);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = d[i] * u[i] * slope[i];
        u[i] = d[i] * a[i];
        sg[i] += g[i];
        su[i] += u[i];
      }
      if (dz) {
        store_bf16<8>(dz + (size_t)t * ldz + n, g, wide, left);
        store_bf16<8>(dz + (size_t)t * ldz + I + n, u, wide, left);
        if (n + 8 >= I)  // the padding columns of this row
          for (int c = 2 * I; c < ldz; ++c) dz[(size_t)t * ldz + c] = 0;
      }
    }
  }
  if (!parts) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[0][ry][cx * 8 + i] = sg[i];
    red[1][ry][cx * 8 + i] = su[i];
  }
  __syncthreads();
  const int c = blockIdx.x * DZ_COLS + threadIdx.x;
  if (c < I) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      a += red[0][r][threadIdx.x];
      b += red[1][r][threadIdx.x];
    }
    parts[(size_t)blockIdx.y * 2 * I + c] = a;
    parts[(size_t)blockIdx.y * 2 * I + I + c] = b;
  }
}

// out[k][c] = sum over strips, in a fixed order, of parts[strip][k][c] for the k whose out is
// set: a workgroup takes 64 columns of one k.  The strips are summed in 16 parts, a part a wave
// or four, and then the parts, in the same order whatever the number of waves W; a wave has 8
// or 16 loads in flight (with 4 parts and one load at a time 512 strips of 3 x 7168 took 35 us,
// 16 waves with 8 take 5).
constexpr int STRIP_PARTS = 16;
struct StripOut {
  float* p[3];
};

template <int W>
__device__ __forceinline__ void strip_sum(float (&red)[STRIP_PARTS][64], const float* __restrict__ parts,
                                          const StripOut& out, int strips, int cols, int arrays, int c0, int k) {
  if (!out.p[k]) return;
  constexpr int PW = STRIP_PARTS / W, U = W == STRIP_PARTS ? 8 : 4;  // parts of a wave, loads of each
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, c = c0 + lane;
  const float* p = parts + (size_t)k * cols + min(c, cols - 1);
  const size_t step = (size_t)arrays * cols;
  float a[PW] = {};
  int i0[PW], i1[PW];
#pragma unroll
  for (int j = 0; j < PW; ++j) {
    i0[j] = strips * (q * PW + j) / STRIP_PARTS;
    i1[j] = strips * (q * PW + j + 1) / STRIP_PARTS;
  }
  for (int i = 0; i < (strips + STRIP_PARTS - 1) / STRIP_PARTS; i += U) {
    float v[PW][U];
#pragma unroll
    for (int j = 0; j < PW; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) v[j][u] = p[min(i0[j] + i + u, strips - 1) * step];
#pragma unroll
    for (int j = 0; j < PW; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) a[j] += i0[j] + i + u < i1[j] ? v[j][u] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < PW; ++j) red[q * PW + j][lane] = a[j];
  __syncthreads();
  if (q == 0 && c < cols) {
    float s = red[0][lane];
#pragma unroll
    for (int w = 1; w < STRIP_PARTS; ++w) s += red[w][lane];
    out.p[k][c] = s;
  }
}

__global__ void __launch_bounds__(STRIP_PARTS * 64) strip_sum_kernel(const float* __restrict__ parts, StripOut out,
                                                                     int strips, int cols, int arrays) {
  __shared__ float red[STRIP_PARTS][64];
  strip_sum<STRIP_PARTS>(red, parts, out, strips, cols, arrays, blockIdx.x * 64, blockIdx.y);
}

int launch_strip_sum(const float* parts, int strips, int cols, int arrays, float* const* out, hipStream_t stream) {
  StripOut o{};
  for (int k = 0; k < arrays; ++k) o.p[k] = out[k];
  hipLaunchKernelGGL(strip_sum_kernel, dim3((cols + 63) / 64, arrays), dim3(STRIP_PARTS * 64), 0, stream, parts, o,
                     strips, cols, arrays);
  return hip_status(hipGetLastError());
}

// ------------------------------------------------------------------ dx = alpha * dz W

// The bias gradient's strips that the same launch sums.
struct BiasStrips {
  const float* parts;
  float* dbias;
  int strips, cols;
};

// Workgroups past the tiles sum the bias gradient's strips, 64 columns each, on CUs that the
// last round of tiles leaves idle (a launch of its own took 5 us).
template <int MT, int NT>
__global__ void __launch_bounds__(256, MT == 4 ? 1 : 2)
    backward_kernel(const uint16_t* __restrict__ dz, const uint8_t* __restrict__ w, const uint8_t* __restrict__ s,
                    uint16_t* __restrict__ dx, float* __restrict__ parts, float alpha, int T, int K, int N, int ldz,
                    int mtiles, int ntiles, int nsplit, BiasStrips bias) {
  constexpr int BM = 2 * MT * 32, BN = 2 * NT * 32;
  typedef BackwardLds<MT, NT> L;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::BYTES];
  const int tiles = mtiles * ntiles * nsplit;
  if ((int)blockIdx.x >= tiles) {
    strip_sum<4>(*reinterpret_cast<float(*)[STRIP_PARTS][64]>(lds), bias.parts, StripOut{{bias.dbias}}, bias.strips,
                 bias.cols, 1, ((int)blockIdx.x - tiles) * 64, 0);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  const int tile = xcd_tile(blockIdx.x, tiles);
  const int split = tile % nsplit, nt = tile / nsplit % ntiles, mt0 = tile / nsplit / ntiles;
  const int m0 = mt0 * BM, k0 = nt * BN;
  const int stages = (N + BWD_KB - 1) / BWD_KB;
  const int st0 = (int)((int64_t)stages * split / nsplit), st1 = (int)((int64_t)stages * (split + 1) / nsplit);
  typename L::Rows zs;
  zs.init(dz, m0, T, ldz, wave, lane);
  f32x16 acc[MT][NT];
  tile_zero(acc);
  backward_tile<MT, NT>(zs, w, s, N, K, k0, st0, st1, lds, wm, wn, lane, acc);
  const int r = lane & 31, g = lane >> 5;
  constexpr int CPT = ColumnStage<NT>::CPT;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = m0 + (wm * MT + m) * 32 + r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // MFMA rows R = 8 (j >> 2) + 4 g + (j & 3) and R + 16 of all tiles: CPT columns
      const int k = k0 + wn * (NT * 32) + CPT * column_of_row(8 * (j >> 2) + 4 * g + (j & 3));
      if (t >= T || k >= K) continue;  // K is a multiple of 32
      float v[CPT];
#pragma unroll
      for (int c = 0; c < CPT; ++c) v[c] = acc[m][c >> 1][j + 8 * (c & 1)];
      if (nsplit > 1) {
        float* p = parts + ((size_t)split * T + t) * (size_t)K + k;
#pragma unroll
        for (int c = 0; c < CPT; c += 4) *reinterpret_cast<f32x4*>(p + c) = f32x4{v[c], v[c + 1], v[c + 2], v[c + 3]};
      } else {
#pragma unroll
        for (int c = 0; c < CPT; ++c) v[c] *= alpha;
        store_bf16<CPT>(dx + (size_t)t * K + k, v, true, CPT);
      }
    }
  }
}

__global__ void __launch_bounds__(256) dx_combine_kernel(const float* __restrict__ parts, uint16_t* __restrict__ dx,
                                                         float alpha, int64_t pieces, int nsplit) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= pieces) return;
  f32x4 a[2] = {};
  for (int z = 0; z < nsplit; ++z) {
    const float* p = parts + ((size_t)z * pieces + id) * 8;
    a[0] += *reinterpret_cast<const f32x4*>(p);
    a[1] += *reinterpret_cast<const f32x4*>(p + 4);
  }
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = alpha * a[j >> 2][j & 3];
  store_bf16<8>(dx + (size_t)id * 8, v, true, 8);
}

// ------------------------------------------------------------------ launch plans

TilePlan backward_plan(int64_t T, int64_t K, int64_t N) {
  TilePlan p{};
  p.mt = T <= 64 ? 1 : tile_choice(T, K, BACKWARD_ROUND_256, BACKWARD_ROUND_128);
  p.nt = p.mt == 4 ? 4 : 2;
  const int bm = 64 * p.mt, bn = 64 * p.nt;
  p.mtiles = (int)((T + bm - 1) / bm);
  p.ntiles = (int)((K + bn - 1) / bn);
  const int64_t stages = (N + BWD_KB - 1) / BWD_KB;
  p.nsplit = (int)tile_split((int64_t)p.mtiles * p.ntiles, stages / 2, p.mt == 2 && stages >= 64);
  if (p.nsplit > 1) p.bytes = (size_t)p.nsplit * T * K * 4;
  return p;
}

// Rows per strip of the dz launch: enough workgroups for the chip, whole groups of 8 rows (64
// rows of 4096 as one strip, which writes the bias gradient itself: 7.2 us; as 8: 3.4).
int dz_strip_rows(int64_t T, int64_t cols) {
  const int64_t ctiles = (cols + DZ_COLS - 1) / DZ_COLS;
  const int64_t want = std::max<int64_t>(1, 4 * GPU_CUS / ctiles);
  int64_t rows = (T + want - 1) / want;
  rows = std::max<int64_t>(8, (rows + 7) / 8 * 8);
  return (int)rows;
}

BackwardPlan backward_workspace(int64_t T, int64_t K, int64_t N, int64_t cols, bool need_dz, bool dx, bool dbias) {
  BackwardPlan b{};
  b.ldz = (int)((N + BWD_KB - 1) / BWD_KB * BWD_KB);  // whole stages, zeros past N
  b.strip_rows = dz_strip_rows(T, cols);
  b.strips = (int)((T + b.strip_rows - 1) / b.strip_rows);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  if (need_dz && dx) b.dz = take((size_t)T * b.ldz * 2);
  if (dbias && b.strips > 1) b.bias_parts = take((size_t)b.strips * N * 4);
  if (dx) {
    b.tile = backward_plan(T, K, N);
    b.parts = take(b.tile.bytes);
  }
  b.bytes = off;
  return b;
}

// dx, and the sums of the bias gradient's strips if there are any.
static int launch_dx(const uint16_t* dz, int ldz, const uint8_t* w, const uint8_t* s, uint16_t* dx, float alpha,
                     const TilePlan& p, float* parts, int T, int K, int N, const BiasStrips& bias, hipStream_t stream) {
  const int sums = bias.strips > 1 ? (bias.cols + 63) / 64 : 0;
  const dim3 grid((unsigned)(p.mtiles * p.ntiles * p.nsplit + sums));
#define MX_TILE(MT, NT)                                                                                        \
  hipLaunchKernelGGL((backward_kernel<MT, NT>), grid, dim3(256), 0, stream, dz, w, s, dx, parts, alpha, T, K, N, \
                     ldz, p.mtiles, p.ntiles, p.nsplit, bias)
  if (p.mt == 4)
    MX_TILE(4, 4);
  else if (p.mt == 2)
    MX_TILE(2, 2);
  else
    MX_TILE(1, 2);
#undef MX_TILE
  if (p.nsplit > 1) {
    const int64_t pieces = (int64_t)T * (K / 8);
    hipLaunchKernelGGL(dx_combine_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, stream, parts, dx, alpha,
                       pieces, p.nsplit);
  }
  return hip_status(hipGetLastError());
}

int launch_linear_fused_backward(const uint16_t* dy, const uint16_t* z, const uint8_t* w, const uint8_t* s, float scale,
                                 int act, uint16_t* dx, float* dbias, int T, int K, int N, void* workspace,
                                 hipStream_t stream) {
  const LinearSlope slope{dy, z, N, act, scale};
  const bool direct = !z && N % BWD_KB == 0;  // dz / alpha is dy itself
  const BackwardPlan b = backward_workspace(T, K, N, N, !direct, dx != nullptr, dbias != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* dz = (dx && !direct) ? reinterpret_cast<uint16_t*>(ws + b.dz) : nullptr;
  float* bp = !dbias ? nullptr : b.strips > 1 ? reinterpret_cast<float*>(ws + b.bias_parts) : dbias;
  if (dz || bp) {
    const dim3 grid((b.ldz + DZ_COLS - 1) / DZ_COLS, b.strips);
    hipLaunchKernelGGL((dz_kernel<LinearSlope>), grid, dim3(256), 0, stream, slope, dz, b.ldz, bp, (int64_t)T,
                       b.strip_rows);
    if (hipGetLastError() != hipSuccess) return MX_ERR_HIP;
  }
  if (!dx) return b.strips > 1 ? launch_strip_sum(bp, b.strips, N, 1, &dbias, stream) : MX_OK;
  return launch_dx(direct ? dy : dz, direct ? N : b.ldz, w, s, dx, slope.alpha(), b.tile,
                   reinterpret_cast<float*>(ws + b.parts), T, K, N, BiasStrips{bp, dbias, bp ? b.strips : 0, N}, stream);
}

int launch_gate_up_backward(const uint16_t* dh, const uint16_t* z, const uint8_t* w, const uint8_t* s, int act,
                            uint16_t* dx, float* dbias, int T, int H, int I, void* workspace, hipStream_t stream) {
  const BackwardPlan b = backward_workspace(T, H, 2 * (int64_t)I, I, true, dx != nullptr, dbias != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* dz = dx ? reinterpret_cast<uint16_t*>(ws + b.dz) : nullptr;
  float* bp = !dbias ? nullptr : b.strips > 1 ? reinterpret_cast<float*>(ws + b.bias_parts) : dbias;
  const dim3 grid((I + DZ_COLS - 1) / DZ_COLS, b.strips);
  hipLaunchKernelGGL(dz_gated_kernel, grid, dim3(256), 0, stream, dh, z, I, act, dz, b.ldz, bp, (int64_t)T, b.strip_rows);
  if (hipGetLastError() != hipSuccess) return MX_ERR_HIP;
  if (!dx) return b.strips > 1 ? launch_strip_sum(bp, b.strips, 2 * I, 1, &dbias, stream) : MX_OK;
  return launch_dx(dz, b.ldz, w, s, dx, 1.f, b.tile, reinterpret_cast<float*>(ws + b.parts), T, H, 2 * I,
                   BiasStrips{bp, dbias, bp ? b.strips : 0, 2 * I}, stream);
}

}  // namespace mx
