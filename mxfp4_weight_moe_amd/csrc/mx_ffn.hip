// Dense feed-forward operators around MXFP4 weights, forward:
//   linear   y = residual + scale * act(x W^T + bias)
//   gate_up  h = act(x Wg^T + bg) * (x Wu^T + bu)     (gate rows [0, I), up rows [I, 2I) of W)
// All products are exact in fp32 (bf16 x E2M1 * 2^s) and accumulate in fp32; bias, activation,
// product, scale and residual are applied to the fp32 sums, and each output is rounded once.
//
// Two kernels, by the number of tokens:
//   * up to STREAM_MAX_T a workgroup owns 16 weight rows (gate_up: 16 gate and the 16 up rows
//     of the same columns), its waves split K, and every weight byte is read once: the time is
//     the weight bytes' (stream_kernel);
//   * beyond, tiles of tokens x rows (mx_tile.hpp), where the matrix instructions set the
//     time; K is split over several workgroups while there are fewer tiles than CUs, and the
//     fp32 parts are summed in a fixed order by a second launch (combine_kernel).
#include "mx_epilogue.hpp"
#include "mx_tile.hpp"

namespace mx {

constexpr int STREAM_MAX_T = 32;

// ------------------------------------------------------------------ few tokens: weight streaming

template <bool GATED>
struct EpilogueOf {
  typedef LinearEpilogue type;
};
template <>
struct EpilogueOf<true> {
  typedef GatedEpilogue type;
};

// SBYTE: scale rows whose length is no multiple of 8 bytes (K % 256 != 0) go byte by byte.
template <int W, int MT, bool GATED, bool SBYTE>
__global__ void __launch_bounds__(W * 64) stream_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w,
                                                        const uint8_t* __restrict__ s,
                                                        typename EpilogueOf<GATED>::type epi, int T, int K, int rows) {
  constexpr int NS = GATED ? 2 : 1;
  constexpr int D = (MT * NS == 1) ? 4 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t slabs[W][NS * SLAB_BYTES];
  __shared__ f32x4 red[(W > 1) ? W * NS * MT * 64 : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n0 = blockIdx.x * SUB_ROWS;
  StreamLanes<NS, MT> L;
  lanes_init_lds(L, lane);
  const size_t kb = (size_t)(K >> 1), ks = (size_t)(K >> 5);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const size_t first = (size_t)i * rows;  // up rows follow the gate rows
#pragma unroll
    for (int q = 0; q < 2; ++q)
      L.w[i][q] = w + (first + min(n0 + (lane >> 3) + 8 * q, rows - 1)) * kb + (lane & 7) * 16;
    L.s[i] = s + (first + min(n0 + (lane & 15), rows - 1)) * ks;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = mt * 16 + (lane & 15);
    L.x[mt] = t < T ? x + (size_t)t * K + 32 * (lane >> 4) : nullptr;
  }
  const int nseg = K / SEG_K, nb_tail = (K % SEG_K) / 32;
  const int sg0 = (int)((long)nseg * wave / W), sg1 = (int)((long)nseg * (wave + 1) / W);
  f32x4 acc[MT][NS];
  acc_zero(acc);
  if (SBYTE) {
    Stage<NS, MT> st;
    stage_zero_x(st);
    for (int sg = sg0; sg < sg1; ++sg) {
      stage_load_tail<NS, MT>(st, L, sg, 8, lane);
      stage_compute(st, L, slabs[wave], acc);
    }
    if (wave == W - 1 && nb_tail > 0) {
      stage_load_tail<NS, MT>(st, L, nseg, nb_tail, lane);
      stage_compute(st, L, slabs[wave], acc);
    }
  } else {
    stream_segments<NS, MT, D>(L, sg0, sg1, 0, slabs[wave], acc, lane);
  }
  wg_reduce<NS, MT, W>(acc, red, wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = mt * 16 + (lane & 15);
    if (t >= T) continue;
    float v[NS][4];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = acc[mt][i][j];
    if constexpr (GATED)
      epi.template store<4>(t, n0 + 4 * (lane >> 4), v[0], v[1]);
    else
      epi.template store<4>(t, n0 + 4 * (lane >> 4), v[0]);
  }
}

// ------------------------------------------------------------------ many tokens: tiles

// Columns per row of the fp32 parts of a split K: each half of gate_up, or all rows of a
// linear layer, rounded up so that a lane's 8 or 16 consecutive values always fit.
static inline int part_cols(int rows, bool gated) { return gated ? (rows + 7) / 8 * 8 : (rows + 15) / 16 * 16; }

// rows: output columns (N, or I for gate_up).  nsplit > 1: part z of K goes to parts[z] as
// fp32 [T][part columns (x 2)].
template <int MT, int WM, int WN, bool GATED>
__global__ void __launch_bounds__(WM * WN * 64, 2)
    forward_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint8_t* __restrict__ s,
                   typename EpilogueOf<GATED>::type epi, float* __restrict__ parts, int T, int K, int rows, int mtiles,
                   int ntiles, int nsplit) {
  constexpr int BM = WM * MT * 16, COLS = GATED ? WN * 32 : WN * 64;
  typedef RowStage<BM, FWD_KB, WM * WN> XStage;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * XStage::BYTES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int tile = xcd_tile(blockIdx.x, mtiles * ntiles * nsplit);
  const int split = tile % nsplit, nt = tile / nsplit % ntiles, mt0 = tile / nsplit / ntiles;
  const int m0 = mt0 * BM, n0 = nt * COLS;
  const int stages = (K + FWD_KB - 1) / FWD_KB;
  const int st0 = (int)((int64_t)stages * split / nsplit), st1 = (int)((int64_t)stages * (split + 1) / nsplit);
  XStage xs;
  xs.init(x, m0, T, K, wave, lane);
  const int r = lane & 15, g = lane >> 4;
  // weight row of MFMA row r of tile i, so that a lane's results are consecutive columns:
  // linear 16 of them (16g + 4i + j), gate_up 8 gate (i = 0, 1) and 8 up (i = 2, 3)
  const uint8_t* wrow[4];
  const uint8_t* srow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int n = GATED ? n0 + wn * 32 + 8 * (r >> 2) + 4 * (i & 1) + (r & 3) : n0 + wn * 64 + 16 * (r >> 2) + 4 * i + (r & 3);
    n = min(n, rows - 1);
    const size_t row = (GATED && i >= 2) ? (size_t)rows + n : (size_t)n;
    wrow[i] = w + row * (size_t)(K >> 1);
    srow[i] = s + row * (size_t)(K >> 5);
  }
  f32x4 acc[MT][4];
  tile_zero(acc);
  forward_tile<MT, WM, WN>(xs, wrow, srow, K, st0, st1, lds, wm, lane, acc);
  const int pc = GATED ? (rows + 7) / 8 * 8 : (rows + 15) / 16 * 16;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = m0 + wm * MT * 16 + m * 16 + r;
    if (t >= T) continue;
    if constexpr (GATED) {
      const int n = n0 + wn * 32 + 8 * g;
      if (nsplit > 1) {
        if (n >= pc) continue;
        float* p = parts + ((size_t)split * T + t) * (2 * (size_t)pc) + n;
        *reinterpret_cast<f32x4*>(p) = acc[m][0];
        *reinterpret_cast<f32x4*>(p + 4) = acc[m][1];
        *reinterpret_cast<f32x4*>(p + pc) = acc[m][2];
        *reinterpret_cast<f32x4*>(p + pc + 4) = acc[m][3];
      } else {
        float a[8], b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = acc[m][j >> 2][j & 3];
          b[j] = acc[m][2 + (j >> 2)][j & 3];
        }
        epi.template store<8>(t, n, a, b);
      }
    } else {
      const int n = n0 + wn * 64 + 16 * g;
      if (nsplit > 1) {
        if (n >= pc) continue;
        float* p = parts + ((size_t)split * T + t) * (size_t)pc + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(p + 4 * i) = acc[m][i];
      } else {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = acc[m][j >> 2][j & 3];
        epi.template store<16>(t, n, v);
      }
    }
  }
}

// Sums the parts of a split K in ascending order and applies the epilogue: 8 columns a thread.
template <bool GATED>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ parts,
                                                      typename EpilogueOf<GATED>::type epi, int T, int pc, int nsplit) {
  const int per_row = pc / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)T * per_row) return;
  const int t = (int)(id / per_row), n = (int)(id % per_row) * 8;
  const size_t ld = GATED ? 2 * (size_t)pc : (size_t)pc;
  const float* p = parts + (size_t)t * ld + n;
  const size_t step = (size_t)T * ld;
  f32x4 a[2] = {}, b[2] = {};
  for (int z = 0; z < nsplit; ++z, p += step) {
    a[0] += *reinterpret_cast<const f32x4*>(p);
    a[1] += *reinterpret_cast<const f32x4*>(p + 4);
    if constexpr (GATED) {
      b[0] += *reinterpret_cast<const f32x4*>(p + pc);
      b[1] += *reinterpret_cast<const f32x4*>(p + pc + 4);
    }
  }
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = a[j >> 2][j & 3], u[j] = b[j >> 2][j & 3];
  if constexpr (GATED)
    epi.template store<8>(t, n, v, u);
  else
    epi.template store<8>(t, n, v);
}

// ------------------------------------------------------------------ launch plans

// Which tile and how many parts of K.  Both depend on the sizes alone, so that the workspace a
// call needs does too.
TilePlan forward_plan(int64_t T, int64_t K, int64_t rows, bool gated) {
  TilePlan p{};
  if (T <= STREAM_MAX_T) return p;
  p.mt = T > 1024 ? 8 : T > 64 ? 4 : 2;
  p.wn = p.mt == 8 ? 4 : 2;
  const int bm = 32 * p.mt, cols = gated ? p.wn * 32 : p.wn * 64;
  p.mtiles = (int)((T + bm - 1) / bm);
  p.ntiles = (int)((rows + cols - 1) / cols);
  const int64_t tiles = (int64_t)p.mtiles * p.ntiles, stages = (K + FWD_KB - 1) / FWD_KB;
  int64_t split = tiles >= GPU_CUS ? 1 : GPU_CUS / tiles;
  p.nsplit = (int)std::max<int64_t>(1, std::min(split, stages / 2));
  if (p.nsplit > 1) p.bytes = (size_t)p.nsplit * T * part_cols((int)rows, gated) * (gated ? 2 : 1) * 4;
  return p;
}

template <bool GATED>
static int launch_forward(const uint16_t* x, const uint8_t* w, const uint8_t* s,
                          const typename EpilogueOf<GATED>::type& epi, void* workspace, int T, int K, int rows,
                          hipStream_t stream) {
  if (T <= STREAM_MAX_T) {
    const int items = (rows + SUB_ROWS - 1) / SUB_ROWS, nseg = K / SEG_K;
    int W = 1;
    while (W < 8 && 2 * W <= nseg && items * W < 2048) W *= 2;
    if (T > 16 && GATED) W = std::min(W, 4);
    const dim3 grid(items), block(W * 64);
#define MX_STREAM(WW, M, SB) \
  hipLaunchKernelGGL((stream_kernel<WW, M, GATED, SB>), grid, block, 0, stream, x, w, s, epi, T, K, rows)
#define MX_STREAM_W(WW)         \
  if (K % SEG_K == 0) {         \
    if (T > 16)                 \
      MX_STREAM(WW, 2, false);  \
    else                        \
      MX_STREAM(WW, 1, false);  \
  } else if (T > 16) {          \
    MX_STREAM(WW, 2, true);     \
  } else {                      \
    MX_STREAM(WW, 1, true);     \
  }
    if (W == 1) {
      MX_STREAM_W(1)
    } else if (W == 2) {
      MX_STREAM_W(2)
    } else if (W == 4) {
      MX_STREAM_W(4)
    } else {
      MX_STREAM_W(8)
    }
#undef MX_STREAM_W
#undef MX_STREAM
    return hip_status(hipGetLastError());
  }
  const TilePlan p = forward_plan(T, K, rows, GATED);
  float* parts = static_cast<float*>(workspace);
  const dim3 grid((unsigned)(p.mtiles * p.ntiles * p.nsplit));
#define MX_TILE(MT, WN)                                                                                           \
  hipLaunchKernelGGL((forward_kernel<MT, 2, WN, GATED>), grid, dim3(2 * WN * 64), 0, stream, x, w, s, epi, parts, T, K, \
                     rows, p.mtiles, p.ntiles, p.nsplit)
  if (p.mt == 8)
    MX_TILE(8, 4);
  else if (p.mt == 4)
    MX_TILE(4, 2);
  else
    MX_TILE(2, 2);
#undef MX_TILE
  if (p.nsplit > 1) {
    const int pc = part_cols(rows, GATED);
    const int64_t pieces = (int64_t)T * (pc / 8);
    hipLaunchKernelGGL((combine_kernel<GATED>), dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, stream, parts,
                       epi, T, pc, p.nsplit);
  }
  return hip_status(hipGetLastError());
}

int launch_linear_fused(const uint16_t* x, const uint8_t* w, const uint8_t* s, const uint16_t* bias,
                        const uint16_t* residual, float scale, int act, uint16_t* y, uint16_t* z, int T, int K, int N,
                        void* workspace, hipStream_t stream) {
  return launch_forward<false>(x, w, s, LinearEpilogue{bias, residual, y, z, N, act, scale}, workspace, T, K, N, stream);
}

int launch_gate_up_dense(const uint16_t* x, const uint8_t* w, const uint8_t* s, const uint16_t* bias, int act,
                         uint16_t* h, uint16_t* z, int T, int H, int I, void* workspace, hipStream_t stream) {
  return launch_forward<true>(x, w, s, GatedEpilogue{bias, h, z, I, act}, workspace, T, H, I, stream);
}

}  // namespace mx
