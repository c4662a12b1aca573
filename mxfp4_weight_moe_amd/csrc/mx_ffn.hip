// Dense feed-forward operators around MXFP4 weights, forward:
//   linear   y = residual + scale * act(x W^T + bias)
//   gate_up  h = act(x Wg^T + bg) * (x Wu^T + bu)     (gate rows [0, I), up rows [I, 2I) of W)
// All products are exact in fp32 (bf16 x E2M1 * 2^s) and accumulate in fp32; bias, activation,
// product, scale and residual are applied to the fp32 sums, and each output is rounded once.
//
// Three kernels, by the number of tokens:
//   * few (up to 8, some sizes to 16, odd K to 32; any for K < 128): a workgroup owns 16 weight rows, its
//     waves split K, and every weight byte is read once (stream_kernel);
//   * up to THIN_MAX_T a wave takes 32 tokens and 32 or 64 weight rows (thin_kernel);
//   * beyond, tiles of tokens x rows (mx_tile.hpp), where the matrix instructions set the time
//     (forward_kernel).
// In the last two K is split over several workgroups while there are fewer tiles than CUs; the
// fp32 parts are then summed in a fixed order by a second launch (combine_kernel).
#include "mx_epilogue.hpp"
#include "mx_grid.hpp"
#include "mx_tile_out.hpp"

namespace mx {

// ------------------------------------------------------------------ few tokens: weight streaming

template <bool GATED>
struct EpilogueOf {
  typedef LinearEpilogue type;
};
template <>
struct EpilogueOf<true> {
  typedef GatedEpilogue type;
};

// A workgroup has one MFMA tile of 16 weight rows: 16 rows of a linear layer, or 8 gate rows and
// the 8 up rows of the same columns (a tile of each would leave half the CUs idle at I = 2048).
// Bound by the latency of a workgroup's few serial steps: 7168 -> 4096 with 4 tokens takes
// 6.8 us (2.3 TB/s of weights), gate_up of 8 tokens, H = 7168, I = 2048, 7.5 us (9.9 with a tile
// of each).
// SBYTE: scale rows whose length is no multiple of 8 bytes (K % 256 != 0) go byte by byte.
// XL: the workgroup first copies x to LDS (dynamic, T * K bf16); read from memory, only T of
// every 16 lanes of a fragment load are active.
constexpr int STREAM_XL = 65536;  // values of x that fit beside the slabs
template <int W, int MT, bool GATED, bool SBYTE, bool XL>
__global__ void __launch_bounds__(W * 64) stream_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w,
                                                        const uint8_t* __restrict__ s,
                                                        typename EpilogueOf<GATED>::type epi, int T, int K, int rows) {
  constexpr int D = MT == 1 ? 4 : 2, COLS = GATED ? SUB_ROWS / 2 : SUB_ROWS;
  __shared__ __attribute__((aligned(16))) uint8_t slabs[W][SLAB_BYTES];
  __shared__ f32x4 red[(W > 1) ? W * MT * 64 : 1];
  extern __shared__ u32x4 xdyn[];
  static_assert(MT <= 2 && STREAM_MAX_T == 32, "a workgroup's tokens");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  // one tile of 16 tokens is all of them
  const int n0 = blockIdx.x * COLS, t0 = MT == 1 ? 0 : (blockIdx.z * gridDim.y + blockIdx.y) * STREAM_MAX_T;
  if (MT > 1 && t0 >= T) return;
  const size_t kb = (size_t)(K >> 1), ks = (size_t)(K >> 5);
  // weight row of MFMA row r; past the last row the last one again
  auto weight_row = [&](int r) {
    if (GATED) return (size_t)min(n0 + (r & 7), rows - 1) + (r >= 8 ? (size_t)rows : 0);
    return (size_t)min(n0 + r, rows - 1);
  };
  StreamLanes<1, MT> L;
  lanes_init_lds(L, lane);
#pragma unroll
  for (int q = 0; q < 2; ++q) L.w[0][q] = w + weight_row((lane >> 3) + 8 * q) * kb + (lane & 7) * 16;
  L.s[0] = s + weight_row(lane & 15) * ks;
  const uint16_t* xs = x;
  if constexpr (XL) {
    static_assert(MT == 1 && !SBYTE, "one tile of tokens, whole segments");
    // 8 loads of a thread in flight at once; a piece past the end is the last piece again
    const int n16 = T * K / 8, nt = W * 64, t = threadIdx.x;
    const u32x4* xv = reinterpret_cast<const u32x4*>(x);
    for (int i0 = t; i0 < n16; i0 += 8 * nt) {
      u32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = xv[min(i0 + u * nt, n16 - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u) xdyn[min(i0 + u * nt, n16 - 1)] = v[u];
    }
    __syncthreads();
    xs = reinterpret_cast<const uint16_t*>(xdyn);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = t0 + mt * 16 + (lane & 15);
    L.x[mt] = t < T ? xs + (size_t)t * K + 32 * (lane >> 4) : nullptr;
  }
  const int nseg = K / SEG_K, nb_tail = (K % SEG_K) / 32;
  const int sg0 = (int)((long)nseg * wave / W), sg1 = (int)((long)nseg * (wave + 1) / W);
  f32x4 acc[MT][1];
  acc_zero(acc);
  if constexpr (SBYTE) {
    Stage<1, MT> st;
    stage_zero_x(st);
    for (int sg = sg0; sg < sg1; ++sg) {
      stage_load_tail<1, MT>(st, L, sg, 8, lane);
      stage_compute(st, L, slabs[wave], acc);
    }
    if (wave == W - 1 && nb_tail > 0) {
      stage_load_tail<1, MT>(st, L, nseg, nb_tail, lane);
      stage_compute(st, L, slabs[wave], acc);
    }
  } else {
    stream_segments<1, MT, D, false, XL>(L, sg0, sg1, 0, slabs[wave], acc, lane);
  }
  wg_reduce<1, MT, W>(acc, red, wave, lane);
  if (wave != 0) return;
  const int g = lane >> 4, n = n0 + 4 * (GATED ? g & 1 : g);
  const auto cols = epi.template columns<4>(n);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = t0 + mt * 16 + (lane & 15);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = acc[mt][0][j];
    if constexpr (GATED) {
      float u[4];  // rows 8 and up of the tile: the lanes 32 on
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __shfl_xor(v[j], 32, 64);
      if (t < T && g < 2) epi.template store<4>(t, n, v, u, cols);
    } else {
      if (t < T) epi.template store<4>(t, n, v, cols, epi.template fetch<4>(t, n));
    }
  }
}

// ------------------------------------------------------------------ many tokens: tiles

// Bound by the matrix units and the power limit: with products alone the clock falls to 1.7 GHz,
// here they are busy for 68% of a launch's cycles (gate_up, epilogue included) at 1.85 GHz.
// 4096 tokens, 7168 -> 4096 with gelu, bias and residual 191 us, 1.26 PFLOP/s; gate_up of the same
// size with z kept 173 us.  The epilogue of a 256 x 256 tile (26 and 10 us of these) has nothing
// to overlap with: its accumulators fill the registers.
//
// rows: output columns (N, or I for gate_up).  nsplit > 1: part z of K goes to parts[z] as
// fp32 [T][part columns (x 2)].  A wave's NT MFMA tiles are 32 consecutive weight rows each;
// for gate_up the first half of them gate rows, the second half the up rows of the same columns.
// D: stages in the LDS (mx_tile.hpp).
template <int MT, int NT, int WM, int WN, int D, bool GATED>
__global__ void __launch_bounds__(WM * WN * 64, MT == 4 || D > 2 ? 1 : 2)
    forward_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint8_t* __restrict__ s,
                   typename EpilogueOf<GATED>::type epi, float* __restrict__ parts, int T, int K, int rows, int mtiles,
                   int ntiles, int nsplit) {
  constexpr int BM = WM * MT * 32, WCOLS = NT * 32 / (GATED ? 2 : 1), HALF = GATED ? NT / 2 : NT;
  typedef ForwardLds<MT, NT, WM, WN, D> L;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::BYTES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int tile = xcd_tile(blockIdx.x, mtiles * ntiles * nsplit);
  const int split = tile % nsplit, nt = tile / nsplit % ntiles, mt0 = tile / nsplit / ntiles;
  const int m0 = mt0 * BM, n0 = nt * (WN * WCOLS);
  const int stages = (K + FWD_KB - 1) / FWD_KB;
  const int st0 = (int)((int64_t)stages * split / nsplit), st1 = (int)((int64_t)stages * (split + 1) / nsplit);
  typename L::Rows xs;
  xs.init(x, m0, T, K, wave, lane);
  // Row r of MFMA tile i (of WN * NT), counted from the tile's first row (32-bit offsets) in
  // the gate or the up half; past the last row the last one again.
  auto row_of = [&](int lr) {
    const int i = lr >> 5;
    return min(i / NT * WCOLS + i % HALF * 32 + (lr & 31), rows - 1 - n0);
  };
  auto first_row = [&](int i) { return (size_t)n0 + (i % NT >= HALF ? (size_t)rows : 0); };
  typename L::Codes cs;
  cs.init(K, min(WN * WCOLS, rows - n0), wave, lane, [&](int i) { return w + first_row(i) * (size_t)(K >> 1); }, row_of);
  const uint8_t* sbase[NT];
  uint32_t soff[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    sbase[i] = s + first_row(i) * (size_t)(K >> 5);
    soff[i] = (uint32_t)row_of((wn * NT + i) * 32 + (lane & 31)) * (uint32_t)(K >> 5);
  }
  typename L::Scales ss;
  if constexpr (D > 2) {  // 32-bit offsets from the first gate row to the up rows (forward_deep)
    ss.wave = wave;
    ss.buf_ = make_buffer(sbase[0], ((uint64_t)min(WN * WCOLS, rows - n0) + (GATED ? rows : 0)) * (uint64_t)(K >> 5));
#pragma unroll
    for (int q = 0; q < L::Scales::COPIES; ++q) {
      const int i = 2 * q + (lane >> 5);
      const uint32_t row = (uint32_t)row_of((wn * NT + i) * 32 + (lane & 31));
      ss.off[q] = (row + (i >= HALF ? (uint32_t)rows : 0u)) * (uint32_t)(K >> 5);
    }
  }
  f32x16 acc[MT][NT];
  tile_zero(acc);
  forward_tile<MT, NT, WM, WN, D>(xs, cs, ss, sbase, (uint32_t)(min(WN * WCOLS, rows - n0) * (K >> 5)), soff, K, st0,
                                  st1, lds, wm, wn, lane, acc);

  tile_output<MT, NT, WM, WN, GATED, L::BYTES>(acc, epi, parts, lds, T, rows, m0, n0, split, nsplit, wave, lane);
}

// ------------------------------------------------------------------ up to 128 tokens: thin tiles

// A workgroup takes 32 NT weight rows (gate_up: half of them gate rows, half the up rows of the
// same columns) and a wave each 32 tokens.  A wave loads everything it needs by itself, its
// activation rows and its own copy of the codes and scales, into a ring of its own in the LDS:
// no barriers in the loop.  Up to 64 tokens the waves that are left over split K.  Where 32 rows
// a workgroup give three quarters of the CUs one, K is not split over workgroups, whose second
// launch costs 3 to 4 us at these sizes; with fewer rows and more than 64 tokens NT = 2 halves the
// activations that a CU reads beside the same weights, and K is split (gate_up of 128 tokens,
// H = 7168, I = 2048: 20.2 us, with NT = 1 and 128 workgroups 21.4).  A CU then reads 0.70 MB
// through its L2: 0.46 MB of activations, and its 57 KB of codes and 4 KB of scales four times, once
// for each wave, which each decodes; about 20 bytes a cycle over the launch's 15 to 17 us.  That the
// read path is what bounds it has not been shown.  77 tokens, 2048 -> 7168: 10 us.  Tiles of
// 128 x 128 with barriers took 17 and 25 us.
constexpr int THIN_MAX_T = 128;
template <int NT>
struct ThinStage {
  static constexpr int D = 3;  // stages in the ring
  static constexpr int CODES = 32 * 256, SCALES = CODES + NT * 32 * 64, BYTES = SCALES + 256;
  static constexpr int LOADS = 8 + 2 * NT + 1;  // a stage's copies to LDS
};

// KS: waves to the same 32 tokens, among which K is split; their sums meet in the LDS.
template <int NT, bool GATED, int KS>
__global__ void __launch_bounds__(256, 1)
    thin_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint8_t* __restrict__ s,
                typename EpilogueOf<GATED>::type epi, float* __restrict__ parts, int T, int K, int rows, int ntiles,
                int nsplit) {
  typedef ThinStage<NT> L;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * L::D * L::BYTES];
  constexpr int COLS = GATED ? 16 * NT : 32 * NT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tile = xcd_tile(blockIdx.x, ntiles * nsplit);
  const int split = tile % nsplit, n0 = tile / nsplit * COLS, m0 = wave / KS * 32;
  const int stages = K / FWD_KB, part = split * KS + wave % KS, of = nsplit * KS;
  const int st0 = (int)((int64_t)stages * part / of), st1 = (int)((int64_t)stages * (part + 1) / of);
  uint8_t* ring = lds + wave * (L::D * L::BYTES);

  // Rows that do not exist lie past the end of their buffers and read as zero.
  const buffer xbuf = make_buffer(x + (size_t)m0 * K, (uint64_t)min(32, T - m0) * (uint64_t)K * 2);
  uint32_t xoff[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int r = q * 4 + (lane >> 4);
    xoff[q] = (uint32_t)r * (uint32_t)(K * 2) + (((lane & 15) ^ (r & 15)) << 4);
  }
  // Row lr of the workgroup's 32 NT: weight row n0 + lr, or column n0 + lr % COLS of half lr / COLS.
  buffer wbuf[2 * NT];
  uint32_t woff[2 * NT];
#pragma unroll
  for (int q = 0; q < 2 * NT; ++q) {
    const int r = q * 16 + (lane >> 2), c = GATED ? q * 16 % COLS : q * 16;
    const int have = max(0, min(16, rows - n0 - c));
    const size_t first = (size_t)n0 + c + (GATED && q >= NT ? (size_t)rows : 0);
    wbuf[q] = make_buffer(w + first * (size_t)(K >> 1), (uint64_t)have * (uint64_t)(K >> 1));
    woff[q] = (uint32_t)(lane >> 2) * (uint32_t)(K >> 1) + (((lane & 3) ^ ((r >> 3) & 3)) << 4);
  }
  const buffer sbuf = make_buffer(s + (size_t)n0 * (K >> 5),
                                  ((uint64_t)min(COLS, rows - n0) + (GATED ? rows : 0)) * (uint64_t)(K >> 5));
  const int slr = lane & (32 * NT - 1);
  const uint32_t soff = (GATED && slr >= COLS ? (uint32_t)rows + slr - COLS : (uint32_t)slr) * (uint32_t)(K >> 5);
  auto load = [&](int st, uint8_t* buf) {
#pragma unroll
    for (int q = 0; q < 8; ++q) copy16_to_lds(xbuf, xoff[q], (uint32_t)st * 256, buf + q * 1024);
#pragma unroll
    for (int q = 0; q < 2 * NT; ++q) copy16_to_lds(wbuf[q], woff[q], (uint32_t)st * 64, buf + L::CODES + q * 1024);
    copy4_to_lds(sbuf, soff, (uint32_t)st * 4, buf + L::SCALES);
  };
  const int r = lane & 31, g = lane >> 5;
  struct Operands {
    u32x4 x[8], code[NT][2];
    uint32_t scale[NT];
  };
  auto read = [&](const uint8_t* buf) {
    Operands o;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      o.scale[i] = *reinterpret_cast<const uint32_t*>(buf + L::SCALES + (i * 32 + r) * 4);
#pragma unroll
      for (int b = 0; b < 2; ++b)
        o.code[i][b] = ld16(buf + L::CODES + (i * 32 + r) * 64 + (((2 * b + g) ^ (r >> 3)) << 4));
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) o.x[u] = ld16(buf + r * 256 + (((8 * (u >> 2) + 4 * g + (u & 3)) ^ (r & 15)) << 4));
    return o;
  };
  f32x16 acc[2][NT] = {};  // even and odd steps: chains of products that do not wait for one another
  uint8_t* cur = ring;
  uint8_t* nxt = ring + L::BYTES;
  uint8_t* fill = ring + 2 * L::BYTES;
  static_assert(L::D == 3, "three buffers");
  Operands o{};
  if (KS == 1 || st0 < st1) {  // K may have fewer stages than parts
    load(st0, cur);
    load(min(st0 + 1, st1 - 1), nxt);
    wait_copies<L::LOADS>();
    o = read(cur);
  }
  for (int st = st0; st < st1; ++st) {
    load(min(st + 2, st1 - 1), fill);  // its last content was used two stages ago
    wait_copies<L::LOADS>();           // the next stage has landed
    const Operands next = read(nxt);
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint32_t d = o.scale[i] >> (8 * g);
        const float sc = e8m0_scale_operand(u < 4 ? d & 0xFFu : (d >> 16) & 0xFFu);
        acc[u & 1][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(decode8(o.code[i][u >> 2][u & 3], sc),
                                                                as_bf16x8(o.x[u]), acc[u & 1][i], 0, 0, 0);
      }
    o = next;
    uint8_t* t = cur;
    cur = nxt;
    nxt = fill;
    fill = t;
  }
  wait_copies();  // the repeated copies of the last stages: the ring is used again
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[0][i] += acc[1][i];
  tile_to_lds<NT>(ring, acc[0], lane);
  const int pc = part_cols(rows);
  constexpr int PIECES = COLS / 8, ROWS = 64 / PIECES;
  const int p = lane % PIECES, n = n0 + p * 8;
  const auto cols = epi.template columns<8>(n);
  // each of the KS waves sums its share of the rows
  constexpr int SHARE = 32 / KS, ITERS = (SHARE + ROWS - 1) / ROWS;
  const uint8_t* first = lds + wave / KS * KS * (L::D * L::BYTES);
  if constexpr (KS > 1) __syncthreads();
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int row = it * ROWS + lane / PIECES + wave % KS * SHARE, t = m0 + row;
    if (t >= T || n >= rows || (ROWS > SHARE && lane / PIECES >= SHARE)) continue;
    f32x4 q[GATED ? 4 : 2];
#pragma unroll
    for (int j = 0; j < (GATED ? 4 : 2); ++j) {
      const uint32_t at = out_at<NT>(row, 2 * p + (j & 1) + (j >> 1) * (4 * NT));
      q[j] = *reinterpret_cast<const f32x4*>(first + at);
#pragma unroll
      for (int k = 1; k < KS; ++k) q[j] += *reinterpret_cast<const f32x4*>(first + k * (L::D * L::BYTES) + at);
    }
    if (nsplit > 1) {
      float* o2 = parts + ((size_t)split * T + t) * ((GATED ? 2 : 1) * (size_t)pc) + n;
#pragma unroll
      for (int j = 0; j < (GATED ? 4 : 2); ++j) *reinterpret_cast<f32x4*>(o2 + (j >> 1) * pc + (j & 1) * 4) = q[j];
      continue;
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q[j >> 2][j & 3];
    if constexpr (GATED) {
      float u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = q[2 + (j >> 2)][j & 3];
      epi.template store<8>(t, n, v, u, cols);
    } else {
      epi.template store<8>(t, n, v, cols, epi.template fetch<8>(t, n));
    }
  }
}

// ------------------------------------------------------------------ launch plans

// Whether the up rows' scales lie within 32-bit offsets of the gate rows'.
static bool scales_in_reach(int64_t K, int64_t rows, bool gated) {
  return !gated || rows * (K >> 5) < ((int64_t)1 << 31);
}
// Thin tiles from 9 tokens on (5, see below), or from 17 where one round of workgroups streams the weights with
// the activations in the LDS (4096 -> 4096, 16 tokens: 6.5 us against 6.9; 4096 -> 7168, two
// rounds: 11.3 against 7.5; at 8 tokens 6.7 and 6.9; 4096 -> 4096 at 32 tokens: 11.4 and 7.0).
// Streaming scales byte by byte (K % 256 != 0) ends earlier: 4224 -> 5000, 8 tokens, 9.9 and 6.9.
static bool takes_thin(int64_t T, int64_t K, int64_t rows, bool gated) {
  if (T <= (K % SEG_K == 0 ? 8 : 4) || T > THIN_MAX_T || K % FWD_KB != 0 || !scales_in_reach(K, rows, gated)) return false;
  return T > 16 || K % SEG_K != 0 || T * K > STREAM_XL || rows > GPU_CUS * (gated ? SUB_ROWS / 2 : SUB_ROWS);
}
static bool takes_stream(int64_t T, int64_t K, int64_t rows, bool gated) {
  return K < FWD_KB || (T <= STREAM_MAX_T && !takes_thin(T, K, rows, gated));
}

// Which tile and how many parts of K.  Both depend on the sizes alone, so that the workspace a
// call needs does too.
TilePlan forward_plan(int64_t T, int64_t K, int64_t rows, bool gated) {
  TilePlan p{};
  if (takes_stream(T, K, rows, gated)) return p;
  const int64_t stages = (K + FWD_KB - 1) / FWD_KB;
  int64_t split;
  if (takes_thin(T, K, rows, gated)) {
    // Waves of a workgroup that 32-token groups leave split K; over workgroups it is split where
    // that saves a wave 12 stages or more, 4 left at least: with fewer the second launch costs
    // more (up to 32 tokens 8192 -> 1000: 9.8 us whole, 8.5 in 4 parts; gate_up with H = 4096,
    // I = 500: 7.1 and 8.9 in 2).
    p.mtiles = 1;
    p.thin = 1;
    p.ks = T <= 32 ? 4 : T <= 64 ? 2 : 1;
    p.ntiles = (int)((rows + (gated ? 15 : 31)) / (gated ? 16 : 32));
    const int64_t per_wave = stages / p.ks;
    const int pairs = (p.ntiles + 1) / 2;
    const bool wide = p.ks == 1 && 4 * p.ntiles < 3 * GPU_CUS;  // see thin_kernel
    split = std::max<int64_t>(1, std::min<int64_t>(GPU_CUS / (wide ? pairs : p.ntiles), per_wave / 4));
    if (per_wave - per_wave / split < 12) {
      split = 1;
    } else if (wide) {
      p.thin = 2;
      p.ntiles = pairs;
    }
  } else {
    p.mt = T <= 64 ? 1 : tile_choice(T, rows * (gated ? 2 : 1), FORWARD_ROUND_256, FORWARD_ROUND_128);
    p.nt = p.mt == 4 ? 4 : 2;
    const int bm = 64 * p.mt, cols = (gated ? 32 : 64) * p.nt;
    p.mtiles = (int)((T + bm - 1) / bm);
    p.ntiles = (int)((rows + cols - 1) / cols);
    split = tile_split((int64_t)p.mtiles * p.ntiles, stages, p.mt == 2 && stages >= 32);
  }
  p.nsplit = (int)std::max<int64_t>(1, split);
  if (p.nsplit > 1) p.bytes = (size_t)p.nsplit * T * part_cols((int)rows) * (gated ? 2 : 1) * 4;
  return p;
}

template <bool GATED>
static int launch_forward(const uint16_t* x, const uint8_t* w, const uint8_t* s,
                          const typename EpilogueOf<GATED>::type& epi, void* workspace, int T, int K, int rows,
                          hipStream_t stream) {
  if (takes_stream(T, K, rows, GATED)) {
    const int cols = GATED ? SUB_ROWS / 2 : SUB_ROWS;
    const StreamGrid sg = stream_grid(T, rows, cols);
    const int items = (int)sg.items, nseg = K / SEG_K;
    int W = 1;
    // as many waves as the CUs hold at once: at more than 256 workgroups of 8 a second round begins
    // (4096 -> 7168, one token: 7.3 us with 8 waves, 5.4 with 4)
    while (W < 8 && 2 * W <= nseg && 2 * W * items <= 2048) W *= 2;
    // up to 16 tokens in whole segments, up to 32 byte by byte; K % 256 == 0 with more than 16 is
    // left for gate_up alone, where its scales are too far apart for the thin tiles
    const bool sbyte = K % SEG_K != 0 || T > 16, xl = T <= 16 && !sbyte && (int64_t)T * K <= STREAM_XL;
    const dim3 grid(sg.items, sg.y, sg.z), block(W * 64);
    const unsigned xl_bytes = xl ? (unsigned)(T * K * 2) : 0u;
#define MX_STREAM(WW, M, SB, XX) \
  hipLaunchKernelGGL((stream_kernel<WW, M, GATED, SB, XX>), grid, block, xl_bytes, stream, x, w, s, epi, T, K, rows)
#define MX_STREAM_W(WW)               \
  if (xl)                             \
    MX_STREAM(WW, 1, false, true);    \
  else if (!sbyte)                    \
    MX_STREAM(WW, 1, false, false);   \
  else if (T <= 16)                   \
    MX_STREAM(WW, 1, true, false);    \
  else                                \
    MX_STREAM(WW, 2, true, false)
    if (W == 1) {
      MX_STREAM_W(1);
    } else if (W == 2) {
      MX_STREAM_W(2);
    } else if (W == 4) {
      MX_STREAM_W(4);
    } else {
      MX_STREAM_W(8);
    }
#undef MX_STREAM_W
#undef MX_STREAM
    return hip_status(hipGetLastError());
  }
  const TilePlan p = forward_plan(T, K, rows, GATED);
  float* parts = static_cast<float*>(workspace);
  const dim3 grid((unsigned)(p.mtiles * p.ntiles * p.nsplit));
  // One tile a CU and K in whole stages: more stages in the LDS (gate_up with H = 7168,
  // I = 2048: 256 tokens 30.6 us, 31.4 with two stages; 500 tokens 42.8 and 44.8).
  const bool deep = (int64_t)p.mtiles * p.ntiles * p.nsplit <= GPU_CUS && K % FWD_KB == 0 &&
                    scales_in_reach(K, rows, GATED);
#define MX_TILE(MT, NT, D)                                                                                           \
  hipLaunchKernelGGL((forward_kernel<MT, NT, 2, 2, D, GATED>), grid, dim3(256), 0, stream, x, w, s, epi, parts, T, K, \
                     rows, p.mtiles, p.ntiles, p.nsplit)
#define MX_THIN(NT, KS)                                                                                                 \
  hipLaunchKernelGGL((thin_kernel<NT, GATED, KS>), grid, dim3(64 * KS * ((T + 31) / 32)), 0, stream, x, w, s, epi, parts, \
                     T, K, rows, p.ntiles, p.nsplit)
  if (p.thin == 2)
    MX_THIN(2, 1);
  else if (p.thin && p.ks == 4)
    MX_THIN(1, 4);
  else if (p.thin && p.ks == 2)
    MX_THIN(1, 2);
  else if (p.thin)
    MX_THIN(1, 1);
  else if (p.mt == 4)
    MX_TILE(4, 4, 2);
  else if (p.mt == 2 && deep)
    MX_TILE(2, 2, 3);
  else if (p.mt == 2)
    MX_TILE(2, 2, 2);
  else
    MX_TILE(1, 2, 2);
#undef MX_TILE
#undef MX_THIN
  if (p.nsplit > 1) {
    const int pc = part_cols(rows);
    const int64_t pieces = (int64_t)T * (pc / 8);
    hipLaunchKernelGGL((combine_kernel<GATED, typename EpilogueOf<GATED>::type>), dim3((unsigned)((pieces + 63) / 64)), dim3(64), 0, stream, parts,
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
