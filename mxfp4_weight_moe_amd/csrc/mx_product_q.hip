// Dense feed-forward operators whose activations are microscaled already:
//   linear   y = residual + scale * act(a W^T + bias)
//   gate_up  h = act(a Wg^T + bg) * (a Wu^T + bu)     (gate rows [0, I), up rows [I, 2I) of W)
// a in MXFP8 or MXFP4, W in MXFP4, fp32 sums; h in bf16, or quantized again from its fp32 value.
//
// Three kernels, by the number of tokens: up to 16 (32 where thin tiles do not apply) the weights are
// streamed once, a workgroup to 16 weight rows (stream_q_kernel); up to 64 a workgroup has all tokens and 32 or
// 64 weight rows, its waves splitting K (thin_q_kernel); beyond, tiles (mx_tile_q.hpp).
#include "mx_grid.hpp"
#include "mx_tile_out.hpp"
#include "mx_tile_q.hpp"

namespace mx {

// h leaves as codes and scales.  I % 32 == 0: the 8 columns of each of 4 lanes are a block.
template <int FMT>
struct GatedQuantEpilogue : GatedEpilogue {
  static constexpr bool WHOLE_BLOCKS = true;
  uint8_t* codes;   // [T, I] or [T, I / 2]
  uint8_t* scales;  // [T, I / 32]
  template <int V>
  __device__ __forceinline__ void store(int t, int n, float (&g)[V], float (&u)[V], const Columns<V>& c) const {
    static_assert(V == 8, "a quad of lanes is a block");
    if (n >= I) return;
    product<V>(t, n, g, u, c);
    uint32_t q[FMT / 4], byte;
    quantize8<FMT>(g, q, byte);
    store_codes8<FMT>(codes, scales, ((size_t)t * I + n) / 8, q, byte);
  }
};

// What a product reads.
struct QOperands {
  const uint8_t* a;   // [T, K] (MXFP8) or [T, K / 2]
  const uint8_t* as;  // [T, K / 32]
  const uint8_t* w;   // [rows (x 2), K / 2]
  const uint8_t* ws;  // [rows (x 2), K / 32]
};

// ------------------------------------------------------------------ few tokens: weight streaming

constexpr int STREAM_Q_MAX_T = 32;

// v_mfma_scale_f32_16x16x128_f8f6f4: lane (r = lane & 15, g = lane >> 4) gives E2M1 block g of row r, or
// E4M3 values 16 g .. + 15 of both halves of the 128.
template <int FMT>
__device__ __forceinline__ f32x4 mfma_stream_q(const u32x4& w, const QFragment<FMT>& a, f32x4 c, int sw, int sa) {
  const i32x8 wo = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wo, q_operand(a), c, 4, FMT == 8 ? 0 : 4, 0, sw, 0, sa);
}

// A workgroup has 16 weight rows (gate_up: 8 gate rows and the 8 up rows of the same columns), its W
// waves split K.  A lane loads its operands straight from memory, 256 values (Q_UNIT) at a time and 4 of
// those ahead: two 16-byte pieces of a weight row, four (two) of a token, 8 scale bytes of each.
// Bound by latency: 7168 -> 4096, 15.6 MB, takes 6.5 us in MXFP8 and 6.1 in MXFP4 for 1 token (2.5 TB/s), 9.0 and 7.6
// for 16, of which a launch and a first load are about 3.  16 waves a workgroup or 2 units ahead are equal.
// 17 to 32 tokens in MXFP8 with 8 waves spill 10 or 11 registers (the four units of two token groups).
constexpr int Q_UNIT = 256;
template <int FMT, int W, int MT, bool GATED, class Epilogue>
__global__ void __launch_bounds__(W * 64) stream_q_kernel(QOperands o, Epilogue epi, float* __restrict__ parts, int T,
                                                          int K, int rows) {
  constexpr int COLS = GATED ? SUB_ROWS / 2 : SUB_ROWS, D = 4, AP = FMT / 4;
  __shared__ f32x4 red[(W > 1) ? W * MT * 64 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * COLS;
  const size_t kb = (size_t)(K >> 1), ks = (size_t)(K >> 5), ka = (size_t)K * FMT / 8;
  // past the last row or token the last one again; what it gives is not stored
  const size_t row = GATED ? (size_t)min(n0 + (r & 7), rows - 1) + (r >= 8 ? (size_t)rows : 0) : (size_t)min(n0 + r, rows - 1);
  const uint8_t* wp = o.w + row * kb + 16 * g;
  const uint8_t* sp = o.ws + row * ks;
  const uint8_t* ap[MT];
  const uint8_t* asp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const size_t t = (size_t)min(m * 16 + r, T - 1);
    ap[m] = o.a + t * ka + 16 * g;
    asp[m] = o.as + t * ks;
  }
  typedef u32x2 scales_any __attribute__((aligned(1)));
  struct Unit {
    u32x4 w[2];
    QFragment<FMT> a[MT][2];
    u32x2 sw, sa[MT];
  };
  auto load = [&](Unit& u, int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) u.w[h] = ld_stream16(wp + (size_t)j * (Q_UNIT / 2) + h * 64);
    u.sw = *reinterpret_cast<const scales_any*>(sp + (size_t)j * (Q_UNIT / 32));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < AP; ++p) u.a[m][h].v[p] = ld16(ap[m] + (size_t)j * (Q_UNIT * FMT / 8) + (h * AP + p) * 64);
      u.sa[m] = *reinterpret_cast<const scales_any*>(asp[m] + (size_t)j * (Q_UNIT / 32));
    }
  };
  f32x4 acc[MT][1];
  acc_zero(acc);
  auto multiply = [&](const Unit& u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[m][0] = mfma_stream_q<FMT>(u.w[h], u.a[m][h], acc[m][0], (int)(u.sw[h] >> (8 * g)), (int)(u.sa[m][h] >> (8 * g)));
  };
  const int units = K / Q_UNIT;
  const int u0 = (int)((int64_t)units * wave / W), u1 = (int)((int64_t)units * (wave + 1) / W);
  Unit q[D];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (u0 + d < u1) load(q[d], u0 + d);
  for (int j = u0; j < u1; j += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (j + d < u1) {
        multiply(q[d]);
        if (j + d + D < u1) load(q[d], j + d + D);
      }
    }
  }
  // What is left of K, fewer than 8 blocks: missing ones are zero codes with zero scales.
  const int left = (K % Q_UNIT) >> 5;
  if (left > 0 && wave == W - 1) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    Unit u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int have = left - 4 * h, b = 8 * units + 4 * h + g;  // this lane's block
      u.w[h] = g < have ? ld16(wp + (size_t)units * (Q_UNIT / 2) + h * 64) : zero;
      u.sw[h] = g < have ? (uint32_t)sp[b] << (8 * g) : 0u;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int p = 0; p < AP; ++p) {
          const int piece = FMT == 8 ? 2 * p + (g >> 1) : g;  // its block of the four
          u.a[m][h].v[p] = piece < have ? ld16(ap[m] + (size_t)units * (Q_UNIT * FMT / 8) + (h * AP + p) * 64) : zero;
        }
        u.sa[m][h] = g < have ? (uint32_t)asp[m][b] << (8 * g) : 0u;
      }
    }
    multiply(u);
  }
  wg_reduce<1, MT, W>(acc, red, wave, lane);
  if (wave != 0) return;
  const int n = n0 + 4 * (GATED ? g & 1 : g);
  const int pc = part_cols(rows);
  const auto cols = epi.template columns<4>(n);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = m * 16 + r;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = acc[m][0][j];
    if (parts) {  // n + 4 <= pc
      if (t < T && n < rows)
        *reinterpret_cast<f32x4*>(parts + (size_t)t * ((GATED ? 2 : 1) * (size_t)pc) + (GATED && g >= 2 ? pc : 0) + n) = acc[m][0];
      continue;
    }
    if constexpr (GATED) {
      float u[4];  // rows 8 and up of the tile: the lanes 32 on
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __shfl_xor(v[j], 32, 64);
      if constexpr (!Epilogue::WHOLE_BLOCKS)
        if (t < T && g < 2) epi.template store<4>(t, n, v, u, cols);
    } else {
      if (t < T) epi.template store<4>(t, n, v, cols, epi.template fetch<4>(t, n));
    }
  }
}

// ------------------------------------------------------------------ tiles

// In a step, half a stage, a wave reads the next step's operands between its products (in the first half of
// them) and issues half of a later stage's copies.  The one barrier of a stage lies between its two steps: the
// second one's operands are in registers then, so the stage's buffer is free for the one D stages on.
//
// 256 x 256 (4096 x 7168 x 4096 with gelu, bias and residual 73 to 74 us in MXFP4; gate_up, H 7168, I 2048,
// 4096 tokens, from and to MXFP8 86 to 91): each of 8 waves has 64 x 128, two waves a SIMD, so that one's products run
// beside the other's reads (4 waves of 128 x 128: 86 for 80 at the time).  What bounds it: the products alone take
// 32 us (MXFP4) and 55 (MXFP8), at the 7.0 and 3.4 PFLOP/s that they reach on random data here; with reads, scales
// and barriers 44 and 64; with the copies 55 and 81; the epilogue of the one round of tiles is 8 to 19 more.  The
// copies bring 1.8 and 2.8 MB to each CU, 24 and 42 us at what a CU reads with nothing else to do.
// MFMA busy 61% of the cycles at 2.0 GHz in MXFP8; LDS conflicts 1 cycle in 10.  Equal or slower: waves of 128 x 64,
// lines requested into L2 6 to 12 stages ahead (80 for 77), other places for the reads among the products, wave
// priorities.
//
// KB: whole lines of either operand in MXFP4 (4096 tokens 75 us for 80, 2048 44 for 51), but not in tiles of few
// waves, which wait for the larger stage (300 tokens 7168 -> 4096 20.5 for 17.7).  MXFP8 has no LDS for it.
// D, stages in the LDS: all that it holds for 256 x 256, half of that where two workgroups share a CU, and where
// one is alone 4 or 3 stages: more only lets the first stage wait behind the others (128 tokens
// 7168 -> 4096 in MXFP8 with 768 values 14.5 us, 512 13.9, 384 14.2; 2048 -> 7168, 300 tokens, 12.1, 11.5 and 11.9).
template <int FMT, int KB, int MT, int NT, int WM, int WN, int D, bool GATED, class Epilogue>
__global__ void __launch_bounds__(64 * WM * WN, (QLds<FMT, KB, MT, NT, WM, WN, D>::PER_SIMD))
    tile_q_kernel(QOperands o, Epilogue epi, float* __restrict__ parts, int T, int K, int rows, int mtiles, int ntiles,
                  int nsplit) {
  typedef QLds<FMT, KB, MT, NT, WM, WN, D> L;
  constexpr int WCOLS = NT * 32 / (GATED ? 2 : 1), HALF = GATED ? NT / 2 : NT, COLS = WN * WCOLS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[L::BYTES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int tile = xcd_tile(blockIdx.x, mtiles * ntiles * nsplit);
  // Four rows of tiles together, column by column: the 32 tiles that an XCD has at once then read fewer
  // rows of both operands than two whole rows of 16 would.
  const int split = tile % nsplit, id = tile / nsplit, band = id / (4 * ntiles), high = min(4, mtiles - 4 * band);
  const int mt0 = 4 * band + (id - 4 * band * ntiles) % high, nt = (id - 4 * band * ntiles) / high;
  const int m0 = mt0 * L::BM, n0 = nt * COLS;
  constexpr int STEPS = L::STEPS, GROUP = L::GROUP;
  const int stages = (K + KB - 1) / KB, full = K / KB, tail = K % KB >> 5;
  // K is split at whole groups of scales
  const int groups = (K + Q_KG - 1) / Q_KG;
  const int g0 = (int)((int64_t)groups * split / nsplit), g1 = (int)((int64_t)groups * (split + 1) / nsplit);
  const int st0 = g0 * GROUP, st1 = min(g1 * GROUP, stages);

  // Row lr of the workgroup's weight rows: row r of MFMA tile lr >> 5, counted from the tile's first row in the
  // gate or the up half; past the last row (or token) the last one again, never stored.
  auto weight_half = [&](int lr) { return (size_t)n0 + ((lr >> 5) % NT >= HALF ? (size_t)rows : 0); };
  auto weight_row = [&](int lr) { return min((lr >> 5) / NT * WCOLS + (lr >> 5) % HALF * 32 + (lr & 31), rows - 1 - n0); };
  auto token_row = [&](int lr) { return min(lr, T - 1 - m0); };
  typename L::Rows as;
  as.init((int64_t)K * FMT / 8, min(L::BM, T - m0), wave, lane,
          [&](int) { return o.a + (size_t)m0 * ((size_t)K * FMT / 8); }, token_row);
  typename L::Codes cs;
  cs.init(K >> 1, min(COLS, rows - n0), wave, lane, [&](int lr) { return o.w + weight_half(lr) * (size_t)(K >> 1); }, weight_row);
  QScales<L::BM, L::BN, 64 * WM * WN> sc;
  const size_t ks = (size_t)(K >> 5);
  sc.init(K, K % Q_KG == 0, [&](int lr) {
    return lr < L::BM ? o.as + (size_t)(m0 + token_row(lr)) * ks
                      : o.ws + (weight_half(lr - L::BM) + weight_row(lr - L::BM)) * ks;
  });

  constexpr int XC = L::Rows::COPIES, LOADS = XC + L::Codes::COPIES, FIRST = LOADS / 2;
  auto copy = [&](uint8_t* buf, int st, auto Q) __attribute__((always_inline)) {
    constexpr int q = Q;
    if constexpr (q < XC)
      as.copy_one(buf, st, q);
    else
      cs.copy_one(buf + L::Rows::BYTES, st, q - XC);
  };
  // ahead of copies [FROM, FROM + N) of stage st, which is the last to come where it is partial
  auto prepare = [&](int st, auto FROM, auto N) __attribute__((always_inline)) {
    if (st != full) return;
    unrolled<decltype(N)::value>([&](auto Q) __attribute__((always_inline)) {
      constexpr int q = FROM + Q;
      if constexpr (q < XC)
        as.only(tail * (FMT / 4), q);
      else
        cs.only(tail, q - XC);
    });
  };
  typedef std::integral_constant<int, 0> FromFirst;
  typedef std::integral_constant<int, FIRST> FirstOnes;
  typedef std::integral_constant<int, LOADS - FIRST> OtherOnes;
  typedef std::integral_constant<int, LOADS> AllOnes;
  const int r = lane & 31, g = lane >> 5;
  constexpr int AF = FMT / 4;  // 16-byte pieces of a fragment
  uint32_t at[STEPS][AF], wat[STEPS];
#pragma unroll
  for (int u = 0; u < STEPS; ++u) {
#pragma unroll
    for (int p = 0; p < AF; ++p) {
      const int c = FMT == 8 ? 4 * u + 2 * p + g : 2 * u + g;
      at[u][p] = (uint32_t)(wm * MT * 32 + r) * L::ARB + ((c ^ q_key<L::ARB>(r)) << 4);
    }
    wat[u] = L::Rows::BYTES + (uint32_t)(wn * NT * 32 + r) * L::WRB + (((2 * u + g) ^ q_key<L::WRB>(r)) << 4);
  }
  const uint32_t sat = L::SCALES_AT + (uint32_t)(wm * MT * 32 + r) * 16;
  const uint32_t wsat = L::SCALES_AT + (uint32_t)(L::BM + wn * NT * 32 + r) * 16;
  auto scales_of = [&](int group) { return lds + L::SCALES_AT + (group & 1) * L::SCALES; };

  f32x16 acc[MT][NT];
  tile_zero(acc);
  QFragment<FMT> frag[2][MT];
  u32x4 w[2][NT];
  // A group's scales, a dword for two steps; shifted right by 8 g ahead of them, so that byte 0 is this
  // lane's in the first and byte 2 in the second.
  uint32_t sa[MT][4], sw[NT][4];
  auto scale_at = [&](int group, int e) {
    return lds + (group & 1) * L::SCALES + (e < MT ? sat + e * 512 : wsat + (e - MT) * 512);
  };
  auto read_scales = [&](int group, int e) {  // of all steps but the last two
    typedef unsigned u32x3 __attribute__((ext_vector_type(3), aligned(16)));
    const u32x3 v = *reinterpret_cast<const u32x3*>(scale_at(group, e));
#pragma unroll
    for (int j = 0; j < 3; ++j) (e < MT ? sa[e][j] : sw[e - MT][j]) = v[j];
  };
  auto read_last_scale = [&](int group, int e) {  // whose register the products still read meanwhile
    (e < MT ? sa[e][3] : sw[e - MT][3]) = *reinterpret_cast<const uint32_t*>(scale_at(group, e) + 12);
  };
  auto shift_scale = [&](int pair, int e) {
    uint32_t& s = e < MT ? sa[e][pair] : sw[e - MT][pair];
    s >>= 8 * g;
  };
  auto read = [&](const uint8_t* buf, int u, int e) {  // piece e of a step's operands
    if (e < NT)
      w[u & 1][e] = ld16(buf + wat[u] + e * (32 * L::WRB));
    else
      frag[u & 1][(e - NT) / AF].v[(e - NT) % AF] = ld16(buf + at[u][(e - NT) % AF] + (e - NT) / AF * (32 * L::ARB));
  };
  constexpr int SLOTS = MT * NT, READS = NT + MT * AF, SCALES = MT + NT;
  auto buffer_of = [&](int i) { return lds + i * L::ONE; };

  sc.load(g0, scales_of(g0));
  sc.store(scales_of(g0));
  unrolled<D - 1>([&](auto J) __attribute__((always_inline)) {
    const int st = min(st0 + J, st1 - 1);
    prepare(st, FromFirst{}, AllOnes{});
    unrolled<LOADS>([&](auto Q) __attribute__((always_inline)) { copy(buffer_of(J), st, Q); });
  });
  prepare(min(st0 + D - 1, st1 - 1), FromFirst{}, FirstOnes{});
  unrolled<FIRST>([&](auto Q) __attribute__((always_inline)) { copy(buffer_of(D - 1), min(st0 + D - 1, st1 - 1), Q); });
  q_barrier<(D - 2) * LOADS + FIRST>();
#pragma unroll
  for (int e = 0; e < SCALES; ++e) read_scales(g0, e);
#pragma unroll
  for (int e = 0; e < READS; ++e) read(lds, 0, e);
#pragma unroll
  for (int e = 0; e < SCALES; ++e) shift_scale(0, e);
  scales_ready(sa, 0);
  scales_ready(sw, 0);
  settle_mfma(acc);  // the accumulators have been cleared

  int cur = 0, fill = D - 1;  // buffers of the current stage, and of the one D - 1 stages on
  for (int group = g0; group < g1; ++group) {
    const bool more = group + 1 < g1;
    unrolled<GROUP>([&](auto G) __attribute__((always_inline)) {
      constexpr int stage = G;
      const int st = group * GROUP + stage;
      if (st >= st1) return;
      if (stage == 0 && more) sc.load(group + 1, scales_of(group + 1));
      const int nxt = cur + 1 == D ? 0 : cur + 1;
      const int c0 = min(st + D - 1, st1 - 1), c1 = min(st + D, st1 - 1);
      unrolled<STEPS>([&](auto U) __attribute__((always_inline)) {
        constexpr int u = U, pair = (stage * STEPS + u) / 2;
        constexpr bool last_step = u == STEPS - 1;
        if constexpr (u == 0) prepare(c0, FirstOnes{}, OtherOnes{});
        if constexpr (last_step) {
          if (stage == GROUP - 1 && more) sc.store(scales_of(group + 1));
          // the next stage has landed for every wave (and, at a group's end, the next one's scales, which
          // the copies of nearly a group follow), and no wave reads the current one any more
          constexpr int LATER = (D - 2) * LOADS, SINCE = GROUP * LOADS - FIRST;
          q_barrier<(stage == GROUP - 1 && SINCE < LATER ? SINCE : LATER)>();
          prepare(c1, FromFirst{}, FirstOnes{});
        }
        unrolled<SLOTS>([&](auto S) __attribute__((always_inline)) {
          constexpr int k = S, m = k / NT, i = k % NT;
          mfma_q<(u & 1)>(acc[m][i], w[u & 1][i], frag[u & 1][m], sw[i][pair], sa[m][pair]);
          // the next step's operands, in the first half
          constexpr bool first_three = last_step && stage == GROUP - 1, last = u == 0 && stage == 0;
          constexpr int RS = first_three || last ? SCALES : 0, HALF_SLOTS = (SLOTS + 1) / 2;
          unrolled<RS + READS>([&](auto E) __attribute__((always_inline)) {
            if constexpr (E * HALF_SLOTS / (RS + READS) == k) {
              if constexpr (E < READS)
                read(buffer_of(last_step ? nxt : cur), (u + 1) % STEPS, E);
              else if constexpr (first_three)
                read_scales(group + 1, E - READS);
              else
                read_last_scale(group, E - READS);
            }
          });
          if constexpr ((u & 1) && k == SLOTS - 1)
            unrolled<SCALES>([&](auto E) __attribute__((always_inline)) { shift_scale((pair + 1) % 4, E); });
          unrolled<LOADS>([&](auto E) __attribute__((always_inline)) {
            if constexpr (last_step && E < FIRST && E * SLOTS / FIRST == k) copy(buffer_of(cur), c1, E);
            if constexpr (u == 0 && E >= FIRST && (E - FIRST) * SLOTS / (LOADS - FIRST) == k) copy(buffer_of(fill), c0, E);
          });
          keep_order();
        });
        if constexpr (u & 1) {
          scales_ready(sa, (pair + 1) % 4);
          scales_ready(sw, (pair + 1) % 4);
        }
      });
      fill = cur;
      cur = nxt;
    });
  }
  settle_mfma(acc);
  wait_copies();  // the repeated copies of the last stages: the LDS is used again
  tile_output<MT, NT, WM, WN, GATED, L::BYTES, (WM * WN > 4 ? 1 : 0)>(acc, epi, parts, lds, T, rows, m0, n0, split, nsplit, wave, lane);
}

// ------------------------------------------------------------------ up to 64 tokens: thin tiles

// A workgroup takes 32 NT weight rows (gate_up: half of them gate rows, half the up rows of the same
// columns) and all tokens; a wave 32 tokens and one of KS parts of K.  A wave copies what it needs into a ring
// of its own in the LDS, no barriers in the loop; the parts' sums meet in the LDS.
// Bound by what a CU reads (50 kB a microsecond): 7168 -> 4096, 32 tokens, 128 workgroups with 0.34 MB each, takes
// 10.5 us in MXFP8, 10.2 in MXFP4; 2048 -> 7168, 64 tokens, 6.8 and 6.5.  gate_up whose output is quantized needs 64
// rows a workgroup, a block of 32 columns: H 7168, I 2048, 24 tokens 13 us on 64 CUs.  (Parts of K over more CUs and
// a second launch to sum them should save some 2 of these in a graph, by what quantized_plan counts, and cost
// other callers a launch and a workspace, some 4.)
constexpr int THIN_Q_MAX_T = 64;
constexpr int Q_KB = 128;  // values of a stage
template <int FMT, int NT>
struct ThinQStage {
  static constexpr int ARB = Q_KB * FMT / 8, A = 32 * ARB, CODES = 32 * NT * (Q_KB / 2);
  static constexpr int SCALES_A = A + CODES, SCALES_W = SCALES_A + 256, BYTES = SCALES_W + 256;
  static constexpr int D = 163840 / 8 / BYTES < 4 ? 163840 / 8 / BYTES : 4;  // stages in the ring of each of 8 waves
  static constexpr int LOADS = A / 1024 + CODES / 1024 + 2;
  static_assert(D >= 2 && D * BYTES >= NT * 4096 && (D - 1) * LOADS < 64, "a ring, also of a wave's sums");
};

template <int FMT, int NT, bool GATED, int KS, class Epilogue>
__global__ void __launch_bounds__(512, 2) thin_q_kernel(QOperands o, Epilogue epi, int T, int K, int rows) {
  typedef ThinQStage<FMT, NT> L;
  constexpr int COLS = GATED ? 16 * NT : 32 * NT, D = L::D;
  __shared__ __attribute__((aligned(16))) uint8_t lds[8 * D * L::BYTES];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n0 = blockIdx.x * COLS, m0 = wave / KS * 32;
  const int stages = K / Q_KB, st0 = stages * (wave % KS) / KS, st1 = stages * (wave % KS + 1) / KS;
  uint8_t* ring = lds + wave * (D * L::BYTES);

  // Tokens and rows past the last: the last one again.
  const int ka = K * FMT / 8;
  constexpr int AC = L::ARB / 16, APER = 64 / AC, ACOPIES = 32 / APER, WCOPIES = 2 * NT;
  const buffer abuf = make_buffer(o.a + (size_t)m0 * ka, (uint64_t)min(32, T - m0) * (uint64_t)ka);
  const buffer asbuf = make_buffer(o.as + (size_t)m0 * (K >> 5), (uint64_t)min(32, T - m0) * (uint64_t)(K >> 5));
  uint32_t aoff[ACOPIES];
#pragma unroll
  for (int q = 0; q < ACOPIES; ++q) {
    const int r = q * APER + lane / AC;
    aoff[q] = (uint32_t)min(r, T - 1 - m0) * (uint32_t)ka + (((lane % AC) ^ q_key<L::ARB>(r)) << 4);
  }
  const uint32_t asoff = (uint32_t)min(lane & 31, T - 1 - m0) * (uint32_t)(K >> 5);
  // Row lr of the 32 NT: weight row n0 + lr, or column n0 + lr % COLS of half lr / COLS.
  auto half_of = [&](int lr) { return (size_t)n0 + (GATED && lr >= COLS ? (size_t)rows : 0); };
  auto row_of = [&](int lr) { return min(lr % COLS, rows - 1 - n0); };
  const int have = min(COLS, rows - n0);
  buffer wbuf[WCOPIES];
  uint32_t woff[WCOPIES];
#pragma unroll
  for (int q = 0; q < WCOPIES; ++q) {
    const int r = q * 16 + (lane >> 2);
    wbuf[q] = make_buffer(o.w + half_of(q * 16) * (size_t)(K >> 1), (uint64_t)have * (uint64_t)(K >> 1));
    woff[q] = (uint32_t)row_of(r) * (uint32_t)(K >> 1) + (((lane & 3) ^ q_key<64>(r)) << 4);
  }
  const uint8_t* wscale = o.ws + (half_of(lane & (32 * NT - 1)) + row_of(lane & (32 * NT - 1))) * (size_t)(K >> 5);
  auto load = [&](int st, uint8_t* buf) {
#pragma unroll
    for (int q = 0; q < ACOPIES; ++q) copy16_to_lds(abuf, aoff[q], (uint32_t)st * L::ARB, buf + q * 1024);
#pragma unroll
    for (int q = 0; q < WCOPIES; ++q) copy16_to_lds(wbuf[q], woff[q], (uint32_t)st * 64, buf + L::A + q * 1024);
    copy4_to_lds(asbuf, asoff, (uint32_t)st * 4, buf + L::SCALES_A);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wscale + st * 4),
                                     (lds_ptr)(buf + L::SCALES_W), 4, 0, 0);
  };
  const int r = lane & 31, g = lane >> 5;
  f32x16 acc[NT] = {};
  int at = 0;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (st0 + d < st1) load(st0 + d, ring + d * L::BYTES);
  for (int st = st0; st < st1; ++st) {
    // this stage has landed; up to D - 1 later ones are under way
    const int later = st1 - 1 - st;
    if (later >= D - 1)
      wait_copies<(D - 1) * L::LOADS>();
    else if (D > 2 && later == D - 2)
      wait_copies<(D - 2) * L::LOADS>();
    else if (D > 3 && later == D - 3)
      wait_copies<(D - 3) * L::LOADS>();
    else
      wait_copies();
    uint8_t* buf = ring + at * L::BYTES;
    QFragment<FMT> a[2];
    u32x4 w[2][NT];
    uint32_t sw[NT];
    const uint32_t sa = *reinterpret_cast<const uint32_t*>(buf + L::SCALES_A + r * 4) >> (8 * g);
#pragma unroll
    for (int i = 0; i < NT; ++i) sw[i] = *reinterpret_cast<const uint32_t*>(buf + L::SCALES_W + (i * 32 + r) * 4) >> (8 * g);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int p = 0; p < FMT / 4; ++p) {
        const int c = FMT == 8 ? 4 * u + 2 * p + g : 2 * u + g;
        a[u].v[p] = ld16(buf + r * L::ARB + ((c ^ q_key<L::ARB>(r)) << 4));
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) w[u][i] = ld16(buf + L::A + (i * 32 + r) * 64 + (((2 * u + g) ^ q_key<64>(r)) << 4));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the buffer may be filled again
    if (st + D < st1) load(st + D, buf);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const i32x8 w0 = {(int)w[0][i][0], (int)w[0][i][1], (int)w[0][i][2], (int)w[0][i][3], 0, 0, 0, 0};
      const i32x8 w1 = {(int)w[1][i][0], (int)w[1][i][1], (int)w[1][i][2], (int)w[1][i][3], 0, 0, 0, 0};
      acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w0, q_operand(a[0]), acc[i], 4, FMT == 8 ? 0 : 4, 0, (int)sw[i], 0, (int)sa);
      acc[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w1, q_operand(a[1]), acc[i], 4, FMT == 8 ? 0 : 4, 2, (int)sw[i], 2, (int)sa);
    }
    at = at + 1 == D ? 0 : at + 1;
  }
  wait_copies();
  tile_to_lds<NT>(ring, acc, lane);
  // each of the KS waves sums its share of the rows
  constexpr int PIECES = COLS / 8, ROWS = 64 / PIECES, SHARE = 32 / KS, ITERS = (SHARE + ROWS - 1) / ROWS;
  const int p = lane % PIECES, n = n0 + p * 8;
  const auto cols = epi.template columns<8>(n);
  const uint8_t* first = lds + wave / KS * KS * (D * L::BYTES);
  __syncthreads();
#pragma unroll
  for (int it = 0; it < ITERS; ++it) {
    const int row = it * ROWS + lane / PIECES + wave % KS * SHARE, t = m0 + row;
    if (t >= T || n >= rows || (ROWS > SHARE && lane / PIECES >= SHARE)) continue;
    f32x4 q[GATED ? 4 : 2];
#pragma unroll
    for (int j = 0; j < (GATED ? 4 : 2); ++j) {
      const uint32_t from = out_at<NT>(row, 2 * p + (j & 1) + (j >> 1) * (4 * NT));
      q[j] = *reinterpret_cast<const f32x4*>(first + from);
#pragma unroll
      for (int k = 1; k < KS; ++k) q[j] += *reinterpret_cast<const f32x4*>(first + k * (D * L::BYTES) + from);
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

// Thin tiles copy a stage's scales as dwords: whole groups of them, whose rows are aligned.  From 33 tokens
// on they read the weights twice and a long reduction goes to tiles (64 tokens in MXFP8: 2048 -> 7168 6.8 us,
// with tiles 14.4; 7168 -> 4096 16.4 and 11.6).
static bool takes_thin_q(int64_t T, int64_t K) {
  return T > 16 && T <= (K <= 4096 ? THIN_Q_MAX_T : 32) && K % Q_KG == 0;
}
static bool takes_stream_q(int64_t T, int64_t K) { return T <= STREAM_Q_MAX_T && !takes_thin_q(T, K); }

// What a round of tiles takes, of 256 x 256 (one a CU) and of 128 x 128 (two a CU), in microseconds at a
// reduction of 7168: MXFP8 92 and 58, MXFP4 66 and 44 (4096 and 2048 tokens, 7168 -> 4096).  E.g. in MXFP8 2048
// tokens take 69 with the large tiles for 58 with the small ones, 4096 tokens 92 for 114.
constexpr int Q8_ROUND_256 = 92, Q8_ROUND_128 = 58, Q4_ROUND_256 = 66, Q4_ROUND_128 = 44;

// quantized: the product's output is, which a workgroup of the streaming kernel, with fewer columns
// than a block, leaves to a second launch.
TilePlan quantized_plan(int64_t T, int64_t K, int64_t rows, bool gated, bool quantized, int format) {
  TilePlan p{};
  p.nsplit = 1;
  if (takes_thin_q(T, K)) {
    // 64 rows a workgroup where an output block needs them, or 32 would give more workgroups than CUs
    const int64_t ones = (rows + (gated ? 15 : 31)) / (gated ? 16 : 32);
    p.thin = quantized || ones > GPU_CUS ? 2 : 1;
    p.ntiles = (int)((ones + p.thin - 1) / p.thin);
    return p;
  }
  bool parts = quantized;
  if (!takes_stream_q(T, K)) {
    const bool eight = format == MX_FORMAT_MXFP8;
    p.mt = T <= 64 ? 1 : tile_choice(T, rows * (gated ? 2 : 1), eight ? Q8_ROUND_256 : Q4_ROUND_256, eight ? Q8_ROUND_128 : Q4_ROUND_128);
    const int64_t bm = 64 * p.mt, all = rows * (gated ? 2 : 1), groups = (K + Q_KG - 1) / Q_KG;
    p.mtiles = (int)((T + bm - 1) / bm);
    p.nt = p.mt == 4 ? 4 : 2;
    auto tiles = [&](int64_t nt) { return (all + 64 * nt - 1) / (64 * nt) * p.mtiles; };
    if (p.mt < 4 && tiles(2) <= GPU_CUS) {
      // Fewer tiles than CUs: 128 or 64 weight rows a tile, K whole or in parts, by what a workgroup reads
      // (a CU's read path gives some 50 kB a microsecond of half lines, which all tiles are counted at, MXFP4's of
      // whole lines too; tiles of 64 tokens beyond 64 are not weighed) and what parts cost (written at 3 and read at
      // 4 MB a microsecond, 2.5 for the second launch).  7168 -> 4096 in MXFP8: 128 tokens 14.3 us with 64 rows in 4
      // parts, 19.3 with 128 rows in 8; 2048 -> 7168, 128 tokens: 10.7 with 64 rows whole, 19.4 with 128 in 4 (14.1 and
      // 9.6 since, with fewer stages ahead).
      double least = 0;
      for (int nt = 2; nt >= 1; --nt)
        for (int64_t split = 1; split <= groups && split * tiles(nt) <= GPU_CUS; ++split) {
          const double read = (double)K * (bm * (eight ? 1.0 : 0.5) + 32.0 * nt) / (double)split / 50e3;
          const double cost = read + (split > 1 ? 2.5 + 4.0 * (double)(split * T * all) * (1 / 3e6 + 1 / 4e6) : 0.0);
          if (least == 0 || cost < least) least = cost, p.nt = nt, p.nsplit = (int)split;
        }
    }
    p.ntiles = (int)(tiles(p.nt) / p.mtiles);
    parts = p.nsplit > 1;
  }
  if (parts) p.bytes = (size_t)p.nsplit * T * part_cols((int)rows) * (gated ? 2 : 1) * 4;
  return p;
}

template <int FMT, bool GATED, class Epilogue>
static int launch_product_q(const QOperands& o, const Epilogue& epi, bool quantized, void* workspace, int T, int K,
                            int rows, hipStream_t stream) {
  const TilePlan p = quantized_plan(T, K, rows, GATED, quantized, FMT == 8 ? MX_FORMAT_MXFP8 : MX_FORMAT_MXFP4);
  float* parts = p.bytes ? static_cast<float*>(workspace) : nullptr;
  if (p.thin) {
#define MX_THIN_Q(NT, KS) \
  hipLaunchKernelGGL((thin_q_kernel<FMT, NT, GATED, KS, Epilogue>), dim3(p.ntiles), dim3(512), 0, stream, o, epi, T, K, rows)
    if constexpr (!Epilogue::WHOLE_BLOCKS) {  // those have p.thin == 2
      if (p.thin == 1 && T <= 32)
        MX_THIN_Q(1, 8);
      else if (p.thin == 1)
        MX_THIN_Q(1, 4);
    }
    if (p.thin == 2 && T <= 32)
      MX_THIN_Q(2, 8);
    else if (p.thin == 2)
      MX_THIN_Q(2, 4);
#undef MX_THIN_Q
  } else if (takes_stream_q(T, K)) {
    const int cols = GATED ? SUB_ROWS / 2 : SUB_ROWS;
    const int items = (rows + cols - 1) / cols, units = K / Q_UNIT;
    int W = 1;
    while (W < 8 && 2 * W <= units && 2 * W * items <= 2048) W *= 2;
#define MX_STREAM_Q(WW, M) \
  hipLaunchKernelGGL((stream_q_kernel<FMT, WW, M, GATED, Epilogue>), dim3(items), dim3(WW * 64), 0, stream, o, epi, parts, T, K, rows)
#define MX_STREAM_Q_W(WW) \
  if (T <= 16)            \
    MX_STREAM_Q(WW, 1);   \
  else                    \
    MX_STREAM_Q(WW, 2)
    if (W == 1) {
      MX_STREAM_Q_W(1);
    } else if (W == 2) {
      MX_STREAM_Q_W(2);
    } else if (W == 4) {
      MX_STREAM_Q_W(4);
    } else {
      MX_STREAM_Q_W(8);
    }
#undef MX_STREAM_Q_W
#undef MX_STREAM_Q
  } else {
    const dim3 grid((unsigned)(p.mtiles * p.ntiles * p.nsplit));
#define MX_TILE_Q(KB, MT, NT, WM, WN, D)                                                                             \
  hipLaunchKernelGGL((tile_q_kernel<FMT, KB, MT, NT, WM, WN, D, GATED, Epilogue>), grid, dim3(64 * WM * WN), 0, stream, \
                     o, epi, p.nsplit > 1 ? parts : nullptr, T, K, rows, p.mtiles, p.ntiles, p.nsplit)
    const bool alone = (int64_t)p.mtiles * p.ntiles * p.nsplit <= GPU_CUS;  // a workgroup has its CU's LDS
    constexpr int LINE = FMT == 8 ? 128 : 256;  // values of a line of activations
    if (p.mt == 4)
      MX_TILE_Q(LINE, 2, 4, 4, 2, (FMT == 8 ? 3 : 2));
    else if (p.mt == 2 && p.nt == 1)
      MX_TILE_Q(128, 1, 2, 4, 1, 4);
    else if (p.mt == 2 && alone)
      MX_TILE_Q(LINE, 1, 2, 4, 2, (FMT == 8 ? 4 : 3));
    else if (p.mt == 2)
      MX_TILE_Q(LINE, 1, 2, 4, 2, (FMT == 8 ? 3 : 2));
    else if (p.nt == 1)
      MX_TILE_Q(128, 1, 2, 2, 1, 4);
    else
      MX_TILE_Q(128, 1, 2, 2, 2, 4);
#undef MX_TILE_Q
  }
  if (parts) {
    const int pc = part_cols(rows);
    const int64_t pieces = (int64_t)T * (pc / 8);
    hipLaunchKernelGGL((combine_kernel<GATED, Epilogue>), dim3((unsigned)((pieces + 63) / 64)), dim3(64), 0, stream, parts,
                       epi, T, pc, p.nsplit);
  }
  return hip_status(hipGetLastError());
}

int launch_linear_quantized(const uint8_t* a, const uint8_t* as, int format, const uint8_t* w, const uint8_t* s,
                            const uint16_t* bias, const uint16_t* residual, float scale, int act, uint16_t* y,
                            uint16_t* z, int T, int K, int N, void* workspace, hipStream_t stream) {
  const QOperands o{a, as, w, s};
  const LinearEpilogue epi{bias, residual, y, z, N, act, scale};
  return format == MX_FORMAT_MXFP8 ? launch_product_q<8, false>(o, epi, false, workspace, T, K, N, stream)
                                   : launch_product_q<4, false>(o, epi, false, workspace, T, K, N, stream);
}

template <int FMT>
static int gate_up_q(const QOperands& o, const GatedEpilogue& epi, int out_format, uint8_t* codes, uint8_t* scales,
                     void* workspace, int T, int H, int I, hipStream_t stream) {
  if (!codes) return launch_product_q<FMT, true>(o, epi, false, workspace, T, H, I, stream);
  if (out_format == MX_FORMAT_MXFP8)
    return launch_product_q<FMT, true>(o, GatedQuantEpilogue<8>{epi, codes, scales}, true, workspace, T, H, I, stream);
  return launch_product_q<FMT, true>(o, GatedQuantEpilogue<4>{epi, codes, scales}, true, workspace, T, H, I, stream);
}

int launch_gate_up_quantized(const uint8_t* a, const uint8_t* as, int format, const uint8_t* w, const uint8_t* s,
                             const uint16_t* bias, int act, uint16_t* h, int out_format, uint8_t* h_codes,
                             uint8_t* h_scales, uint16_t* z, int T, int H, int I, void* workspace, hipStream_t stream) {
  const QOperands o{a, as, w, s};
  const GatedEpilogue epi{bias, h, z, I, act};
  return format == MX_FORMAT_MXFP8 ? gate_up_q<8>(o, epi, out_format, h_codes, h_scales, workspace, T, H, I, stream)
                                   : gate_up_q<4>(o, epi, out_format, h_codes, h_scales, workspace, T, H, I, stream);
}

}  // namespace mx
