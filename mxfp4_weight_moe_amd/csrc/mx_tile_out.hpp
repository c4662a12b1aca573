// What tiled products do with their sums: from the accumulators through the LDS, by rows, into the
// epilogue or into the fp32 parts of a split reduction; and the launch that sums those parts.
#pragma once
#include "mx_epilogue.hpp"
#include "mx_tile.hpp"

namespace mx {

// Columns per row of the fp32 parts of a split K (each half of gate_up, or all rows of a
// linear layer), rounded up so that a lane's 8 consecutive values always fit.
__host__ __device__ static inline int part_cols(int rows) { return (rows + 7) / 8 * 8; }

// The end of a tiled product of WM x WN waves: wave (wm, wn) holds MT x NT MFMA tiles, 32 tokens
// by 32 weight rows each; for gate_up the first half of them gate rows, the second half the up rows
// of the same columns.  m0, n0: the workgroup's first token and output column.  nsplit > 1: part
// `split` of the reduction goes to parts[split] as fp32 [T][part columns (x 2)].  LDS_BYTES of `lds`
// are free once every wave is here.  ROWS_AT_ONCE: rows of MFMA tiles through the LDS at a time (0: two,
// or the one there is).
template <int MT, int NT, int WM, int WN, bool GATED, int LDS_BYTES, int ROWS_AT_ONCE = 0, class Epilogue>
__device__ __forceinline__ void tile_output(const f32x16 (&acc)[MT][NT], const Epilogue& epi, float* __restrict__ parts,
                                            uint8_t* lds, int T, int rows, int m0, int n0, int split, int nsplit,
                                            int wave, int lane) {
  constexpr int WCOLS = NT * 32 / (GATED ? 2 : 1);
  const int wm = wave / WN, wn = wave % WN;
  const int pc = part_cols(rows);
  // MB rows of MFMA tiles at a time through the LDS; then row by row, PIECES lanes a row with 8
  // columns each, so a lane has the same columns in all its rows.  U rows of a lane go
  // together, and what the next ones read (the residual) is fetched meanwhile.
  constexpr int MB = ROWS_AT_ONCE ? ROWS_AT_ONCE : MT < 2 ? 1 : 2;
  static_assert(WM * WN * MB * NT * 4096 <= LDS_BYTES, "results of all waves in the stages' LDS");
  uint8_t* mine = lds + wave * (MB * NT * 4096);
  constexpr int PIECES = WCOLS / 8, ROWS = 64 / PIECES, ITERS = MB * 32 / ROWS, U = ITERS < 4 ? ITERS : 4;
  const int p = lane % PIECES, n = n0 + wn * WCOLS + p * 8;
  const int t0 = m0 + wm * MT * 32 + lane / PIECES;
  const auto cols = epi.template columns<8>(n);
  struct Ahead {
    Piece<8> r[U];
  };
  auto fetch = [&](int it) {  // row t0 + it * ROWS and the U - 1 after it
    Ahead f{};
    if constexpr (!GATED) {
      if (nsplit == 1)
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int t = t0 + (it + k) * ROWS;
          if (t < T) f.r[k] = epi.template fetch<8>(t, n);
        }
    }
    return f;
  };
  Ahead next = fetch(0);
  __syncthreads();  // every wave has read its last fragments
#pragma unroll
  for (int b = 0; b < MT / MB; ++b) {
#pragma unroll
    for (int m = 0; m < MB; ++m) tile_to_lds<NT>(mine + m * NT * 4096, acc[b * MB + m], lane);
#pragma unroll 1
    for (int it = 0; it < ITERS; it += U) {
      const Ahead now = next;
      if (b * ITERS + it + U < MT / MB * ITERS) next = fetch(b * ITERS + it + U);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int row = (it + k) * ROWS + lane / PIECES;
        const int t = t0 + (b * ITERS + it + k) * ROWS;
        if (t >= T || n >= rows) continue;
        f32x4 q[GATED ? 4 : 2];
        q[0] = *reinterpret_cast<const f32x4*>(mine + out_at<NT>(row, 2 * p));
        q[1] = *reinterpret_cast<const f32x4*>(mine + out_at<NT>(row, 2 * p + 1));
        if constexpr (GATED) {
          q[2] = *reinterpret_cast<const f32x4*>(mine + out_at<NT>(row, 4 * NT + 2 * p));
          q[3] = *reinterpret_cast<const f32x4*>(mine + out_at<NT>(row, 4 * NT + 2 * p + 1));
        }
        if (nsplit > 1) {
          f32x4* o = reinterpret_cast<f32x4*>(parts + ((size_t)split * T + t) * ((GATED ? 2 : 1) * (size_t)pc) + n);
          o[0] = q[0];
          o[1] = q[1];
          if constexpr (GATED) {
            o = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(o) + pc);
            o[0] = q[2];
            o[1] = q[3];
          }
        } else {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = q[j >> 2][j & 3];
          if constexpr (GATED) {
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = q[2 + (j >> 2)][j & 3];
            epi.template store<8>(t, n, v, u, cols);
          } else {
            epi.template store<8>(t, n, v, cols, now.r[k]);
          }
        }
      }
    }
  }
}

// Sums the parts of a split K in ascending order and applies the epilogue: 8 columns a thread.
template <bool GATED, class Epilogue>
__global__ void __launch_bounds__(64) combine_kernel(const float* __restrict__ parts,
                                                      Epilogue epi, int T, int pc, int nsplit) {
  const int per_row = pc / 8;
  const int64_t id = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (id >= (int64_t)T * per_row) return;
  const int t = (int)(id / per_row), n = (int)(id % per_row) * 8;
  const size_t ld = GATED ? 2 * (size_t)pc : (size_t)pc;
  const float* p = parts + (size_t)t * ld + n;
  const size_t step = (size_t)T * ld;
  f32x4 a[2] = {}, b[2] = {};
  for (int z0 = 0; z0 < nsplit; z0 += 4) {  // four parts' loads at a time
    f32x4 q[4][GATED ? 4 : 2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* r = p + min(z0 + k, nsplit - 1) * step;
      q[k][0] = *reinterpret_cast<const f32x4*>(r);
      q[k][1] = *reinterpret_cast<const f32x4*>(r + 4);
      if constexpr (GATED) {
        q[k][2] = *reinterpret_cast<const f32x4*>(r + pc);
        q[k][3] = *reinterpret_cast<const f32x4*>(r + pc + 4);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (z0 + k >= nsplit) break;
      a[0] += q[k][0];
      a[1] += q[k][1];
      if constexpr (GATED) {
        b[0] += q[k][2];
        b[1] += q[k][3];
      }
    }
  }
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = a[j >> 2][j & 3], u[j] = b[j >> 2][j & 3];
  const auto cols = epi.template columns<8>(n);
  if constexpr (GATED)
    epi.template store<8>(t, n, v, u, cols);
  else
    epi.template store<8>(t, n, v, cols, epi.template fetch<8>(t, n));
}

}  // namespace mx
