// Tiled products of bf16 rows with MXFP4 weights for more tokens than one weight-streaming
// pass covers: the shared pieces of the forward (x W^T) and the backward (dz W) kernels.
//
// A workgroup of WM x WN waves owns a tile of WM*MT*16 tokens by WN*64 weight rows (forward)
// or columns (backward).  Each wave holds MT x 4 MFMA tiles (16x16x32 bf16) in registers.
// The activation tile goes from global memory to LDS without passing through registers
// (global_load_lds, 16 bytes a lane) into the buffer that the waves are not reading, one
// barrier a stage.  The weights stay 4-bit until they are in the registers of the wave that
// multiplies with them: a wave decodes 4 fragments (16 conversions) for 4*MT matrix
// instructions, so decoding costs a quarter of the issue slots at MT = 4 and an eighth at 8.
#pragma once
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace mx {

typedef __attribute__((address_space(1))) const void* global_cptr;
typedef __attribute__((address_space(3))) void* lds_ptr;

// 16 bytes a lane from global memory to LDS: lane l's bytes land at `lds` + 16 * l.
__device__ __forceinline__ void copy16_to_lds(const void* g, void* lds) {
  __builtin_amdgcn_global_load_lds((global_cptr)g, (lds_ptr)lds, 16, 0, 0);
}

// This wave's copies to LDS have landed (they count as vector memory operations, which a
// barrier alone does not wait for).
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Consecutive tiles go to one XCD (workgroups are dealt to the 8 XCDs in turn), so that the
// tiles that share activation rows share an L2.
constexpr int XCDS = 8;
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int x = b % XCDS, i = b / XCDS, q = total / XCDS, r = total % XCDS;
  return x * q + min(x, r) + i;
}

// ------------------------------------------------------------------ activation stages

// A stage is KB reduction values of BM rows: rows of KB * 2 bytes in 16-byte chunks, chunk c
// of row r stored at chunk position c ^ (r & (C - 1) & 15), so that 16 rows' reads of one
// logical chunk spread over all banks.  The copy to LDS writes 1 KB a wave at consecutive
// addresses; the permutation is in which chunk of its row each lane fetches.
template <int BM, int KB, int NW>
struct RowStage {
  static constexpr int C = KB / 8;                 // chunks per row
  static constexpr int BYTES = BM * KB * 2;
  static constexpr int ROWS_PER_COPY = 64 / C;     // rows of one wave-wide copy
  static constexpr int COPIES = BM / ROWS_PER_COPY / NW;  // wave-wide copies per wave
  static_assert(BM % (ROWS_PER_COPY * NW) == 0, "whole copies");

  uint32_t off[COPIES];  // byte offset of this lane's chunk from the tile's first row, stage 0
  const uint8_t* base;
  int wave, lane;

  // Rows past `rows` fetch the last row again; their results are never stored.
  __device__ __forceinline__ void init(const uint16_t* x, int m0, int rows, int64_t ld, int wave_, int lane_) {
    wave = wave_, lane = lane_;
    base = reinterpret_cast<const uint8_t*>(x + (size_t)m0 * ld);
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const int r = (q * NW + wave) * ROWS_PER_COPY + lane / C;
      const int c = (lane % C) ^ (r & (C - 1));
      off[q] = (uint32_t)min(r, rows - 1 - m0) * (uint32_t)(ld * 2) + c * 16;
    }
  }
  __device__ __forceinline__ void copy(uint8_t* buf, int stage) const {
    const uint8_t* p = base + (size_t)stage * (KB * 2);
#pragma unroll
    for (int q = 0; q < COPIES; ++q) copy16_to_lds(p + off[q], buf + (q * NW + wave) * 1024);
  }
  // The last, partial stage: `valid` (< KB, a multiple of 8) values of each row, zeros beyond.
  __device__ __forceinline__ void copy_tail(uint8_t* buf, int stage, int valid) const {
    const uint8_t* p = base + (size_t)stage * (KB * 2);
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const int r = (q * NW + wave) * ROWS_PER_COPY + lane / C;
      const int c = (lane % C) ^ (r & (C - 1));
      const u32x4 v = c * 8 < valid ? ld16(p + off[q]) : u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(buf + (q * NW + wave) * 1024 + lane * 16) = v;
    }
  }
};

template <int MT>
__device__ __forceinline__ void tile_zero(f32x4 (&acc)[MT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// ------------------------------------------------------------------ forward: x W^T

constexpr int FWD_KB = 128;  // reduction values per stage: one MX block per MFMA lane group

// acc[m][i] += W rows (as the MFMA's rows) x activation rows (its columns) over the stages
// [st0, st1) of K.  Lane (r = lane & 15, g = lane >> 4) holds MX block g of the stage of
// weight row wrow[i], 16 code bytes and a scale byte; MFMA step c takes values 8c .. 8c + 7 of
// every lane's block, and the activations are read in the same order.
template <int MT, int WM, int WN>
__device__ __forceinline__ void forward_tile(const RowStage<WM * MT * 16, FWD_KB, WM * WN>& rows,
                                             const uint8_t* const (&wrow)[4], const uint8_t* const (&srow)[4], int K,
                                             int st0, int st1, uint8_t* lds, int wm, int lane, f32x4 (&acc)[MT][4]) {
  using Stage = RowStage<WM * MT * 16, FWD_KB, WM * WN>;
  const int r = lane & 15, g = lane >> 4, blocks = K >> 5;
  u32x4 codes[4];
  uint32_t sb[4];
  // blocks past K read as zero codes with scale 1
  auto load_w = [&](int st) {
    const int b = st * 4 + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = b < blocks;
      codes[i] = ok ? ld16(wrow[i] + (size_t)b * 16) : u32x4{0u, 0u, 0u, 0u};
      sb[i] = ok ? srow[i][b] : 127u;
    }
  };
  auto load_x = [&](int st, uint8_t* buf) {
    const int valid = K - st * FWD_KB;
    if (valid >= FWD_KB)
      rows.copy(buf, st);
    else
      rows.copy_tail(buf, st, valid);
  };
  uint32_t at[4];  // LDS byte offset of this lane's activation chunk at step c, first MFMA tile
#pragma unroll
  for (int c = 0; c < 4; ++c) at[c] = (uint32_t)(wm * MT * 16 + r) * 256 + (((4 * g + c) ^ r) << 4);

  load_x(st0, lds);
  load_w(st0);
  for (int st = st0; st < st1; ++st) {
    uint8_t* cur = lds + ((st - st0) & 1) * Stage::BYTES;
    uint8_t* nxt = lds + ((st - st0 + 1) & 1) * Stage::BYTES;
    u32x4 wc[4];
    float sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wc[i] = codes[i];
      sc[i] = e8m0_scale_operand(sb[i]);
    }
    wait_copies();
    __syncthreads();  // this stage is in LDS, and nobody reads the other buffer any more
    if (st + 1 < st1) {
      load_x(st + 1, nxt);
      load_w(st + 1);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      bf16x8 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = decode8(wc[i][c], sc[i]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bf16x8 a = as_bf16x8(ld16(cur + at[c] + m * 4096));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = mfma_bf16(w[i], a, acc[m][i]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward: dz W

constexpr int BWD_KB = 64;  // reduction values (weight rows) per stage

// The weight side of a stage: 64 weight rows n of BN columns.  MFMA lane (r, g) takes columns
// 4r .. 4r + 3 of its wave's 64 (one for each of the 4 tiles) and the 8 rows of octet g, which
// it finds as 16 consecutive bytes: the 2-byte code quads of 8 rows, gathered by the threads
// that load them.  Scales are kept as fp32 per (block of 32 columns, row).
template <int BN>
struct WeightStage {
  static constexpr int QUADS = BN / 4;
  static constexpr int CODE_BYTES = BWD_KB * BN / 2;
  static constexpr int BLOCKS = BN / 32;
  static constexpr int SCALE_LD = BWD_KB + 16;
  static constexpr int BYTES = CODE_BYTES + BLOCKS * SCALE_LD * 4;
};

template <int MT, int WM, int WN>
__device__ __forceinline__ void backward_tile(const RowStage<WM * MT * 16, BWD_KB, WM * WN>& rows,
                                              const uint8_t* __restrict__ w, const uint8_t* __restrict__ s, int N,
                                              int K, int k0, int valid_n, int st0, int st1, uint8_t* lds, int wm,
                                              int wn, int lane, f32x4 (&acc)[MT][4]) {
  using Stage = RowStage<WM * MT * 16, BWD_KB, WM * WN>;
  using WS = WeightStage<WN * 64>;
  constexpr int ONE = Stage::BYTES + WS::BYTES;
  static_assert(WM * WN * 64 == 8 * WS::QUADS && WM * WN * 64 == BWD_KB * WS::BLOCKS, "one gather per thread");
  const int tid = threadIdx.x;
  const int r = lane & 15, g = lane >> 4;
  // codes: octet o of the stage's rows, column quad q of the tile (clamped inside K)
  const int o = tid / WS::QUADS, q = tid % WS::QUADS;
  const uint8_t* wp = w + (min(k0 + 4 * q, K - 4) >> 1);
  const size_t wld = (size_t)(K >> 1), sld = (size_t)(K >> 5);
  // scales: row sn, column block sk
  const int sn = tid / WS::BLOCKS, sk = tid % WS::BLOCKS;
  const uint8_t* sp = s + min((k0 >> 5) + sk, (K >> 5) - 1);
  uint32_t quad[8];
  uint32_t sb;
  // rows past N read as zero codes with scale 1
  auto load_w = [&](int st) {
    const int n = st * BWD_KB;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = n + o * 8 + i;
      quad[i] = row < N ? *reinterpret_cast<const uint16_t*>(wp + (size_t)row * wld) : 0u;
    }
    sb = n + sn < N ? sp[(size_t)(n + sn) * sld] : 127u;
  };
  auto store_w = [&](uint8_t* buf) {
    *reinterpret_cast<u32x4*>(buf + Stage::BYTES + (o * WS::QUADS + q) * 16) =
        u32x4{quad[0] | quad[1] << 16, quad[2] | quad[3] << 16, quad[4] | quad[5] << 16, quad[6] | quad[7] << 16};
    reinterpret_cast<float*>(buf + Stage::BYTES + WS::CODE_BYTES)[sk * WS::SCALE_LD + sn] = e8m0_scale_operand(sb);
  };
  auto load_x = [&](int st, uint8_t* buf) {
    const int valid = valid_n - st * BWD_KB;
    if (valid >= BWD_KB)
      rows.copy(buf, st);
    else
      rows.copy_tail(buf, st, valid);
  };
  load_x(st0, lds);
  load_w(st0);
  store_w(lds);
  for (int st = st0; st < st1; ++st) {
    uint8_t* cur = lds + ((st - st0) & 1) * ONE;
    uint8_t* nxt = lds + ((st - st0 + 1) & 1) * ONE;
    wait_copies();
    __syncthreads();
    if (st + 1 < st1) {
      load_x(st + 1, nxt);
      load_w(st + 1);
    }
    const float* scales = reinterpret_cast<const float*>(cur + Stage::BYTES + WS::CODE_BYTES);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const u32x4 d = ld16(cur + Stage::BYTES + ((4 * c + g) * WS::QUADS + wn * 16 + r) * 16);
      const float* sf = scales + (wn * 2 + (r >> 3)) * WS::SCALE_LD + c * 32 + g * 8;
      u32x4 frag[4];  // the 8 rows of columns 4r + i
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // rows 2p and 2p + 1
        const float s0 = sf[2 * p], s1 = sf[2 * p + 1];
        const uint32_t a0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[p], s0, 0));
        const uint32_t a1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[p], s0, 1));
        const uint32_t b0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[p], s1, 2));
        const uint32_t b1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[p], s1, 3));
        frag[0][p] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);  // low halves: column 4r
        frag[1][p] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
        frag[2][p] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
        frag[3][p] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = wm * MT * 16 + m * 16 + r;
        const bf16x8 a = as_bf16x8(ld16(cur + row * 128 + (((4 * c + g) ^ (r & 7)) << 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = mfma_bf16(as_bf16x8(frag[i]), a, acc[m][i]);
      }
    }
    if (st + 1 < st1) store_w(nxt);
  }
}

}  // namespace mx
