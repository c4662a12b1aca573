// Tiled products of bf16 rows with MXFP4 weights for more tokens than one weight-streaming
// pass covers: the shared pieces of the forward (x W^T) and the backward (dz W) kernels.
//
// A workgroup of WM x WN waves owns a tile of WM*MT*32 tokens by WN*NT*32 weight rows (forward)
// or columns (backward).  Each wave holds MT x NT MFMA tiles (32x32x16 bf16) in registers: a
// wave issues an instruction about every 8 cycles, and a 32x32x16 product takes 32, which
// leaves room for three others beside it (16x16x32: 16 cycles, room for one; with it the same
// tile of 128 x 128 a wave ran at 47% of the matrix rate instead).
// The activation tile goes from global memory to LDS without passing through registers
// (buffer loads to LDS, 16 bytes a lane) into the buffer that the waves are not reading, one
// barrier a stage.  The weights stay 4-bit until they are in the registers of the wave that
// multiplies with them: 4 conversions decode a fragment that MT matrix instructions use.
//
// 16-byte LDS reads go 16 lanes at a time over 64 banks, in the lane groups 0-3, 12-15, 20-23,
// 24-27 and 4-7, 8-11, 16-19, 28-31 (and the same 32 lanes on), 16-byte writes 8 consecutive
// lanes at a time over 32 banks (as the conflict counter has it for test patterns); the layouts
// below give the lanes of a group different 16-byte columns.
#pragma once
#include <utility>

#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace mx {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
typedef __attribute__((address_space(3))) void* lds_ptr;

// A buffer of up to 4 GB from a uniform address: its loads take a 32-bit offset per lane and a
// uniform one, no address arithmetic per lane; what lies past its end reads as zero.
typedef __amdgpu_buffer_rsrc_t buffer;
__device__ __forceinline__ buffer make_buffer(const void* base, uint64_t bytes) {
  const uint32_t n = bytes < 0xFFFFFFFFull ? (uint32_t)bytes : 0xFFFFFFFFu;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);  // 32-bit data, no stride
}
// 16 (4) bytes a lane from memory to LDS: lane l's bytes land at `lds` + 16 (4) * l.
__device__ __forceinline__ void copy16_to_lds(buffer b, uint32_t lane_offset, uint32_t offset, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr)lds, 16, lane_offset, offset, 0, 0);
}
__device__ __forceinline__ void copy4_to_lds(buffer b, uint32_t lane_offset, uint32_t offset, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr)lds, 4, lane_offset, offset, 0, 0);
}

// This wave's copies to LDS have landed (they count as vector memory operations, which a
// barrier alone does not wait for).
// LATER: all but the last LATER vector memory operations, which return in order.
template <int LATER = 0>
__device__ __forceinline__ void wait_copies() {
  static_assert(LATER < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER) : "memory");
}

// Consecutive tiles go to one XCD (workgroups are dealt to the 8 XCDs in turn), so that the
// tiles that share activation rows share an L2.
constexpr int XCDS = 8;
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int x = b % XCDS, i = b / XCDS, q = total / XCDS, r = total % XCDS;
  return x * q + min(x, r) + i;
}

// A value that the compiler must compute where it stands instead of keeping it in a register
// across the main loop.
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// No instruction moves across: the compiler otherwise puts the reads of the next step right
// before their use, to save registers.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// f(integral_constant<int, 0>), f(integral_constant<int, 1>), ... f(N - 1): a loop whose
// every iteration is its own code, however long (the compiler gives up unrolling a long one,
// and arrays indexed by its counter then leave the registers).
template <class F, int... I>
__device__ __forceinline__ void unrolled(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  unrolled(f, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------------------ activation stages

// A stage is KB reduction values of BM rows: rows of KB * 2 bytes in C = KB / 8 chunks of 16
// bytes, chunk c of row r at position c ^ row_key<C>(r).  The copy to LDS writes 1 KB a wave at
// consecutive addresses; the permutation is in which chunk of its row each lane fetches.
template <int C>
__device__ __forceinline__ int row_key(int r) {
  return C == 16 ? r & 15 : (r >> 1) & 7;  // rows of 256 bytes; of 128 (two to a line of banks)
}
template <int BM, int KB, int NW>
struct RowStage {
  static constexpr int C = KB / 8;                 // chunks per row
  static constexpr int BYTES = BM * KB * 2;
  static constexpr int ROWS_PER_COPY = 64 / C;     // rows of one wave-wide copy
  static constexpr int COPIES = BM / ROWS_PER_COPY / NW;  // wave-wide copies per wave
  static_assert(BM % (ROWS_PER_COPY * NW) == 0, "whole copies");

  const uint8_t* base;   // the tile's first row
  buffer buf_;           // the tile's rows
  uint32_t off[COPIES];  // byte offset of this lane's chunk in each copy
  int chunk, wave, lane;
  static_assert(NW * ROWS_PER_COPY % 16 == 0, "a lane's chunk is the same in all its copies");

  // Rows past `rows` fetch the last row again; their results are never stored.
  __device__ __forceinline__ void init(const uint16_t* x, int m0, int rows, int64_t ld, int wave_, int lane_) {
    wave = wave_, lane = lane_;
    base = reinterpret_cast<const uint8_t*>(x + (size_t)m0 * ld);
    buf_ = make_buffer(base, (uint64_t)min(BM, rows - m0) * (uint64_t)(ld * 2));
    const int r = wave * ROWS_PER_COPY + lane / C;
    chunk = (lane % C) ^ row_key<C>(r);
#pragma unroll
    for (int q = 0; q < COPIES; ++q)
      off[q] = (uint32_t)min(r + q * (NW * ROWS_PER_COPY), rows - 1 - m0) * (uint32_t)(ld * 2) + chunk * 16;
  }
  // copy q of COPIES of this wave
  __device__ __forceinline__ void copy_one(uint8_t* buf, int stage, int q) const {
    copy16_to_lds(buf_, off[q], (uint32_t)stage * (KB * 2), buf + (q * NW + wave) * 1024);
  }
  __device__ __forceinline__ void copy(uint8_t* buf, int stage) const {
#pragma unroll
    for (int q = 0; q < COPIES; ++q) copy_one(buf, stage, q);
  }
  // The last, partial stage: `valid` (< KB, a multiple of 8) values of each row, zeros beyond.
  __device__ __forceinline__ void copy_tail(uint8_t* buf, int stage, int valid) const {
    const uint8_t* p = base + (size_t)stage * (KB * 2);
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const u32x4 v = chunk * 8 < valid ? ld16(p + here(off[q])) : u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(buf + (q * NW + wave) * 1024 + lane * 16) = v;
    }
  }
};

template <int MT, int NT>
__device__ __forceinline__ void tile_zero(f32x16 (&acc)[MT][NT]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[m][i][j] = 0.f;
}

// ------------------------------------------------------------------ which tiles

// Tiles of 256 x 256 (one a CU) or 128 x 128 (two a CU)?  The large ones take less time for the
// same work, the small ones leave fewer CUs idle in the last round.  What a round of each takes
// (of 256 and of 512 tiles; microseconds at a reduction of 7168 forward and 4096 backward):
//   forward   174 and 106     gate_up of 1536 to 4096 tokens, H = 7168, I = 2048
//   backward   99 and 80      7168 <- 4096, 2048 and 1024 tokens
// e.g. gate_up at 2048 tokens takes 108 with the small tiles and 111 with the large ones, at
// 3000 tokens 174 and 143; the backward of 4096 tokens 270 and 200.
constexpr int FORWARD_ROUND_256 = 174, FORWARD_ROUND_128 = 106;
constexpr int BACKWARD_ROUND_256 = 99, BACKWARD_ROUND_128 = 80;
inline int tile_choice(int64_t T, int64_t cols, int64_t round_256, int64_t round_128) {
  const int64_t large = ((T + 255) / 256) * ((cols + 255) / 256), small = ((T + 127) / 128) * ((cols + 127) / 128);
  return (large + GPU_CUS - 1) / GPU_CUS * round_256 <= (small + 2 * GPU_CUS - 1) / (2 * GPU_CUS) * round_128 ? 4 : 2;
}
// Over how many workgroups the reduction of a tile is split, each with two stages or more: as
// many as there are CUs for, and two (fill_second) where tiles of 128 x 128 then take the second
// place on each CU and the reduction is long (gate_up, H = 7168: 768 tokens 65 -> 57 us; not
// 2048 -> 7168, 31 -> 45).
inline int64_t tile_split(int64_t tiles, int64_t stages, bool fill_second) {
  const int64_t split = std::max<int64_t>(GPU_CUS / tiles, fill_second && tiles <= GPU_CUS ? 2 : 1);
  return std::max<int64_t>(1, std::min(split, stages / 2));
}

// ------------------------------------------------------------------ matrix instructions

// acc += a x b in place: lane (r = lane & 31, g = lane >> 5) gives values 8g .. 8g + 7 of row r
// of a and of column r of b, and holds rows 8 (j >> 2) + 4 g + (j & 3) of column r of acc.
// The compiler's own choice of registers for accumulators that fill all 256 accumulation
// registers moves them about between matrix instructions (as many moves as products); tied
// operands cannot move.  See settle_mfma and operands_ready.
__device__ __forceinline__ void mfma_in_place(f32x16& acc, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// The compiler does not see that the instructions above multiply, so it keeps none of their
// distances.  This stands between them and what writes or reads their accumulators otherwise
// (before the first and after the last): it waits out the longest of them (18 wait states),
// and the ties keep those writes and reads on their side of it.
template <int MT, int NT>
__device__ __forceinline__ void settle_mfma(f32x16 (&acc)[MT][NT]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) asm volatile("" : "+a"(acc[m][i]));
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) asm volatile("" : "+a"(acc[m][i]));
}
// Two wait states between the vector instructions that write these operands and the product.
// The operands are tied: what computes them cannot move behind this.
template <int NT>
__device__ __forceinline__ void operands_ready(u32x4 (&w)[NT]) {
  static_assert(NT == 2 || NT == 4, "tiles of a wave");
  if constexpr (NT == 2)
    asm volatile("s_nop 1" : "+v"(w[0]), "+v"(w[1]));
  else
    asm volatile("s_nop 1" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
}

// Value pair Q of 8 codes.
template <int Q>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, Q));
}

// ------------------------------------------------------------------ forward: x W^T

constexpr int FWD_KB = 128;  // reduction values per stage: 4 MX blocks, two per MFMA lane group

// The weight codes of a stage: BN rows of 64 bytes (4 MX blocks); LDS row 32 i + r is MFMA row
// r of the workgroup's MFMA tile i.  Block b of row r sits at chunk b ^ (r >> 3).
template <int BN, int NW>
struct CodeStage {
  static constexpr int BYTES = BN * 64;
  static constexpr int COPIES = BN / 16 / NW;  // wave-wide copies of 16 rows per wave
  static_assert(BN % (16 * NW) == 0, "whole copies");
  const uint8_t* base[COPIES];  // the first weight row of the copy's half (the same in a wave)
  buffer buf_[COPIES];          // that half's rows of the tile
  uint32_t off[COPIES];         // this lane's chunk from there, stage 0
  int wave, lane;

  // which of a stage's 4 blocks the lane copies
  __device__ __forceinline__ int block(int q) const {
    return (lane & 3) ^ ((((q * NW + wave) * 16 + (lane >> 2)) >> 3) & 3);
  }
  // half_of(MFMA tile) = first row of that tile's half, of which the tile has tile_rows;
  // row_of(LDS row) = row within it
  template <class F, class G>
  __device__ __forceinline__ void init(int K, int tile_rows, int wave_, int lane_, F half_of, G row_of) {
    wave = wave_, lane = lane_;
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      base[q] = half_of((q * NW + wave) >> 1);
      buf_[q] = make_buffer(base[q], (uint64_t)tile_rows * (uint64_t)(K >> 1));
      off[q] = (uint32_t)row_of((q * NW + wave) * 16 + (lane >> 2)) * (uint32_t)(K >> 1) + block(q) * 16;
    }
  }
  __device__ __forceinline__ void copy_one(uint8_t* buf, int stage, int q) const {
    copy16_to_lds(buf_[q], off[q], (uint32_t)stage * 64, buf + (q * NW + wave) * 1024);
  }
  // The last, partial stage: `valid` (< 4) blocks of each row, zero codes beyond.
  __device__ __forceinline__ void copy_tail(uint8_t* buf, int stage, int valid) const {
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const u32x4 v = block(q) < valid ? ld16(base[q] + (size_t)stage * 64 + here(off[q])) : u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(buf + (q * NW + wave) * 1024 + lane * 16) = v;
    }
  }
};

// The scale bytes of a stage (4 a row) of a wave's weight rows, where they pass through the
// LDS: 64 rows a copy, each wave its own.
template <int NT, int NW>
struct ScaleStage {
  static constexpr int COPIES = NT / 2, BYTES = NW * COPIES * 256;
  buffer buf_;
  uint32_t off[COPIES];
  int wave;
  __device__ __forceinline__ void copy_one(uint8_t* buf, int stage, int q) const {
    copy4_to_lds(buf_, off[q], (uint32_t)stage * 4, buf + (wave * COPIES + q) * 256);
  }
};

// D: stages in the LDS.
template <int MT, int NT, int WM, int WN, int D>
struct ForwardLds {
  typedef RowStage<WM * MT * 32, FWD_KB, WM * WN> Rows;
  typedef CodeStage<WN * NT * 32, WM * WN> Codes;
  typedef ScaleStage<NT, WM * WN> Scales;
  static constexpr int CODES_AT = Rows::BYTES, SCALES_AT = CODES_AT + Codes::BYTES;
  static constexpr int ONE = SCALES_AT + (D > 2 ? Scales::BYTES : 0);
  static constexpr int BYTES = D * ONE;
};

// acc[m][i] += W rows (as the MFMA's rows) x activation rows (its columns) over the stages
// [st0, st1) of K (K >= FWD_KB).  Lane (r = lane & 31, g = lane >> 5) holds MX blocks g and
// g + 2 of the stage of MFMA row r of tile i, 16 code bytes and a scale byte each.  A stage is
// 8 steps; step u multiplies values 8 (u & 3) .. + 7 of every lane's block g + 2 (u >> 2), and
// the activations are read in the same order.
//
// Between the matrix instructions of a step, in slots that they leave free, the wave reads the
// activation fragments and decodes the weights of the next step and, early in the stage,
// copies a later stage to LDS.  The stage's only barrier stands before its last step, whose
// operands are already in registers.
//
// D = 2 (the tiles of 256 x 256 fill the LDS with that): copies are one stage ahead, scales
// are loaded to registers.  D > 2, for products with one small tile a CU and few stages, which
// wait for memory: copies are D - 1 stages ahead, scales among them; K % FWD_KB == 0 then, and
// scale rows are 4-byte aligned.
template <int MT, int NT, int WM, int WN, int D>
__device__ __forceinline__ void forward_tile(const typename ForwardLds<MT, NT, WM, WN, D>::Rows& rows,
                                             const typename ForwardLds<MT, NT, WM, WN, D>::Codes& codes,
                                             const typename ForwardLds<MT, NT, WM, WN, D>::Scales& scales,
                                             const uint8_t* const (&sbase)[NT], uint32_t scale_bytes,
                                             const uint32_t (&soff)[NT], int K, int st0, int st1, uint8_t* lds,
                                             int wm, int wn, int lane, f32x16 (&acc)[MT][NT]) {
  typedef ForwardLds<MT, NT, WM, WN, D> L;
  constexpr bool DEEP = D > 2;
  constexpr int STEPS = 8, SLOTS = MT * NT;
  constexpr int XC = L::Rows::COPIES, WC = L::Codes::COPIES;
  // loads from memory: one every LOAD_EVERY slots of the first five steps, or several a slot
  constexpr int LOADS = XC + WC + (DEEP ? L::Scales::COPIES : NT), LOAD_SLOTS = 5 * SLOTS;
  constexpr int LOADS_AT_ONCE = (LOADS + LOAD_SLOTS - 1) / LOAD_SLOTS;
  constexpr int LOAD_EVERY = LOADS > LOAD_SLOTS ? 1 : LOAD_SLOTS / LOADS < 3 ? LOAD_SLOTS / LOADS : 3;
  const int r = lane & 31, g = lane >> 5, blocks = K >> 5;
  const int full = K / FWD_KB;  // stages of FWD_KB values
  const uint32_t xrow = (uint32_t)(wm * MT * 32 + r) * 256;
  const uint32_t wrow = L::CODES_AT + (uint32_t)(wn * NT * 32 + r) * 64;
  uint32_t at[8];  // LDS byte offset of this lane's activation chunk at step u, first tile
#pragma unroll
  for (int u = 0; u < 8; ++u) at[u] = xrow + (((8 * (u >> 2) + 4 * g + (u & 3)) ^ (r & 15)) << 4);
  uint32_t wat[2];  // of its blocks
#pragma unroll
  for (int b = 0; b < 2; ++b) wat[b] = wrow + (((2 * b + g) ^ (r >> 3)) << 4);
  const uint32_t sat = L::SCALES_AT + (uint32_t)(wm * WN + wn) * (L::Scales::COPIES * 256) + r * 4;  // of its scales
  u32x4 wc[2][NT], frag[2][MT], w[2][NT];
  uint32_t sd[NT];  // a stage's 4 scale bytes of the row of tile i
  float sc[2][NT];
  buffer sbuf[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) sbuf[i] = make_buffer(sbase[i], scale_bytes);
  // load q of LOADS of a stage
  auto load = [&](uint8_t* buf, int st, auto Q) __attribute__((always_inline)) {
    constexpr int q = Q;
    if constexpr (q < XC)
      rows.copy_one(buf, st, q);
    else if constexpr (q < XC + WC)
      codes.copy_one(buf + L::CODES_AT, st, q - XC);
    else if constexpr (DEEP)
      scales.copy_one(buf + L::SCALES_AT, st, q - XC - WC);
    else
      sd[q - XC - WC] = __builtin_amdgcn_raw_buffer_load_b32(sbuf[q - XC - WC], soff[q - XC - WC], st * 4, 0);
  };
  // The partial stage, through registers, and its scales byte by byte (a row may end with the
  // tensor); blocks past K have zero codes and scale 1.
  auto load_tail = [&](uint8_t* buf) {
    rows.copy_tail(buf, full, K - full * FWD_KB);
    codes.copy_tail(buf + L::CODES_AT, full, blocks & 3);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint32_t d = 0x7F7F7F7Fu;
      for (int b = 0; b < (blocks & 3); ++b)
        d = (d & ~(0xFFu << (8 * b))) | (uint32_t)sbase[i][soff[i] + full * 4 + b] << (8 * b);
      sd[i] = d;
    }
  };
  auto read_scale = [&](const uint8_t* buf, int i) {
    if constexpr (DEEP) sd[i] = *reinterpret_cast<const uint32_t*>(buf + sat + (i >> 1) * 256 + (i & 1) * 128);
  };
  // of tile i: this lane's blocks g and g + 2
  auto use_scale = [&](int i) {
    const uint32_t d = sd[i] >> (8 * g);
    sc[0][i] = e8m0_scale_operand(d & 0xFFu);
    sc[1][i] = e8m0_scale_operand((d >> 16) & 0xFFu);
  };
  // the buffers of the current and of the next stage, and the one that is filled meanwhile
  uint8_t* cur = lds;
  uint8_t* nxt = lds + L::ONE;
  uint8_t* fill = lds + (D - 1) * L::ONE;
  if (DEEP || st0 < full) {
    unrolled<D - 1>([&](auto J) __attribute__((always_inline)) {
      unrolled<LOADS>([&](auto Q) __attribute__((always_inline)) { load(lds + J * L::ONE, min(st0 + J, full - 1), Q); });
    });
  } else {
    load_tail(cur);
  }
  wait_copies<(D - 2) * LOADS>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    read_scale(cur, i);
    use_scale(i);
#pragma unroll
    for (int b = 0; b < 2; ++b) wc[b][i] = ld16(cur + wat[b] + i * 2048);
    w[0][i] = __builtin_bit_cast(u32x4, decode8(wc[0][i][0], sc[0][i]));
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) frag[0][m] = ld16(cur + at[0] + m * 8192);
  settle_mfma(acc);  // the accumulators have been cleared
  operands_ready<NT>(w[0]);
  for (int st = st0; st < st1; ++st) {
    // The stage that is copied meanwhile.  Past the last full one its copy repeats that one:
    // the partial stage is written over it, and after the last stage nothing reads it.
    const int cs = min(st + D - 1, full - 1);
    unrolled<STEPS>([&](auto U) __attribute__((always_inline)) {
      constexpr int u = U, next = (u + 1) % STEPS;
      constexpr bool last = u == STEPS - 1;
      if constexpr (last) {
        wait_copies<(D - 2) * LOADS>();  // the next stage has landed
        if constexpr (!DEEP) {
          if (st + 1 == full && st + 1 < st1) load_tail(nxt);
        }
        __syncthreads();  // for every wave, and no wave reads `cur` any more
      }
      // The slots' reads and conversions; in the last step the reads, which the conversions
      // wait for, fill the first half.
      constexpr int SR = last && DEEP ? NT : 0, CR = last ? 2 * NT : 0;
      constexpr int reads = SR + CR + MT, converts = 4 * NT;
      constexpr int first = last ? SLOTS / 2 : 0;  // slot of the first conversion
      constexpr int per_read = (reads + (last ? (SLOTS + 1) / 2 : SLOTS) - 1) / (last ? (SLOTS + 1) / 2 : SLOTS);
      constexpr int per_convert = (converts + SLOTS - first - 1) / (SLOTS - first);
      unrolled<SLOTS>([&](auto S) __attribute__((always_inline)) {
        constexpr int k = S, m = k / NT, i = k % NT;
        mfma_in_place(acc[m][i], w[u & 1][i], frag[u & 1][m]);
        unrolled<per_read>([&](auto E) __attribute__((always_inline)) {
          constexpr int e = k * per_read + E;
          if constexpr (e < SR)
            read_scale(nxt, e);
          else if constexpr (e < SR + CR)
            wc[(e - SR) / NT][(e - SR) % NT] = ld16(nxt + wat[(e - SR) / NT] + ((e - SR) % NT) * 2048);
          else if constexpr (e < reads)
            frag[next & 1][e - SR - CR] = ld16((last ? nxt : cur) + at[next] + (e - SR - CR) * 8192);
        });
        // the next stage's scales, before its first conversion
        if constexpr (last && DEEP && k == first) {
#pragma unroll
          for (int j = 0; j < NT; ++j) use_scale(j);
        }
        if constexpr (last && !DEEP && k < SLOTS / 2) {
          constexpr int per_scale = (NT + SLOTS / 2 - 1) / (SLOTS / 2);
#pragma unroll
          for (int j = k * per_scale; j < (k + 1) * per_scale && j < NT; ++j) use_scale(j);
        }
        unrolled<per_convert>([&](auto E) __attribute__((always_inline)) {
          constexpr int e = (k - first) * per_convert + E;
          if constexpr (e >= 0 && e < converts) {
            constexpr int j = e / 4, q = e & 3;
            w[next & 1][j][q] = decode2<q>(wc[next >> 2][j][next & 3], sc[next >> 2][j]);
          }
        });
        // loads, one every few slots from the stage's first on
        constexpr int n = u * SLOTS + k;
        if constexpr (n % LOAD_EVERY == LOAD_EVERY - 1)
          unrolled<LOADS_AT_ONCE>([&](auto E) __attribute__((always_inline)) {
            constexpr int q = n / LOAD_EVERY * LOADS_AT_ONCE + E;
            if constexpr (q < LOADS) load(fill, cs, std::integral_constant<int, q>{});
          });
        keep_order();
      });
      operands_ready<NT>(w[next & 1]);
    });
    fill = cur;
    cur = nxt;
    nxt = nxt == lds + (D - 1) * L::ONE ? lds : nxt + L::ONE;
  }
  settle_mfma(acc);
  if constexpr (DEEP) wait_copies();  // the last stages' repeated copies: the LDS is used again
}

// A wave's results, one row of MFMA tiles (32 tokens) at a time, through its own part of the
// LDS (free after the main loop and a barrier): rows of NT * 32 floats, 4 to a chunk.  The
// epilogue then reads them back by rows, so that its accesses to memory are whole lines.
template <int NT>
__device__ __forceinline__ uint32_t out_at(int row, int chunk) {
  return (uint32_t)row * (NT * 128) + ((chunk ^ (row & 15 & (NT * 8 - 1))) << 4);
}
// Writes tile row m of acc there.
template <int NT>
__device__ __forceinline__ void tile_to_lds(uint8_t* mine, const f32x16 (&acc)[NT], int lane) {
  const int r = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4*>(mine + out_at<NT>(r, 8 * i + 2 * j + g)) =
          f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
}

// ------------------------------------------------------------------ backward: dz W

constexpr int BWD_KB = 64;  // reduction values (weight rows) per stage

// Here the reduction runs over weight rows, across the packing and the scales (a block of 32
// shares one along the columns).  A thread takes CPT columns (CPT / 2 bytes) of 8 consecutive
// weight rows, an octet, of the stage, decodes each row's pairs with that row's scale and
// exchanges halves between two rows, and writes each column's 8 bf16 values as one 16-byte
// chunk, so that every weight is decoded once a workgroup and the LDS holds both operands in
// the same form: rows of 64 reduction values.  (Decoding in the registers of each wave that
// multiplies takes twice the conversions and as many LDS reads: 64 x 256 weights a stage.)
// Column CPT q + 2 i + (R >> 4) of a wave's, with R & 15 = column_row(q), is MFMA row R of its
// tile i: a lane's results are then CPT consecutive columns, and the rows that 8 consecutive
// threads write (every other one) have different keys.
__device__ __forceinline__ int column_row(int q) { return ((q & 7) << 1) | (q >> 3); }   // q < 16
__device__ __forceinline__ int column_of_row(int r) { return (r >> 1) | ((r & 1) << 3); }  // its inverse
template <int NT>
struct ColumnStage {
  static constexpr int CPT = 2 * NT;              // columns of a thread: WN * NT * 32 over 32 threads
  static constexpr int BYTES = 2 * NT * 32 * 128;  // two wave columns
};

template <int MT, int NT>
struct BackwardLds {
  typedef RowStage<2 * MT * 32, BWD_KB, 4> Rows;
  static constexpr int ONE = Rows::BYTES + ColumnStage<NT>::BYTES;
  static constexpr int BYTES = 2 * ONE;
};

// acc[m][i] += W columns (as the MFMA's rows) x dz rows (its columns) over the stages
// [st0, st1) of weight rows, for a workgroup of 2 x 2 waves.  dz has a multiple of 64 columns,
// those past N zero.  A stage is 4 steps, and as in forward_tile what prepares later ones goes
// between the matrix instructions.  Both operands' fragments come from the LDS here (192 KB of
// its traffic a stage of 256 x 256, three quarters of the time of the products), so they are
// read two steps ahead, one every other slot, and the barrier stands in the middle of the
// stage: from step 2 on the next stage's fragments are read, and the buffer of the current one
// is filled again, dz rows by copies, weights by decoding codes that were loaded nearly a stage
// before.  The gate_up backward of 4096 tokens (H = 7168, I = 2048) takes 220 us with the work
// spread like this, 221 with all reads in the first half of a step and decoding in two of the
// four, and 225 with the codes loaded 30 products before their use as well.  The products are busy
// for 54% of the launch's cycles, at 2.0 GHz; alone they would hold the clock at 1.7 (1.2 us a
// stage, 1.5 with all of the work beside them).
template <int MT, int NT>
__device__ __forceinline__ void backward_tile(const typename BackwardLds<MT, NT>::Rows& rows,
                                              const uint8_t* __restrict__ w, const uint8_t* __restrict__ s, int N,
                                              int K, int k0, int st0, int st1, uint8_t* lds, int wm, int wn, int lane,
                                              f32x16 (&acc)[MT][NT]) {
  typedef BackwardLds<MT, NT> L;
  constexpr int STEPS = 4, SLOTS = MT * NT, CPT = ColumnStage<NT>::CPT, COPIES = L::Rows::COPIES;
  constexpr int READS = MT + NT;
  const int r = lane & 31, g = lane >> 5, o = threadIdx.x >> 5, q = threadIdx.x & 31;
  const int wld = K >> 1, sld = K >> 5;
  const int col = min(k0 + CPT * q, K - CPT);  // columns past K: the last ones again, never stored
  // byte offsets of this thread's 8 rows from the stage's first
  uint32_t woff[8], soff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    woff[i] = (uint32_t)((o * 8 + i) * wld + (col >> 1));
    soff[i] = (uint32_t)((o * 8 + i) * sld + (col >> 5));
  }
  uint32_t at[4], wat[4];  // LDS byte offsets of this lane's chunks at step u, first tile
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    at[u] = (uint32_t)(wm * MT * 32 + r) * 128 + (((2 * u + g) ^ row_key<8>(r)) << 4);
    wat[u] = L::Rows::BYTES + (uint32_t)(wn * NT * 32 + r) * 128 + (((2 * u + g) ^ row_key<8>(r)) << 4);
  }
  // where this thread's columns go: LDS row 16 i + column_row(q & 15) of its wave column, chunk o
  const int qrow = column_row(q & 15);
  const uint32_t put = L::Rows::BYTES + (uint32_t)((q >> 4) * NT * 32 + qrow) * 128 + ((o ^ row_key<8>(qrow)) << 4);
  uint32_t code[8];  // of the stage after the current one, and its rows' scales
  float scale[8];
  uint32_t code2[8], scale2[8];  // of the stage after that, as loaded
  u32x4 frag[STEPS][MT], wf[STEPS][NT], column[2];
  // The first weight row of the stage that load_one loads from, moved on a stage at a time.
  const uint8_t* wstage = w + (size_t)st0 * BWD_KB * wld;
  const uint8_t* sstage = s + (size_t)st0 * BWD_KB * sld;
  auto load_one = [&](int i) {
    if constexpr (CPT == 8)
      code2[i] = *reinterpret_cast<const uint32_t*>(wstage + woff[i]);
    else
      code2[i] = *reinterpret_cast<const uint16_t*>(wstage + woff[i]);
    scale2[i] = sstage[soff[i]];
  };
  auto take_one = [&](int i) {
    code[i] = here(code2[i]);
    scale[i] = __uint_as_float(here(__float_as_uint(e8m0_scale_operand(scale2[i]))));
  };
  auto move_on = [&](bool yes) {
    wstage += yes ? BWD_KB * wld : 0;
    sstage += yes ? BWD_KB * sld : 0;
  };
  // Rows past N (in the last stage): their addresses are moved to row N - 1 before they are
  // loaded, and their values replaced by zero codes with scale 1 before they are used.
  const int last_stage = (N - 1) / BWD_KB, left = N - last_stage * BWD_KB;
  auto clamp_rows = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = min(o * 8 + i, left - 1);
      woff[i] = (uint32_t)(row * wld + (col >> 1));
      soff[i] = (uint32_t)(row * sld + (col >> 5));
    }
  };
  auto clear_rows = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (o * 8 + i >= left) code[i] = 0u, scale[i] = 1.f;
  };
  // half of column pair b, row pair p2: rows 2 p2 and 2 p2 + 1
  auto decode_pair = [&](auto B, auto P2) __attribute__((always_inline)) {
    constexpr int b = B, p2 = P2;
    const uint32_t lo = decode2<b>(code[2 * p2], scale[2 * p2]);
    const uint32_t hi = decode2<b>(code[2 * p2 + 1], scale[2 * p2 + 1]);
    column[0][p2] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);  // low halves: column 2b
    column[1][p2] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
  };
  auto put_column = [&](uint8_t* buf, int b, int h) {
    *reinterpret_cast<u32x4*>(buf + put + (2 * b + h) * 2048) = column[h];
  };
  auto read_one = [&](const uint8_t* buf, int u, int e) {  // operand e of step u
    if (e < MT)
      frag[u][e] = ld16(buf + at[u] + e * 4096);
    else
      wf[u][e - MT] = ld16(buf + wat[u] + (e - MT) * 4096);
  };
  // Decoding takes the slots of steps 2, 3 and the next 0: unit e of UNITS is a row pair of a
  // column pair, whose columns are written after its last.
  constexpr int UNITS = 4 * NT;
  auto unit = [&](uint8_t* buf, auto E) __attribute__((always_inline)) {
    constexpr int e = E;
    decode_pair(std::integral_constant<int, e / 4>{}, std::integral_constant<int, e % 4>{});
    if constexpr (e % 4 == 3) {
      put_column(buf, e / 4, 0);
      put_column(buf, e / 4, 1);
    }
  };

  // the first stage, the second as far as a step 3 leaves it, and the third's codes
  const bool ragged = left < BWD_KB;
  uint8_t* cur = lds;
  uint8_t* nxt = lds + L::ONE;
  const int second = min(st0 + 1, st1 - 1), third = min(st0 + 2, st1 - 1);
  auto load_stage = [&](int st) {
    if (ragged && st == last_stage) clamp_rows();
#pragma unroll
    for (int i = 0; i < 8; ++i) load_one(i);
  };
  auto take_stage = [&](int st) {
#pragma unroll
    for (int i = 0; i < 8; ++i) take_one(i);
    if (ragged && st == last_stage) clear_rows();
  };
  load_stage(st0);
  rows.copy(cur, st0);
  rows.copy(nxt, second);
  take_stage(st0);
  move_on(second > st0);
  load_stage(second);
  unrolled<UNITS>([&](auto E) __attribute__((always_inline)) { unit(cur, E); });
  take_stage(second);
  move_on(third > second);
  load_stage(third);
  unrolled<UNITS>([&](auto E) __attribute__((always_inline)) {
    if constexpr (3 * E < 2 * UNITS) unit(nxt, E);
  });
  wait_copies();
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < READS; ++e) read_one(cur, u, e);
  settle_mfma(acc);  // the accumulators have been cleared

  for (int st = st0; st < st1; ++st) {
    // the stages that are decoded and copied, and loaded, from step 2 on; past the last one that
    // one again, which nothing uses
    const int cs = min(st + 2, st1 - 1), ls = min(st + 3, st1 - 1);
    unrolled<STEPS>([&](auto U) __attribute__((always_inline)) {
      constexpr int u = U;
      if constexpr (u == 2) {
        if (ragged) {
          if (cs == last_stage) clear_rows();
          if (ls == last_stage) clamp_rows();
        }
        move_on(ls > cs);
        wait_copies();
        __syncthreads();  // the next stage is whole, and every wave has read the last of `cur`
      }
      unrolled<SLOTS>([&](auto S) __attribute__((always_inline)) {
        constexpr int k = S, m = k / NT, i = k % NT;
        mfma_in_place(acc[m][i], wf[u][i], frag[u][m]);
        // of n items E stands in slot E * slots / n, the reads half a distance later
        unrolled<READS>([&](auto E) __attribute__((always_inline)) {
          if constexpr ((2 * E + 1) * SLOTS / (2 * READS) == k) read_one(u < 2 ? cur : nxt, (u + 2) % STEPS, E);
        });
        constexpr int d = (u + 2) % STEPS * SLOTS + k;  // slot of the decoding
        unrolled<UNITS>([&](auto E) __attribute__((always_inline)) {
          if constexpr (E * (3 * SLOTS) / UNITS == d) unit(u == 0 ? nxt : cur, E);
        });
        // step 1: what was loaded in step 3 is taken over; step 2: copies of dz rows; step 3:
        // loads of codes and scales
        unrolled<8>([&](auto E) __attribute__((always_inline)) {
          if constexpr (E * SLOTS / 8 == k) {
            if constexpr (u == 1) take_one(E);
            if constexpr (u == 3) load_one(E);
          }
        });
        if constexpr (u == 2)
          unrolled<COPIES>([&](auto E) __attribute__((always_inline)) {
            if constexpr (E * SLOTS / COPIES == k) rows.copy_one(cur, cs, E);
          });
        keep_order();
      });
    });
    uint8_t* t = cur;
    cur = nxt;
    nxt = t;
  }
  settle_mfma(acc);
}

}  // namespace mx
