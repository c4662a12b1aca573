// Tiled products of MXFP8 or MXFP4 rows with MXFP4 weights on the scaled matrix instructions:
// neither side is decoded, both go from memory to the LDS by buffer loads and from there into the
// operand registers as they are stored.
//
// A workgroup of WM x WN waves owns 32 WM MT tokens by 32 WN NT weight rows; a wave holds MT x NT tiles of
// v_mfma_scale_f32_32x32x64_f8f6f4 (weights are its rows, tokens its columns).  Lane (r = lane & 31,
// g = lane >> 5) of an instruction over 64 values (two blocks) gives
//   E2M1: the 32 values of block g, 16 bytes;
//   E4M3: values 16 g .. 16 g + 15 of each of the two blocks, 2 x 16 bytes;
//   and in either case the scale byte of block g,
// and holds rows 8 (j >> 2) + 4 g + (j & 3) of column r of the result.
//
// A stage is 128 or 256 values of the reduction, two or four steps of 64.  Rows of 128 bytes a stage are whole
// lines of memory: a CU reads 75 kB a microsecond of those, 52 of halves (512 rows of 3584 bytes, copies to the LDS
// and nothing else).
// Scales stay in the LDS 512 values at a time: 16 bytes a row, so that a row's line is touched once
// for them (a dword each 128 would touch as many lines as the codes do).
#pragma once
#include "mx_quant.hpp"
#include "mx_tile.hpp"

namespace mx {

constexpr int Q_KG = 512;              // whose scales go together
constexpr uint32_t Q_NOWHERE = 1u << 31;  // a lane offset past the end of every buffer here: reads as zero

// This wave's copies but the last LATER have landed and its LDS accesses are done; then the barrier.
// (__syncthreads would wait for all copies, those of later stages among them.)
template <int LATER>
__device__ __forceinline__ void q_barrier() {
  static_assert(LATER < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
}

// ROWS rows of RB bytes a stage, in chunks of 16 bytes: chunk c of row r lies at c ^ q_key(r), which
// puts the lanes that one LDS access serves together into different banks (mx_tile.hpp).
template <int RB>
__device__ __forceinline__ int q_key(int r) {
  return RB == 128 ? (r >> 1) & 7 : (r >> 3) & 3;
}
template <int ROWS, int RB, int NW>
struct QStage {
  static constexpr int C = RB / 16, PER_COPY = 64 / C, COPIES = ROWS / PER_COPY / NW, BYTES = ROWS * RB;
  static_assert(ROWS % (PER_COPY * NW) == 0 && 32 % PER_COPY == 0, "whole copies, each within an MFMA tile");
  static_assert(RB == 128 ? NW * PER_COPY % 16 == 0 : NW * PER_COPY % 32 == 0, "a lane's chunk is the same in all its copies");
  buffer buf_[COPIES];   // the rows of the copy's half
  uint32_t off[COPIES];  // this lane's chunk from there, stage 0
  int chunk, wave;

  // base_of(row) = first row of the half that LDS row `row` lies in, of which `have` exist; row_of(row) =
  // its row within the half
  template <class F, class G>
  __device__ __forceinline__ void init(int64_t row_bytes, int have, int wave_, int lane, F base_of, G row_of) {
    wave = wave_;
    chunk = (lane % C) ^ q_key<RB>(wave * PER_COPY + lane / C);
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
      const int first = (q * NW + wave) * PER_COPY;
      buf_[q] = make_buffer(base_of(first), (uint64_t)have * (uint64_t)row_bytes);
      off[q] = (uint32_t)row_of(first + lane / C) * (uint32_t)row_bytes + chunk * 16;
    }
  }
  __device__ __forceinline__ void copy_one(uint8_t* lds, int stage, int q) const {
    copy16_to_lds(buf_[q], off[q], (uint32_t)stage * RB, lds + (q * NW + wave) * 1024);
  }
  // Before the copies of the last, partial stage: `chunks` of a row's exist there, the others become zeros.
  __device__ __forceinline__ void only(int chunks, int q) {
    if (chunk >= chunks) off[q] = Q_NOWHERE;
  }
};

// KB: values of a stage; D: stages in the LDS.
template <int FMT, int KB, int MT, int NT, int WM, int WN, int D>
struct QLds {
  static constexpr int NW = WM * WN, BM = 32 * WM * MT, BN = 32 * WN * NT;
  static constexpr int STEPS = KB / 64, GROUP = Q_KG / KB;  // of a stage, stages of a group
  static constexpr int ARB = KB * FMT / 8, WRB = KB / 2;  // bytes of a stage of a row
  typedef QStage<BM, ARB, NW> Rows;
  typedef QStage<BN, WRB, NW> Codes;
  static constexpr int ONE = Rows::BYTES + Codes::BYTES;
  static constexpr int SCALES_AT = D * ONE, SCALES = (BM + BN) * 16;
  static constexpr int BYTES = SCALES_AT + 2 * SCALES;
  static constexpr int PER_SIMD = NW < 4 ? 1 : NW / 4 * (BYTES > 81920 ? 1 : 2);  // waves
};

template <int FMT>
struct QFragment {
  u32x4 v[FMT / 4];
};
__device__ __forceinline__ i32x8 q_operand(const QFragment<8>& f) {
  return __builtin_bit_cast(i32x8, __builtin_shufflevector(f.v[0], f.v[1], 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ i32x8 q_operand(const QFragment<4>& f) {
  return i32x8{(int)f.v[0][0], (int)f.v[0][1], (int)f.v[0][2], (int)f.v[0][3], 0, 0, 0, 0};
}

// acc += w x a over 64 values in place; the scales are byte 2 U of sw and sa.  As an instruction of our own:
// the compiler moves products that it knows past the barrier, away from the reads and copies that they
// should run beside.  It keeps no distances for it either: see settle_mfma, and scales_ready for the scales,
// which vector instructions write (the codes come from the LDS, for which the compiler waits).
template <int U>
__device__ __forceinline__ void mfma_q(f32x16& acc, const u32x4& w, const QFragment<8>& a, uint32_t sw, uint32_t sa) {
  const i32x8 v = __builtin_bit_cast(i32x8, __builtin_shufflevector(a.v[0], a.v[1], 0, 1, 2, 3, 4, 5, 6, 7));
  asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[%5,%5,0] cbsz:4"
               : "+a"(acc) : "v"(w), "v"(v), "v"(sw), "v"(sa), "n"(U));
}
template <int U>
__device__ __forceinline__ void mfma_q(f32x16& acc, const u32x4& w, const QFragment<4>& a, uint32_t sw, uint32_t sa) {
  asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[%5,%5,0] cbsz:4 blgp:4"
               : "+a"(acc) : "v"(w), "v"(a.v[0]), "v"(sw), "v"(sa), "n"(U));
}
// Two wait states between the last of these scales' shifts and a product.
template <int N, int M>
__device__ __forceinline__ void scales_ready(uint32_t (&s)[N][M], int m) {
  static_assert(N == 1 || N == 2 || N == 4, "tiles of a wave");
  if constexpr (N == 1)
    asm volatile("s_nop 1" : "+v"(s[0][m]));
  else if constexpr (N == 2)
    asm volatile("s_nop 1" : "+v"(s[0][m]), "+v"(s[1][m]));
  else
    asm volatile("s_nop 1" : "+v"(s[0][m]), "+v"(s[1][m]), "+v"(s[2][m]), "+v"(s[3][m]));
}

// Scales of 512 values of a workgroup's BM + BN rows, 16 bytes each, into the LDS.  Rows that start at
// multiples of 16 bytes go there directly, others through registers.
template <int BM, int BN, int THREADS>
struct QScales {
  static constexpr int ROWS = BM + BN, EACH = (ROWS + THREADS - 1) / THREADS;
  const uint8_t* row[EACH];  // this thread's rows
  u32x4 held[EACH];
  int bytes;                 // of a row
  bool direct;

  template <class F>
  __device__ __forceinline__ void init(int K, bool direct_, F row_of) {
    bytes = K >> 5, direct = direct_;
#pragma unroll
    for (int i = 0; i < EACH; ++i) row[i] = row_of(min((int)threadIdx.x + THREADS * i, ROWS - 1));
  }
  // Starts group `g`; past the end of a row zeros (2^-127; the codes there are zero too).
  __device__ __forceinline__ void load(int g, uint8_t* lds) {
    const int at = g * 16;
    if (direct) {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (THREADS * i + wave * 64 < ROWS)
          __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(row[i] + at),
                                           (lds_ptr)(lds + (THREADS * i + wave * 64) * 16), 16, 0, 0);
      return;
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (at + 16 <= bytes) {
        typedef u32x4 any __attribute__((aligned(1)));
        held[i] = *reinterpret_cast<const any*>(row[i] + at);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t d = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (at + 4 * j + b < bytes) d |= (uint32_t)row[i][at + 4 * j + b] << (8 * b);
          held[i][j] = d;
        }
      }
    }
  }
  // Finishes it: ahead of the barrier that opens the group's first stage.
  __device__ __forceinline__ void store(uint8_t* lds) const {
    if (direct) return;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if ((int)threadIdx.x + THREADS * i < ROWS) *reinterpret_cast<u32x4*>(lds + (threadIdx.x + THREADS * i) * 16) = held[i];
  }
};

}  // namespace mx
