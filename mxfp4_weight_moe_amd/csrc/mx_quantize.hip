// Rows of bf16 or fp32 to MXFP8 or MXFP4, optionally with the values that the codes stand for.
#include "mx_quant.hpp"
#include "mx_internal.hpp"

namespace mx {

// A thread takes 8 values: blocks of 32 are whole quads of lanes wherever rows begin, since a row is
// a multiple of 32.  Bound by memory: 16384 x 7168 from bf16 to MXFP4 with the values, 536 MB, in 88 us, 6.1 TB/s;
// 4 x 7168 to MXFP8 in 2.2 us.
template <int FMT, bool F32, bool VALUES>
__global__ void __launch_bounds__(256) quantize_kernel(const void* __restrict__ x, int64_t pieces,
                                                       uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                       uint16_t* __restrict__ values) {
  const int64_t p = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  if (p >= pieces) return;  // pieces % 4 == 0: a block's four lanes are all in or all out
  float v[8];
  if constexpr (F32) {
    const float* f = static_cast<const float*>(x) + p * 8;
    const u32x4 a = ld16(f), b = ld16(f + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
  } else {
    const u32x4 a = ld16(static_cast<const uint16_t*>(x) + p * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
  uint32_t c[FMT / 4], byte;
  quantize8<FMT>(v, c, byte);
  store_codes8<FMT>(codes, scales, (size_t)p, c, byte);
  if constexpr (VALUES) *reinterpret_cast<u32x4*>(values + p * 8) = code_values8<FMT>(c, byte);
}

template <int FMT, bool F32>
static void quantize(const void* x, int64_t pieces, uint8_t* codes, uint8_t* scales, uint16_t* values,
                     hipStream_t stream) {
  // a launch takes fewer than 2^32 threads along x
  const int64_t groups = (pieces + 255) / 256, x_groups = std::min<int64_t>(groups, 1 << 22);
  const dim3 grid((unsigned)x_groups, (unsigned)((groups + x_groups - 1) / x_groups));
  if (values)
    hipLaunchKernelGGL((quantize_kernel<FMT, F32, true>), grid, dim3(256), 0, stream, x, pieces, codes, scales, values);
  else
    hipLaunchKernelGGL((quantize_kernel<FMT, F32, false>), grid, dim3(256), 0, stream, x, pieces, codes, scales, values);
}

int launch_quantize(const void* x, bool f32, int format, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales,
                    uint16_t* values, hipStream_t stream) {
  const int64_t pieces = rows * (K / 8);
  if (format == MX_FORMAT_MXFP8)
    f32 ? quantize<8, true>(x, pieces, codes, scales, values, stream)
        : quantize<8, false>(x, pieces, codes, scales, values, stream);
  else
    f32 ? quantize<4, true>(x, pieces, codes, scales, values, stream)
        : quantize<4, false>(x, pieces, codes, scales, values, stream);
  return hip_status(hipGetLastError());
}

}  // namespace mx
