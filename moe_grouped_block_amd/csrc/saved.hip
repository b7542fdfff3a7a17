// Rows kept in 8 bits: BF16 or fp32 to MX codes with E8M0 scales, and back.
//
// Both directions are one pass bound by HBM.  Rows are dense and a block of 32
// never leaves its row, so the tensor is one long row of blocks: a lane holds
// 16 values of it whatever the width, a wave 1024.
#include "mx_rows.h"

namespace moegg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

template <int KIND, bool F32>
__global__ __launch_bounds__(256) void quantise_kernel(const void* x, uint8_t* codes, uint8_t* scales, bool kplanes, int64_t rows,
                                                       int width) {
  const int64_t n = rows * width;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kSavedChunk + threadIdx.x * 16;
  const bool in = i < n;
  v4u q{};
  uint32_t word;
  if constexpr (F32) {
    float f[16] = {};
    if (in) {
      const v4f* const p = reinterpret_cast<const v4f*>(static_cast<const float*>(x) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f v = p[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * j + e] = v[e];
      }
    }
    word = mx_from_f32<KIND>(f, q);
  } else {
    v4u u0{}, u1{};
    if (in) {
      const v4u* const p = reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(x) + i);
      u0 = p[0];
      u1 = p[1];
    }
    word = mx_from_bf16<KIND>(u0, u1, q);
  }
  if (!in) return;
  *reinterpret_cast<v4u*>(codes + i) = q;
  const int lane = threadIdx.x & 63;
  if (kplanes) {                               // (128 columns of a row in 8 lanes)
    if ((lane & 7) == 0) {
      const int64_t r = i / width;
      reinterpret_cast<uint32_t*>(scales)[(i - r * width) / 128 * rows + r] = word;
    }
  } else if ((i & ~int64_t{127}) + 128 <= n) {
    if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(scales)[i >> 7] = word;
  } else if ((lane & 1) == 0) {                // the last blocks, no whole word of scales
    scales[i >> 5] = static_cast<uint8_t>(word >> (8 * ((lane >> 1) & 3)));
  }
}

template <int KIND, bool F32>
__global__ __launch_bounds__(256) void dequantise_kernel(SavedRows s, void* out, int64_t rows, int width) {
  dequantise_chunk<KIND, F32>(s, out, rows, width, blockIdx.x);
}

unsigned blocks_of(int64_t rows, int width) { return static_cast<unsigned>((rows * width + kSavedChunk - 1) / kSavedChunk); }

}  // namespace

hipError_t launch_quantise(const void* x, bool x_f32, uint8_t* codes, uint8_t* scales, int kind, bool kplanes, int64_t rows,
                           int32_t width, hipStream_t s) {
  const dim3 grid(blocks_of(rows, width)), block(256);
  if (kind == ROW_E4M3) {
    if (x_f32) hipLaunchKernelGGL((quantise_kernel<ROW_E4M3, true>), grid, block, 0, s, x, codes, scales, kplanes, rows, width);
    else hipLaunchKernelGGL((quantise_kernel<ROW_E4M3, false>), grid, block, 0, s, x, codes, scales, kplanes, rows, width);
  } else {
    if (x_f32) hipLaunchKernelGGL((quantise_kernel<ROW_E5M2, true>), grid, block, 0, s, x, codes, scales, kplanes, rows, width);
    else hipLaunchKernelGGL((quantise_kernel<ROW_E5M2, false>), grid, block, 0, s, x, codes, scales, kplanes, rows, width);
  }
  return hipGetLastError();
}

hipError_t launch_dequantise(const SavedRows& q, void* out, bool out_f32, int64_t rows, int32_t width, hipStream_t s) {
  const dim3 grid(blocks_of(rows, width)), block(256);
  if (q.kind == ROW_E4M3) {
    if (out_f32) hipLaunchKernelGGL((dequantise_kernel<ROW_E4M3, true>), grid, block, 0, s, q, out, rows, width);
    else hipLaunchKernelGGL((dequantise_kernel<ROW_E4M3, false>), grid, block, 0, s, q, out, rows, width);
  } else {
    if (out_f32) hipLaunchKernelGGL((dequantise_kernel<ROW_E5M2, true>), grid, block, 0, s, q, out, rows, width);
    else hipLaunchKernelGGL((dequantise_kernel<ROW_E5M2, false>), grid, block, 0, s, q, out, rows, width);
  }
  return hipGetLastError();
}

}  // namespace moegg
