// MX rows: 8- or 4-bit codes in blocks of 32 with an E8M0 scale byte each, from
// BF16 or fp32 and (8 bits) back.
#pragma once

#include "lanes.h"
#include "layer_internal.h"

namespace moegg {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// E8M0 byte of the smallest power of two s with amax <= s q_max, q_max =
// (1 + M / 8) 2^EMAX, read off the bits of amax (fp32, >= 0), so that no
// rounding decides it; 0 for a block of zeros, 255 (NaN) for one that holds a
// NaN or an infinity.
template <int EMAX, uint32_t M>
__device__ __forceinline__ uint32_t mx_byte(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  if (e == 255) return 255u;
  const int byte = e - EMAX + ((amax & 0x7FFFFFu) > (M << 20) ? 1 : 0);
  return static_cast<uint32_t>(byte < 0 ? 0 : byte);
}

// Scale byte of a block whose largest magnitude has the fp32 bits amax.
template <int KIND>
__device__ __forceinline__ uint32_t mx_block_byte(uint32_t amax) {
  if constexpr (KIND == ROW_E4M3) return mx_byte<8, 6>(amax);
  else if constexpr (KIND == ROW_E5M2) return mx_byte<15, 6>(amax);
  else return mx_byte<2, 4>(amax);
}

// MX rows: lane l holds columns 16 l + [0, 16) of a 1024-column chunk; a block
// of 32 is 2 lanes, a scale word (128 columns) 8.

// A block's amax (fp32 bits) in its lanes -> its scale byte; the scale word of
// the lane's 128 columns (all 8 lanes alike).
template <int KIND>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax, uint32_t& word) {
  amax = max(amax, dpp_u<0xB1>(amax));
  const uint32_t byte = mx_block_byte<KIND>(amax);
  word = byte << (8 * ((threadIdx.x >> 1) & 3));
  word |= dpp_u<0x4E>(word);        // lanes 2 apart: two bytes
  word |= dpp_u<0x141>(word);       // mirrored halves of 8: all four
  return byte;
}

// The scaled conversions divide by the power of two given as fp32 (2^-127 is
// its subnormal) and round to nearest even.
typedef short v2s __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float mx_factor(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// 16 bf16 (two 16-byte pieces) -> codes: 16 bytes, or 8 of E2M1; zeros in a
// block that holds a NaN or an infinity.
template <int KIND>
__device__ __forceinline__ uint32_t mx_from_bf16(v4u a, v4u b, v4u& codes) {
  typedef uint16_t v2h __attribute__((ext_vector_type(2)));
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  v2h m = __builtin_bit_cast(v2h, u[0] & 0x7FFF7FFFu);       // magnitudes; NaN bits are the largest
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2h, u[i] & 0x7FFF7FFFu));
  uint32_t word;
  const uint32_t byte = mx_scale<KIND>(static_cast<uint32_t>(max(m.x, m.y)) << 16, word);
  const float f = mx_factor(byte);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2b x = __builtin_bit_cast(v2b, u[2 * i]), y = __builtin_bit_cast(v2b, u[2 * i + 1]);
    if constexpr (KIND == ROW_E4M3) {
      v2s c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v2s{0, 0}, x, f, false);
      w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, y, f, true));
    } else if constexpr (KIND == ROW_E5M2) {
      v2s c = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(v2s{0, 0}, x, f, false);
      w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(c, y, f, true));
    } else if (i & 1) {
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i / 2], x, f, 2);
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i / 2], y, f, 3);
    } else {
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i / 2], x, f, 0);
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i / 2], y, f, 1);
    }
  }
  const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;
  codes = v4u{w[0] & keep, w[1] & keep, w[2] & keep, w[3] & keep};
  return word;
}

// The same from 16 fp32.
template <int KIND>
__device__ __forceinline__ uint32_t mx_from_f32(const float* v, v4u& codes) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  uint32_t word;
  const uint32_t byte = mx_scale<KIND>(amax, word);
  const float f = mx_factor(byte);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* const q = v + 4 * i;
    if constexpr (KIND == ROW_E4M3) {
      v2s c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2s{0, 0}, q[0], q[1], f, false);
      w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, q[2], q[3], f, true));
    } else if constexpr (KIND == ROW_E5M2) {
      v2s c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(v2s{0, 0}, q[0], q[1], f, false);
      w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, q[2], q[3], f, true));
    } else if (i & 1) {
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i / 2], q[0], q[1], f, 2);
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i / 2], q[2], q[3], f, 3);
    } else {
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i / 2], q[0], q[1], f, 0);
      w[i / 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i / 2], q[2], q[3], f, 1);
    }
  }
  const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;
  codes = v4u{w[0] & keep, w[1] & keep, w[2] & keep, w[3] & keep};
  return word;
}

// Four fp32 of a block with the scale factor f -> four codes of 8 bits.
template <int KIND>
__device__ __forceinline__ uint32_t mx_codes(const float* v, float f) {
  if constexpr (KIND == ROW_E4M3) {
    const v2s c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2s{0, 0}, v[0], v[1], f, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[2], v[3], f, true));
  } else {
    const v2s c = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(v2s{0, 0}, v[0], v[1], f, false);
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(c, v[2], v[3], f, true));
  }
}

// U fp32 a lane (4 or 8), a block of 32 in 32 / U neighbouring lanes: the codes
// (4 of 8 bits or 8 of 4 a word; 4 of 4 bits in the low half) and the scale word
// of the 128 columns in 128 / U lanes (all of them alike).
template <int KIND, int U>
__device__ __forceinline__ void mx_unit(const float* v, uint32_t* codes, uint32_t& word) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  amax = max(amax, dpp_u<0xB1>(amax));
  amax = max(amax, dpp_u<0x4E>(amax));
  if constexpr (U == 4) amax = max(amax, dpp_u<0x141>(amax));
  const uint32_t byte = mx_block_byte<KIND>(amax), keep = byte == 255u ? 0u : 0xFFFFFFFFu;
  const float f = mx_factor(byte);
  if constexpr (KIND == ROW_E2M1) {
    codes[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], f, 0);
    codes[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], v[2], v[3], f, 1);
    if constexpr (U == 8) {
      codes[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], v[4], v[5], f, 2);
      codes[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes[0], v[6], v[7], f, 3);
    }
    codes[0] &= keep;
  } else {
#pragma unroll
    for (int i = 0; i < U / 4; ++i) codes[i] = mx_codes<KIND>(v + 4 * i, f) & keep;
  }
  word = byte << (8 * ((threadIdx.x / (32 / U)) & 3));
  if constexpr (U == 8) word |= partner<2>(word);        // the other block of 8 lanes
  word |= partner<3>(word);                              // the other 8 of 16 lanes
  if constexpr (U == 4) word |= partner<4>(word);        // the other 16 of 32
}

// ---- back ------------------------------------------------------------------

// What a scale byte stands for: NaN for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return byte == 255u ? __builtin_nanf("") : mx_factor(byte);
}

// Place of the scale byte of 32-column block b of row r.
__device__ __forceinline__ int64_t scale_at(const SavedRows& s, int64_t rows, int32_t width, int64_t r, int b) {
  return s.kplanes ? ((b >> 2) * rows + r) * 4 + (b & 3) : r * (width >> 5) + b;
}

// Four codes -> what they stand for under the scale f.
template <int KIND>
__device__ __forceinline__ void mx_four(uint32_t codes, float f, float* v) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  f2 a, b;
  if constexpr (KIND == ROW_E4M3) {
    a = __builtin_amdgcn_cvt_pk_f32_fp8(codes, false);
    b = __builtin_amdgcn_cvt_pk_f32_fp8(codes, true);
  } else {
    a = __builtin_amdgcn_cvt_pk_f32_bf8(codes, false);
    b = __builtin_amdgcn_cvt_pk_f32_bf8(codes, true);
  }
  v[0] = a.x * f;
  v[1] = a.y * f;
  v[2] = b.x * f;
  v[3] = b.y * f;
}

// Four codes -> what they stand for in BF16, rounded to nearest even (the
// conversion unit multiplies by the power of two; a NaN scale gives NaN).
template <int KIND>
__device__ __forceinline__ v2u mx_four_bf16(uint32_t codes, float f) {
  if constexpr (KIND == ROW_E4M3)
    return v2u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, f, true))};
  else
    return v2u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, f, true))};
}

// Elements of a workgroup of 4 waves that brings rows to 8 bits or back.
constexpr int kSavedChunk = 4096;

// Chunk number `chunk` of the rows, back to BF16 or fp32: 16 values a thread.
template <int KIND, bool F32>
__device__ __forceinline__ void dequantise_chunk(const SavedRows& s, void* out, int64_t rows, int width, int64_t chunk) {
  const int64_t i = chunk * kSavedChunk + threadIdx.x * 16;
  if (i >= rows * width) return;
  const v4u q = *reinterpret_cast<const v4u*>(s.codes + i);
  int64_t at = i >> 5;
  if (s.kplanes) {
    const int64_t r = i / width;
    at = scale_at(s, rows, width, r, static_cast<int>(i - r * width) >> 5);
  }
  const float f = mx_scale_value(s.scales[at]);
  if constexpr (F32) {
    typedef float v4f __attribute__((ext_vector_type(4)));
    v4f* const p = reinterpret_cast<v4f*>(static_cast<float*>(out) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
      mx_four<KIND>(q[j], f, v);
      p[j] = v4f{v[0], v[1], v[2], v[3]};
    }
  } else {
    v4u* const p = reinterpret_cast<v4u*>(static_cast<uint16_t*>(out) + i);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const v2u lo = mx_four_bf16<KIND>(q[2 * j], f), hi = mx_four_bf16<KIND>(q[2 * j + 1], f);
      p[j] = v4u{lo.x, lo.y, hi.x, hi.y};
    }
  }
}

}  // namespace
}  // namespace moegg
