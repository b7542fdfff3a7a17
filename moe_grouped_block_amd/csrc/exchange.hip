// Tokens sorted by expert and back.
//
//   sort       a stable counting sort of the T * k slots (token t, choice j:
//              slot t k + j) by expert; expert g's rows start where the
//              padded rows of the experts before it end
//   dispatch   rows[row_of[t, j]] = x[t]: BF16, or an MX format with its E8M0
//              scales; padding rows become zero
//   combine    y[t] = residual[t] + sum_j w[t, j] rows[row_of[t, j]]
//   backward   drows[row_of[t, j]] = w[t, j] dy[t],
//              dw[t, j] = sum_h dy[t, h] rows[row_of[t, j], h]
//
// All but the sort are bound by HBM.  They go by tokens, not by rows: a
// token's data is read (and brought to the MX format) once for all its k
// rows, and a sum over its rows needs no atomics, so results do not depend
// on the order in which workgroups run.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "layer_internal.h"

namespace moegg {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------

__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t slot) {
  const int e = a.ids[slot];
  return e >= 0 && e < a.experts ? e : -1;
}

// Slots of every expert in block b's chunk.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int32_t count[kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int64_t beg = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t end = min(beg + a.chunk, a.slots);
  for (int64_t i = beg + threadIdx.x; i < end; i += kSortThreads) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.hist[blockIdx.x * a.experts + e] = count[e];
}

// Rows of block b's slots.  Wave w owns the w-th part of the chunk, so that
// (block, wave, position) runs in slot order and the sort is stable:
//   row = start of the expert + its slots in blocks before b
//         + its slots in the block's waves before w + rank inside the wave
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  constexpr int NW = kSortThreads / 64;
  __shared__ int32_t count[NW][kMaxExperts];    // a wave's slots per expert, then its next row
  __shared__ int32_t base[kMaxExperts];         // first row of the expert, then + rows of the blocks before
  __shared__ int32_t total[kMaxExperts];        // slots of the expert in all blocks
  __shared__ int32_t wsum[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.experts, nb = gridDim.x, b = blockIdx.x;
  for (int i = tid; i < NW * kMaxExperts; i += kSortThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  const int64_t beg = static_cast<int64_t>(b) * a.chunk;
  const int64_t end = min(beg + a.chunk, a.slots);
  const int64_t part = a.chunk / NW;            // a multiple of 64
  const int64_t wbeg = beg + wave * part, wend = min(wbeg + part, end);
  for (int64_t i = wbeg + lane; i < wend; i += 64) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&count[wave][e], 1);
  }
  __syncthreads();
  // per expert: its slots before this block and in all blocks
  for (int e = tid; e < E; e += kSortThreads) {
    int before = 0, all = 0;
    if (nb > 1) {
      for (int q = 0; q < nb; ++q) {
        const int h = a.hist[q * E + e];
        before += q < b ? h : 0;
        all += h;
      }
    } else {
      for (int w = 0; w < NW; ++w) all += count[w][e];
    }
    base[e] = before;
    total[e] = all;
  }
  __syncthreads();
  // padded starts: a scan over the experts, kSortThreads at a time
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    const int all = e < E ? total[e] : 0;
    const int padded = (all + a.m_aligned - 1) / a.m_aligned * a.m_aligned;
    int scan = padded;
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(scan, d);
      if (lane >= d) scan += y;
    }
    if (lane == 63) wsum[wave] = scan;
    __syncthreads();
    int add = carry;
    for (int w = 0; w < NW; ++w) {
      if (w < wave) add += wsum[w];
      carry += wsum[w];
    }
    const int finish = add + scan;              // end of expert e's rows
    if (e < E) {
      const int start = finish - padded;
      if (b == 0) a.padded_offsets[e] = finish;
      // padding rows of the experts, dealt out over the blocks
      if (e % nb == b)
        for (int64_t r = start + all; r < min(static_cast<int64_t>(finish), a.rows); ++r) {
          a.slot_of[r] = -1;
          if (a.prob) a.prob[r] = 0.0f;
        }
      int at = start + base[e];
      for (int w = 0; w < NW; ++w) {
        const int c = count[w][e];
        count[w][e] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  // rows behind the last expert
  for (int64_t r = carry + static_cast<int64_t>(b) * kSortThreads + tid; r < a.rows;
       r += static_cast<int64_t>(nb) * kSortThreads) {
    a.slot_of[r] = -1;
    if (a.prob) a.prob[r] = 0.0f;
  }
  // ranks: lanes with the same expert find each other by ballots over the
  // bits of its number
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  for (int64_t i0 = wbeg; i0 < wend; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = i < wend ? expert_of(a, i) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int q = 0; q < bits; ++q) {
      const uint64_t set = __ballot(e >= 0 && ((e >> q) & 1));
      same &= (e >> q) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (e >= 0) row = count[wave][e] + rank;
    // every lane has read its counter before one of them moves it on (the
    // LDS runs a wave's accesses in order)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (e >= 0 && rank == 0) count[wave][e] = row + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (i < wend) {
      a.row_of[i] = row;
      if (row >= 0 && row < a.rows) {
        a.slot_of[row] = static_cast<int32_t>(i);
        if (a.prob) a.prob[row] = a.weights[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two fp32 -> two bf16 (a in the low half), round to nearest even.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf2));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xF, 0xF, false));
}

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

// One wave's share of a row in an MX format: lane l holds columns 8 l + [0, 8)
// of a 512-column chunk; a block of 32 is 4 lanes, a scale word (128 columns)
// a 16-lane row.  Returns the lane's scale byte's word (all 16 lanes alike);
// codes: 8 bytes, or 4 of E2M1.
template <int KIND>
__device__ __forceinline__ uint32_t mx_codes(const float* v, v2u& codes) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);   // NaN bits are the largest
  amax = max(amax, dpp_u<0xB1>(amax));
  amax = max(amax, dpp_u<0x4E>(amax));
  uint32_t byte;
  if constexpr (KIND == ROW_E4M3) byte = mx_byte<8, 6>(amax);
  else if constexpr (KIND == ROW_E5M2) byte = mx_byte<15, 6>(amax);
  else byte = mx_byte<2, 4>(amax);
  // 2^(127 - byte), exact (2^-126 for 253, 2^-127 for 254); zero codes in a NaN block
  const float inv = byte == 255u ? 0.0f : byte == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = byte == 255u ? 0.0f : v[i] * inv;
  if constexpr (KIND == ROW_E4M3) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
    codes = v2u{static_cast<uint32_t>(a), static_cast<uint32_t>(b)};
  } else if constexpr (KIND == ROW_E5M2) {
    int a = __builtin_amdgcn_cvt_pk_bf8_f32(q[0], q[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_bf8_f32(q[2], q[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_bf8_f32(q[4], q[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_bf8_f32(q[6], q[7], b, true);
    codes = v2u{static_cast<uint32_t>(a), static_cast<uint32_t>(b)};
  } else {
    uint32_t a = 0;
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, q[0], q[1], 1.0f, 0);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, q[2], q[3], 1.0f, 1);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, q[4], q[5], 1.0f, 2);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(a, q[6], q[7], 1.0f, 3);
    codes = v2u{a, 0u};
  }
  uint32_t word = byte << (8 * ((threadIdx.x >> 2) & 3));
  word |= dpp_u<0x124>(word);       // row_ror 4
  word |= dpp_u<0x128>(word);       // row_ror 8
  return word;
}

// Store lane `lane`'s 8 columns (col .. col + 8) of a row.
template <int KIND>
__device__ __forceinline__ void store_row(const ExchangeArgs& a, int64_t row, int col, int lane, v4u bf, v2u codes,
                                          uint32_t word) {
  if constexpr (KIND == ROW_BF16) {
    *reinterpret_cast<v4u*>(a.rows_out + (row * a.width + col) * 2) = bf;
  } else {
    if constexpr (KIND == ROW_E2M1) *reinterpret_cast<uint32_t*>(a.rows_out + (row * a.width + col) / 2) = codes.x;
    else *reinterpret_cast<v2u*>(a.rows_out + row * a.width + col) = codes;
    if ((lane & 15) == 0) {
      const int64_t w = col >> 7;
      uint32_t* const s = reinterpret_cast<uint32_t*>(a.scales);
      s[a.kplanes ? w * a.rows + row : row * (a.width >> 7) + w] = word;
    }
  }
}

// Zero the padding rows among rows [64 q, 64 q + 64) (one wave).
template <int KIND>
__device__ __forceinline__ void zero_padding(const ExchangeArgs& a, int64_t q, int lane) {
  const int64_t last = a.offsets[a.experts - 1];
  const int64_t end = last < a.rows ? last : a.rows;
  const int64_t r = 64 * q + lane;
  uint64_t pad = __ballot(r < end && a.slot_of[r < a.rows ? r : 0] < 0);
  while (pad) {
    const int64_t row = 64 * q + __builtin_ctzll(pad);
    pad &= pad - 1;
    for (int col = lane * 8; col < a.width; col += 512) store_row<KIND>(a, row, col, lane, v4u{}, v2u{}, 0u);
  }
}

// Row of slot s, or -1.
__device__ __forceinline__ int64_t row_at(const ExchangeArgs& a, int64_t s) {
  const int64_t r = a.row_of[s];
  return r >= 0 && r < a.rows ? r : -1;
}

// dispatch: one wave for 512 columns of a token; the waves behind them zero
// the padding.
template <int KIND>
__global__ __launch_bounds__(256) void dispatch_kernel(ExchangeArgs a, int64_t token_waves) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (wave >= token_waves) {
    const int64_t q = wave - token_waves;
    if (64 * q < a.rows) zero_padding<KIND>(a, q, lane);
    return;
  }
  const int chunks = (a.width + 511) / 512;
  const int64_t t = wave / chunks;
  const int col = static_cast<int>(wave - t * chunks) * 512 + lane * 8;
  const bool in = col < a.width;
  v4u u{};
  if (in) u = *reinterpret_cast<const v4u*>(a.x + t * a.width + col);
  v2u codes{};
  uint32_t word = 0;
  if constexpr (KIND != ROW_BF16) {
    const float v[8] = {lo(u.x), hi(u.x), lo(u.y), hi(u.y), lo(u.z), hi(u.z), lo(u.w), hi(u.w)};
    word = mx_codes<KIND>(v, codes);
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t row = row_at(a, t * a.top_k + j);
    if (row >= 0 && in) store_row<KIND>(a, row, col, lane, u, codes, word);
  }
}

// combine: one wave for 512 columns of a token.
__global__ __launch_bounds__(256) void combine_kernel(ExchangeArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int chunks = (a.width + 511) / 512;
  const int64_t t = wave / chunks;
  const int col = static_cast<int>(wave - t * chunks) * 512 + lane * 8;
  if (t >= a.tokens || col >= a.width) return;
  float v[8] = {};
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t row = row_at(a, t * a.top_k + j);
    if (row < 0) continue;
    const float w = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
    const v4u u = *reinterpret_cast<const v4u*>(a.rows_in + row * a.width + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = fmaf(w, lo(u[i]), v[2 * i]);
      v[2 * i + 1] = fmaf(w, hi(u[i]), v[2 * i + 1]);
    }
  }
  if (a.residual) {
    const v4u u = *reinterpret_cast<const v4u*>(a.residual + t * a.width + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] += lo(u[i]);
      v[2 * i + 1] += hi(u[i]);
    }
  }
  *reinterpret_cast<v4u*>(a.y + t * a.width + col) =
      v4u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// backward of combine: one wave for a token (the dot products run over the
// whole row); the waves behind them zero the padding of drows.
template <int KIND>
__global__ __launch_bounds__(256) void combine_backward_kernel(ExchangeArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (wave >= a.tokens) {
    const int64_t q = wave - a.tokens;
    if (64 * q < a.rows) zero_padding<KIND>(a, q, lane);
    return;
  }
  const int64_t t = wave;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t slot = t * a.top_k + j, row = row_at(a, slot);
    const float w = a.weights ? a.weights[slot] : 1.0f;
    float dot = 0.0f;
    if (row >= 0) {
      for (int c0 = 0; c0 < a.width; c0 += 512) {
        const int col = c0 + lane * 8;
        const bool in = col < a.width;
        v4u u{}, r{};
        if (in) u = *reinterpret_cast<const v4u*>(a.x + t * a.width + col);
        if (in && a.dweights) r = *reinterpret_cast<const v4u*>(a.rows_in + row * a.width + col);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot = fmaf(lo(u[i]), lo(r[i]), dot);
          dot = fmaf(hi(u[i]), hi(r[i]), dot);
          v[2 * i] = w * lo(u[i]);
          v[2 * i + 1] = w * hi(u[i]);
        }
        v2u codes{};
        uint32_t word = 0;
        v4u bf{};
        if constexpr (KIND == ROW_BF16)
          bf = v4u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
        else
          word = mx_codes<KIND>(v, codes);
        if (in) store_row<KIND>(a, row, col, lane, bf, codes, word);
      }
    }
    if (a.dweights) {
      dot = wave_sum(dot);
      if (lane == 0) a.dweights[slot] = dot;
    }
  }
}

__global__ __launch_bounds__(256) void unsort_kernel(const float* rows, const int32_t* row_of, float* values,
                                                     int64_t slots, int64_t n_rows) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= slots) return;
  const int64_t r = row_of[i];
  values[i] = r >= 0 && r < n_rows ? rows[r] : 0.0f;
}

template <typename F>
hipError_t by_kind(int kind, F&& f) {
  switch (kind) {
    case ROW_BF16: return f(std::integral_constant<int, ROW_BF16>{});
    case ROW_E4M3: return f(std::integral_constant<int, ROW_E4M3>{});
    case ROW_E5M2: return f(std::integral_constant<int, ROW_E5M2>{});
    case ROW_E2M1: return f(std::integral_constant<int, ROW_E2M1>{});
    default: return hipErrorInvalidValue;
  }
}

// Workgroups of 4 waves for `waves` waves; 0 if there are too many.
unsigned blocks_of(int64_t waves) {
  const int64_t b = (waves + 3) / 4;
  return b > 0x7FFFFFFF ? 0u : static_cast<unsigned>(b);
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, hipStream_t s) {
  if (a.blocks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sort_place_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const ExchangeArgs& a, hipStream_t s) {
  const int64_t token_waves = a.tokens * ((a.width + 511) / 512);
  const unsigned blocks = blocks_of(token_waves + (a.rows + 63) / 64);
  if (!blocks) return hipErrorInvalidValue;
  return by_kind(a.kind, [&](auto c) {
    hipLaunchKernelGGL((dispatch_kernel<decltype(c)::value>), dim3(blocks), dim3(256), 0, s, a, token_waves);
    return hipGetLastError();
  });
}

hipError_t launch_combine(const ExchangeArgs& a, hipStream_t s) {
  const unsigned blocks = blocks_of(a.tokens * ((a.width + 511) / 512));
  if (!blocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL(combine_kernel, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t s) {
  const unsigned blocks = blocks_of(a.tokens + (a.rows + 63) / 64);
  if (!blocks) return hipErrorInvalidValue;
  return by_kind(a.kind, [&](auto c) {
    hipLaunchKernelGGL((combine_backward_kernel<decltype(c)::value>), dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_unsort(const float* rows, const int32_t* row_of, float* values, int64_t slots, int64_t n_rows,
                         hipStream_t s) {
  const int64_t b = (slots + 255) / 256;
  if (b > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(unsort_kernel, dim3(static_cast<unsigned>(b)), dim3(256), 0, s, rows, row_of, values, slots, n_rows);
  return hipGetLastError();
}

}  // namespace moegg
