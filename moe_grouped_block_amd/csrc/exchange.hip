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
// Every block sums the counts of all blocks itself (they are small and in
// L2), all threads at once: no block waits for another.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  constexpr int NW = kSortThreads / 64;
  __shared__ int32_t count[NW][kMaxExperts];    // a wave's slots per expert, then its next row
  __shared__ int32_t base[kMaxExperts];         // slots of the expert in the blocks before
  __shared__ int32_t total[kMaxExperts];        // slots of the expert in all blocks
  __shared__ int32_t finish[kMaxExperts];       // end of the expert's padded rows
  __shared__ int32_t wsum[NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.experts, nb = gridDim.x, b = blockIdx.x;
  for (int e = tid; e < E; e += kSortThreads) {
    base[e] = 0;
    total[e] = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) count[w][e] = 0;
  }
  __syncthreads();
  const int64_t beg = static_cast<int64_t>(b) * a.chunk;
  const int64_t end = min(beg + a.chunk, a.slots);
  const int64_t part = a.chunk / NW;            // a multiple of 64
  const int64_t wbeg = beg + wave * part, wend = min(wbeg + part, end);
  for (int64_t i = wbeg + lane; i < wend; i += 64) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&count[wave][e], 1);
  }
  if (nb > 1) {
    // threads = (group of blocks, expert); sums of whole numbers, so their
    // order does not matter
    const int lanes = E < kSortThreads ? E : kSortThreads, groups = kSortThreads / lanes;
    const int q0 = tid / lanes, e0 = tid % lanes;
    if (q0 < groups)
      for (int e = e0; e < E; e += lanes) {
        int before = 0, all = 0;
#pragma unroll 8
        for (int q = q0; q < nb; q += groups) {
          const int h = a.hist[q * E + e];
          before += q < b ? h : 0;
          all += h;
        }
        atomicAdd(&base[e], before);
        atomicAdd(&total[e], all);
      }
    __syncthreads();
  } else {
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) {
      int all = 0;
      for (int w = 0; w < NW; ++w) all += count[w][e];
      total[e] = all;
    }
    __syncthreads();
  }
  // padded starts: a scan over the experts, kSortThreads at a time
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    const int all = e < E ? total[e] : 0;
    // (without a sign: the sum before the division may reach 2^31)
    const uint32_t ma = a.m_aligned;
    const int padded = static_cast<int>((all + ma - 1u) / ma * ma);
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
    if (e < E) {
      finish[e] = add + scan;
      if (b == 0) a.padded_offsets[e] = add + scan;
      int at = add + scan - padded + base[e];
      total[e] += add + scan - padded;          // first padding row
      for (int w = 0; w < NW; ++w) {
        const int c = count[w][e];
        count[w][e] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  // padding rows of the experts, dealt out over the blocks, and rows behind
  // the last expert (rows are counted in 64 bits: a thread's first may pass 2^31)
  for (int e = b; e < E; e += nb)
    for (int64_t r = static_cast<int64_t>(total[e]) + tid; r < min(static_cast<int64_t>(finish[e]), a.rows); r += kSortThreads) {
      a.slot_of[r] = -1;
      if (a.prob) a.prob[r] = 0.0f;
    }
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

// MX rows: lane l holds columns 16 l + [0, 16) of a 1024-column chunk; a block
// of 32 is 2 lanes, a scale word (128 columns) 8.

// A block's amax (fp32 bits) in its lanes -> its scale byte; the scale word of
// the lane's 128 columns (all 8 lanes alike).
template <int KIND>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax, uint32_t& word) {
  amax = max(amax, dpp_u<0xB1>(amax));
  uint32_t byte;
  if constexpr (KIND == ROW_E4M3) byte = mx_byte<8, 6>(amax);
  else if constexpr (KIND == ROW_E5M2) byte = mx_byte<15, 6>(amax);
  else byte = mx_byte<2, 4>(amax);
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

// Columns of a row that a wave holds at a time, and a lane's part of them.
template <int KIND>
constexpr int kLaneCols = KIND == ROW_BF16 ? 8 : 16;

// A lane's columns of a row (from col on): BF16 bits in q, or codes in q and
// the scale word.
template <int KIND>
__device__ __forceinline__ void store_row(const ExchangeArgs& a, int64_t row, int col, int lane, v4u q, uint32_t word) {
  if constexpr (KIND == ROW_BF16) {
    *reinterpret_cast<v4u*>(a.rows_out + (row * a.width + col) * 2) = q;
  } else {
    if constexpr (KIND == ROW_E2M1) *reinterpret_cast<v2u*>(a.rows_out + (row * a.width + col) / 2) = v2u{q.x, q.y};
    else *reinterpret_cast<v4u*>(a.rows_out + row * a.width + col) = q;
    if ((lane & 7) == 0) {
      const int64_t w = col >> 7;
      uint32_t* const s = reinterpret_cast<uint32_t*>(a.scales);
      s[a.kplanes ? w * a.rows + row : row * (a.width >> 7) + w] = word;
    }
  }
}

// Zero the padding rows among rows [kPadRows q, kPadRows (q + 1)) (one wave).
// These waves come first in a launch and take few rows each: with 64 rows a
// wave, behind the tokens' waves, the last of them ended 10 us after all
// others.
template <int KIND>
__device__ __forceinline__ void zero_padding(const ExchangeArgs& a, int64_t q, int lane) {
  const int64_t last = a.offsets[a.experts - 1];
  const int64_t end = last < a.rows ? last : a.rows;
  const int64_t r = kPadRows * q + lane;
  uint64_t pad = __ballot(lane < kPadRows && r < end && a.slot_of[r < end ? r : 0] < 0);
  while (pad) {
    const int64_t row = kPadRows * q + __builtin_ctzll(pad);
    pad &= pad - 1;
    for (int col = lane * kLaneCols<KIND>; col < a.width; col += 64 * kLaneCols<KIND>)
      store_row<KIND>(a, row, col, lane, v4u{}, 0u);
  }
}

// This wave's number among the launch's waves of 4 a workgroup, in scalar
// registers: what is the same for a wave (its token's rows and weights) then
// comes by scalar loads.
__device__ __forceinline__ int64_t wave_number() {
  return static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// Row of slot s, or -1.
__device__ __forceinline__ int64_t row_at(const ExchangeArgs& a, int64_t s) {
  const int64_t r = a.row_of[s];
  return r >= 0 && r < a.rows ? r : -1;
}

__device__ __forceinline__ void unpack(v4u u, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = lo(u[i]);
    v[2 * i + 1] = hi(u[i]);
  }
}

// dispatch: one wave for 512 columns of a token (1024 of an MX row), read
// and brought to the rows' format once.
template <int KIND>
__global__ __launch_bounds__(256) void dispatch_kernel(ExchangeArgs a, int64_t pad_waves) {
  constexpr int C = kLaneCols<KIND>;
  const int lane = threadIdx.x & 63;
  int64_t wave = wave_number();
  if (wave < pad_waves) {
    zero_padding<KIND>(a, wave, lane);
    return;
  }
  wave -= pad_waves;
  const int chunks = (a.width + 64 * C - 1) / (64 * C);
  const int64_t t = wave / chunks;
  if (t >= a.tokens) return;
  const int col = static_cast<int>(wave - t * chunks) * 64 * C + lane * C;
  const bool in = col < a.width;
  v4u u{};
  uint32_t word = 0;
  const v4u* const src = reinterpret_cast<const v4u*>(a.x + t * a.width + col);
  if (in) u = src[0];
  if constexpr (KIND != ROW_BF16) {
    v4u u1{};
    if (in) u1 = src[1];
    word = mx_from_bf16<KIND>(u, u1, u);
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t row = row_at(a, t * a.top_k + j);
    if (row >= 0 && in) store_row<KIND>(a, row, col, lane, u, word);
  }
}

// combine: one wave for 512 columns of a token, the gathers of eight rows in
// flight at once.
__global__ __launch_bounds__(256) void combine_kernel(ExchangeArgs a) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 63;
  const int64_t wave = wave_number();
  const int chunks = (a.width + 511) / 512;
  const int64_t t = wave / chunks;
  const int col = static_cast<int>(wave - t * chunks) * 512 + lane * 8;
  if (t >= a.tokens || col >= a.width) return;
  v4u res{};
  if (a.residual) res = *reinterpret_cast<const v4u*>(a.residual + t * a.width + col);
  float v[8] = {};
  for (int j0 = 0; j0 < a.top_k; j0 += U) {
    v4u u[U];
    float w[U];
    bool there[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = min(j0 + i, a.top_k - 1);
      const int64_t row = row_at(a, t * a.top_k + j);
      there[i] = row >= 0 && j0 + i < a.top_k;
      w[i] = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
      u[i] = v4u{};
      if (there[i]) u[i] = *reinterpret_cast<const v4u*>(a.rows_in + row * a.width + col);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (there[i]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[2 * q] = fmaf(w[i], lo(u[i][q]), v[2 * q]);
          v[2 * q + 1] = fmaf(w[i], hi(u[i][q]), v[2 * q + 1]);
        }
      }
  }
  if (a.residual) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] += lo(res[q]);
      v[2 * q + 1] += hi(res[q]);
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
// whole row), kSame rows of it at once, so that dy is read once for them.
template <int KIND>
__global__ __launch_bounds__(256) void combine_backward_kernel(ExchangeArgs a, int64_t pad_waves) {
  constexpr int C = kLaneCols<KIND>, kSame = KIND == ROW_BF16 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t wave = wave_number();
  if (wave < pad_waves) {
    zero_padding<KIND>(a, wave, lane);
    return;
  }
  const int64_t t = wave - pad_waves;
  if (t >= a.tokens) return;
  for (int j0 = 0; j0 < a.top_k; j0 += kSame) {
    int64_t row[kSame];
    float w[kSame], dot[kSame];
#pragma unroll
    for (int i = 0; i < kSame; ++i) {
      const int64_t slot = t * a.top_k + min(j0 + i, a.top_k - 1);
      row[i] = j0 + i < a.top_k ? row_at(a, slot) : -1;
      w[i] = a.weights ? a.weights[slot] : 1.0f;
      dot[i] = 0.0f;
    }
    for (int c0 = 0; c0 < a.width; c0 += 64 * C) {
      const int col = c0 + lane * C;
      const bool in = col < a.width;
      v4u d[C / 8], r[kSame][C / 8];
#pragma unroll
      for (int h = 0; h < C / 8; ++h) {
        d[h] = v4u{};
        if (in) d[h] = reinterpret_cast<const v4u*>(a.x + t * a.width + col)[h];
#pragma unroll
        for (int i = 0; i < kSame; ++i) {
          r[i][h] = v4u{};
          if (in && a.dweights && row[i] >= 0) r[i][h] = reinterpret_cast<const v4u*>(a.rows_in + row[i] * a.width + col)[h];
        }
      }
      float dv[C];
#pragma unroll
      for (int h = 0; h < C / 8; ++h) unpack(d[h], dv + 8 * h);
#pragma unroll
      for (int i = 0; i < kSame; ++i) {
        if (row[i] < 0) continue;
        float v[C];
#pragma unroll
        for (int h = 0; h < C / 8; ++h) unpack(r[i][h], v + 8 * h);
#pragma unroll
        for (int e = 0; e < C; ++e) {
          dot[i] = fmaf(dv[e], v[e], dot[i]);
          v[e] = w[i] * dv[e];
        }
        v4u q{};
        uint32_t word = 0;
        if constexpr (KIND == ROW_BF16)
          q = v4u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
        else
          word = mx_from_f32<KIND>(v, q);
        if (in) store_row<KIND>(a, row[i], col, lane, q, word);
      }
    }
    if (a.dweights) {
#pragma unroll
      for (int i = 0; i < kSame; ++i) {
        const float s = wave_sum(dot[i]);
        if (lane == 0 && j0 + i < a.top_k) a.dweights[t * a.top_k + j0 + i] = row[i] >= 0 ? s : 0.0f;
      }
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

// Workgroups of 4 waves for `waves` waves (the host has checked exchange_waves()).
unsigned blocks_of(int64_t waves) { return static_cast<unsigned>((waves + 3) / 4); }

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
  const int cols = a.kind == ROW_BF16 ? 512 : 1024;
  const int64_t token_waves = a.tokens * ((a.width + cols - 1) / cols);
  const int64_t pad_waves = (a.rows + kPadRows - 1) / kPadRows;
  const unsigned blocks = blocks_of(token_waves + pad_waves);
  return by_kind(a.kind, [&](auto c) {
    hipLaunchKernelGGL((dispatch_kernel<decltype(c)::value>), dim3(blocks), dim3(256), 0, s, a, pad_waves);
    return hipGetLastError();
  });
}

hipError_t launch_combine(const ExchangeArgs& a, hipStream_t s) {
  const unsigned blocks = blocks_of(a.tokens * ((a.width + 511) / 512));
  hipLaunchKernelGGL(combine_kernel, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t s) {
  const int64_t pad_waves = (a.rows + kPadRows - 1) / kPadRows;
  const unsigned blocks = blocks_of(a.tokens + pad_waves);
  return by_kind(a.kind, [&](auto c) {
    hipLaunchKernelGGL((combine_backward_kernel<decltype(c)::value>), dim3(blocks), dim3(256), 0, s, a, pad_waves);
    return hipGetLastError();
  });
}

hipError_t launch_unsort(const float* rows, const int32_t* row_of, float* values, int64_t slots, int64_t n_rows,
                         hipStream_t s) {
  const int64_t b = (slots + 255) / 256;
  hipLaunchKernelGGL(unsort_kernel, dim3(static_cast<unsigned>(b)), dim3(256), 0, s, rows, row_of, values, slots, n_rows);
  return hipGetLastError();
}

}  // namespace moegg
