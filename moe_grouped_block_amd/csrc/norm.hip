// Root-mean-square norm with the residual's addition, and its gradient.
//
//   h  = x + residual, rounded once to the stream's type; the norm goes on with
//        the rounded h, so that the gradient taken from the stored h is the one
//        of what was computed
//   r  = 1 / sqrt(mean(h^2) + eps),  y = (h r) w
//
//   g  = dy w,  xh = h r
//   dx = r (g - xh mean(g xh)) + dh       (of x and of the residual alike)
//   dw = sum over rows of dy xh
//
// Both are bound by HBM: every value is read once and stays in registers until
// its row's sums are known.  A row belongs to one wave (up to 1024 columns), to a
// part of one, or to several of a workgroup, whose sums meet in LDS.
//
// Squares and products are summed in 64 bits: no h in range overflows or
// vanishes in them, and the rate of 64-bit operations is far from being needed.
// r is kept as a power of two a and a factor b in [0.5, 1]: (h a) b does not
// leave the range of fp32 where the result does not.
#include "mx_rows.h"

namespace moegg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf2));
}
// U values of a BF16 or fp32 tensor from element i (a multiple of U) on: 8 or 16
// bytes of BF16, 16 or 32 of fp32.
template <bool F32, int U>
struct Unit {
  static constexpr int W = U * (F32 ? 4 : 2) / 4;        // words
  typedef uint32_t vec __attribute__((ext_vector_type(W > 4 ? 4 : W)));
  static constexpr int N = W > 4 ? W / 4 : 1;
  vec u[N];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const vec* const p = reinterpret_cast<const vec*>(static_cast<const uint8_t*>(base) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int q = 0; q < N; ++q) u[q] = p[q];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < N; ++q) u[q] = vec{};
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t x = u[i >> 2][i & 3];
      if constexpr (F32) {
        f[i] = __uint_as_float(x);
      } else {
        f[2 * i] = __uint_as_float(x << 16);
        f[2 * i + 1] = __uint_as_float(x & 0xFFFF0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (F32) u[i >> 2][i & 3] = __float_as_uint(f[i]);
      else u[i >> 2][i & 3] = bf16x2(f[2 * i], f[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t i) const {
    vec* const p = reinterpret_cast<vec*>(static_cast<uint8_t*>(base) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int q = 0; q < N; ++q) p[q] = u[q];
  }
};

// 1 / sqrt(v) = a b for v > 0 (NaN: b is NaN; +inf: b is 0): a a power of two, b in [0.5, 1].
// b is what the unit gives of the rounded argument, without a step of Newton's: one
// in 64 bits brought no more E4M3 codes onto those of the 64-bit values (8 instead
// of 7 of 8388608 differ, 4096 x 2048: on a rounding's edge, where the fp32
// products by r and the weight decide).
__device__ __forceinline__ void inverse_root(double v, float& a, float& b) {
  const int e = (static_cast<int>(__builtin_bit_cast(uint64_t, v) >> 52) - 1023) & ~1;      // even, so that its half is whole
  a = ldexpf(1.0f, -e / 2);
  b = __builtin_amdgcn_rsqf(static_cast<float>(ldexp(v, -e)));                              // of [1, 4)
}

// Who has a row: LPR lanes (64, or fewer of narrow rows, of which a wave then
// has several), of `waves` waves.
template <int LPR>
struct Team {
  int lane, wave, w, teams, team;
  __device__ __forceinline__ Team(int waves) {
    const int whole = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & (LPR - 1);
    wave = whole;
    w = whole & (waves - 1);
    teams = static_cast<int>(blockDim.x >> 6) / waves * (64 / LPR);
    team = whole / waves * (64 / LPR) + (threadIdx.x & 63) / LPR;
  }
};

// The sums over a row's lanes, the same in all of them (`two`: of s and t).
// Every thread of the workgroup calls it; a second call needs another place.
template <int LPR>
__device__ __forceinline__ void row_sums(double& s, double& t, int waves, int wave, double (*place)[2], bool two) {
  s = lanes_sum<LPR>(s);
  if (two) t = lanes_sum<LPR>(t);
  if (LPR < 64 || waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
    place[wave][0] = s;
    place[wave][1] = t;
  }
  __syncthreads();
  const int first = wave & ~(waves - 1);
  s = t = 0.0;
  for (int i = 0; i < waves; ++i) {
    s += place[first + i][0];
    t += place[first + i][1];
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// P pieces of U columns a lane: piece p of wave w of the row's `waves` starts at
// column ((p waves + w) 64 + lane) U.  U is what makes 16 bytes of the stream, so
// that every access of a wave is one run: with 16 columns a lane (as dispatch has
// them for MX rows) 16381 x 2048 with an fp32 stream took 102 us, 4999 x 4096
// with E4M3 rows 33.
template <bool XF32, bool SF32, int KIND, int P, int LPR>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a, int waves) {
  constexpr int U = SF32 ? 4 : 8;
  static_assert(LPR == 64 || (P == 1 && (KIND == ROW_BF16 || LPR * U >= 128)), "narrow rows; a scale word is one row's");
  __shared__ double place[16][2];
  const Team<LPR> me(waves);
  const int lane = me.lane;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * me.teams + me.team;
  const bool live = row < a.rows;
  const int64_t first = (live ? row : 0) * a.width;
  const int col0 = (me.w * 64 + lane) * U, step = waves * 64 * U;
  Unit<XF32, U> x[P];
  Unit<SF32, U> r[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = col0 + p * step;
    x[p].clear();
    r[p].clear();
    if (live && col < a.width) {
      x[p].load(a.x, first + col);
      if (a.residual) r[p].load(a.residual, first + col);
    }
  }
  float h[P][U];
  double sum = 0.0, none = 0.0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = col0 + p * step;
    x[p].get(h[p]);
    if (a.residual) {
      float g[U];
      r[p].get(g);
#pragma unroll
      for (int i = 0; i < U; ++i) g[i] += h[p][i];
      r[p].set(g);
      r[p].get(h[p]);                            // as it is kept
      if (live && col < a.width) r[p].store(a.h, first + col);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) sum = fma(static_cast<double>(h[p][i]), static_cast<double>(h[p][i]), sum);
  }
  row_sums<LPR>(sum, none, waves, me.wave, place, false);
  float ra, rb;
  inverse_root(sum * a.inverse_width + a.eps, ra, rb);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = col0 + p * step;
    const bool in = live && col < a.width;
    const int64_t at = first + col;
#pragma unroll
    for (int i = 0; i < U; i += 4) {
      v4f v{};
      if (in) v = *reinterpret_cast<const v4f_any*>(a.weight + col + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) h[p][i + q] = h[p][i + q] * ra * rb * v[q];
    }
    if (KIND == ROW_BF16 || a.y) {
      Unit<false, U> y;
      y.set(h[p]);
      if (in) y.store(a.y, at);
    }
    if constexpr (KIND != ROW_BF16) {
      uint32_t codes[U / 4], word;
      mx_unit<KIND, U>(h[p], codes, word);
      if (!in) continue;
      if constexpr (KIND == ROW_E2M1 && U == 4) *reinterpret_cast<uint16_t*>(a.codes + at / 2) = static_cast<uint16_t>(codes[0]);
      else if constexpr (KIND == ROW_E2M1) *reinterpret_cast<uint32_t*>(a.codes + at / 2) = codes[0];
      else if constexpr (U == 4) *reinterpret_cast<uint32_t*>(a.codes + at) = codes[0];
      else *reinterpret_cast<v2u*>(a.codes + at) = v2u{codes[0], codes[1]};
      if ((lane & (128 / U - 1)) == 0) {
        const int64_t k = col >> 7;
        reinterpret_cast<uint32_t*>(a.scales)[a.kplanes ? k * a.rows + row : at >> 7] = word;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// Beyond 16384 columns the 128 registers of 16 waves do not hold a lane's part of
// a row with its weights, its sums and dh: weights and dh are read when they are
// wanted.  Kept all the same they spill.  This kernel for 1024 x 32768, BF16: 101 us
// with dh, 80 without, kept 176 and 163; 2048 x 16384, where they are kept: 61 and 45.
// (norm_dw_kernel is 20 and 12 us more: 512 parts of dw of 32768 or 16384 columns are
// 67 or 34 MB, written and read again.)
// A workgroup's teams take rows in turn and add up their part of dw in
// registers; the teams' parts meet in LDS, the workgroups' in norm_dw_kernel,
// in a fixed order.
template <bool SF32, int P, int THREADS, int LPR>
__global__ __launch_bounds__(THREADS) void rms_norm_backward_kernel(NormArgs a, int waves) {
  constexpr bool KEPT = P < 4;
  __shared__ double place[2][16][2];
  __shared__ v4f part[4][P * 2][64];
  const Team<LPR> me(waves);
  const int lane = threadIdx.x & 63, wave = me.wave, w = me.w, teams = me.teams;
  int col[P];
  float kept[KEPT ? P : 1][8], acc[P][8];
  auto load_weights = [&](int p, float* f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      v4f v{};
      if (col[p] < a.width) v = *reinterpret_cast<const v4f_any*>(a.weight + col[p] + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) f[i + q] = v[q];
    }
  };
#pragma unroll
  for (int p = 0; p < P; ++p) {
    col[p] = ((p * waves + w) * 64 + me.lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[p][i] = 0.0f;
    if constexpr (KEPT) load_weights(p, kept[p]);
  }
  auto weights = [&](int p, float* f) __attribute__((always_inline)) {
    if constexpr (KEPT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = kept[p][i];
    } else {
      load_weights(p, f);
    }
  };
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * teams; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * teams, turn ^= 1) {
    const int64_t row = base + me.team;
    const bool live = row < a.rows;
    const int64_t first = (live ? row : 0) * a.width;
    Unit<false, 8> dy[P];
    Unit<SF32, 8> h[P], dh[KEPT ? P : 1];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      dy[p].clear();
      h[p].clear();
      if constexpr (KEPT) dh[p].clear();
      if (live && col[p] < a.width) {
        dy[p].load(a.dy, first + col[p]);
        h[p].load(a.stored, first + col[p]);
        if (KEPT && a.dh) dh[p].load(a.dh, first + col[p]);
      }
    }
    double sq = 0.0, dot = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float d[8], v[8], wt[8];
      dy[p].get(d);
      h[p].get(v);
      weights(p, wt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), sq);
        dot = fma(static_cast<double>(d[i] * wt[i]), static_cast<double>(v[i]), dot);
      }
    }
    row_sums<LPR>(sq, dot, waves, wave, place[turn], true);
    float ra, rb;
    inverse_root(sq * a.inverse_width + a.eps, ra, rb);
    const float mean = static_cast<float>(dot * a.inverse_width * ra * rb);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float d[8], v[8], g[8], wt[8];
      dy[p].get(d);
      h[p].get(v);
      if constexpr (!KEPT) {
        dh[0].clear();
        if (a.dh && live && col[p] < a.width) dh[0].load(a.dh, first + col[p]);
      }
      dh[KEPT ? p : 0].get(g);
      weights(p, wt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = v[i] * ra * rb;
        acc[p][i] = fmaf(d[i], xh, acc[p][i]);
        v[i] = fmaf((d[i] * wt[i] - xh * mean) * ra, rb, g[i]);
      }
      if (a.dx && live && col[p] < a.width) {
        h[p].set(v);
        h[p].store(a.dx, first + col[p]);
      }
    }
  }
  if (!a.partial) return;
  // the rows of a wave, then the waves with the same columns (4, where there are several)
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] += __shfl_xor(acc[0][i], d);
  const int team = wave / waves, same = static_cast<int>(blockDim.x >> 6) / waves;
  if (same > 1) {
    if (team > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          part[wave][2 * p + q][lane] = v4f{acc[p][4 * q], acc[p][4 * q + 1], acc[p][4 * q + 2], acc[p][4 * q + 3]};
    }
    __syncthreads();
    if (team > 0) return;
    for (int t = 1; t < same; ++t)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const v4f v = part[t * waves + w][2 * p + q][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[p][4 * q + i] += v[i];
        }
  }
  if (LPR < 64 && lane >= LPR) return;
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (col[p] < a.width) {
      v4f* const out = reinterpret_cast<v4f*>(a.partial + static_cast<int64_t>(blockIdx.x) * a.width + col[p]);
      out[0] = v4f{acc[p][0], acc[p][1], acc[p][2], acc[p][3]};
      out[1] = v4f{acc[p][4], acc[p][5], acc[p][6], acc[p][7]};
    }
}

// dw of 16 columns: 16 threads a column share the workgroups' parts.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* partial, float* dw, int width, int parts) {
  __shared__ float red[16][17];
  const int x = threadIdx.x & 15, q = threadIdx.x >> 4, col = blockIdx.x * 16 + x;
  float s = 0.0f;
  if (col < width) {
#pragma unroll 8
    for (int i = q; i < parts; i += 16) s += partial[static_cast<int64_t>(i) * width + col];
  }
  red[q][x] = s;
  __syncthreads();
  if (q == 0 && col < width) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[i][x];
    dw[col] = v;
  }
}

// ---------------------------------------------------------------------------
// choices
// ---------------------------------------------------------------------------

// Pieces a lane, waves a row and lanes a row, all powers of two, for `unit`
// columns a lane and piece: 1024 columns a wave, 2048 where 16 waves would not
// hold the row otherwise, and several narrow rows a wave.  Measured against 2048
// a wave (and 512), 2048 columns: forward with an fp32 stream 78.6 us against 85.6
// (77.2), backward 49.7 against 50.8 (61); 4096 columns with E4M3 rows 28.3
// against 29.1 (29.5).  524288 x 64 with residual: eight rows a wave 45 us forward
// and 48 backward, a row a wave 151 and 280.
struct Shape {
  int p, waves, lanes;
};
Shape shape_of(int width, int unit, int least_lanes) {
  Shape s{1, 1, 64};
  const int pieces = (width + 64 * unit - 1) / (64 * unit), most = (width <= 16384 ? 1024 : 2048) / (64 * unit);
  while (s.p < most && s.p < pieces) s.p *= 2;
  while (s.p * s.waves < pieces) s.waves *= 2;
  while (s.lanes > least_lanes && s.lanes / 2 * unit >= width) s.lanes /= 2;
  return s;
}
int threads_of(const Shape& s) { return s.waves > 4 ? 64 * s.waves : 256; }
int64_t blocks_of(const Shape& s, int64_t rows) {
  const int teams = threads_of(s) / 64 / s.waves * (64 / s.lanes);
  return (rows + teams - 1) / teams;
}

template <typename F>
hipError_t by_pieces(int p, F&& f) {
  switch (p) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

// Columns a lane and piece of the forward, and the least lanes a row: what a
// scale word's 128 columns take, or 8.
constexpr int forward_unit(bool stream_f32) { return stream_f32 ? 4 : 8; }
constexpr int forward_lanes(bool stream_f32, int kind) { return kind == ROW_BF16 ? 8 : 128 / forward_unit(stream_f32); }

template <bool XF32, bool SF32, int KIND, int P, int LPR>
hipError_t launch_norm_kernel(const NormArgs& a, const Shape& sh, hipStream_t s) {
  hipLaunchKernelGGL((rms_norm_kernel<XF32, SF32, KIND, P, LPR>), dim3(static_cast<unsigned>(blocks_of(sh, a.rows))),
                     dim3(threads_of(sh)), 0, s, a, sh.waves);
  return hipGetLastError();
}
template <bool XF32, bool SF32, int KIND>
hipError_t launch_norm_kind(const NormArgs& a, hipStream_t s) {
  constexpr int U = forward_unit(SF32), kMost = 2048 / (64 * U), kLeast = forward_lanes(SF32, KIND);
  const Shape sh = shape_of(a.width, U, kLeast);
  if constexpr (kLeast <= 8)
    if (sh.lanes == 8) return launch_norm_kernel<XF32, SF32, KIND, 1, 8>(a, sh, s);
  if constexpr (kLeast <= 16)
    if (sh.lanes == 16) return launch_norm_kernel<XF32, SF32, KIND, 1, 16>(a, sh, s);
  if (sh.lanes == 32) return launch_norm_kernel<XF32, SF32, KIND, 1, 32>(a, sh, s);
  return by_pieces(sh.p, [&](auto p) {
    return launch_norm_kernel<XF32, SF32, KIND, decltype(p)::value < kMost ? decltype(p)::value : kMost, 64>(a, sh, s);
  });
}
template <bool XF32, bool SF32>
hipError_t launch_norm_types(const NormArgs& a, hipStream_t s) {
  switch (a.kind) {
    case ROW_E4M3: return launch_norm_kind<XF32, SF32, ROW_E4M3>(a, s);
    case ROW_E5M2: return launch_norm_kind<XF32, SF32, ROW_E5M2>(a, s);
    case ROW_E2M1: return launch_norm_kind<XF32, SF32, ROW_E2M1>(a, s);
    default: return launch_norm_kind<XF32, SF32, ROW_BF16>(a, s);
  }
}

Shape backward_shape(int width) { return shape_of(width, 8, 8); }

// Workgroups of the backward: two of four waves to a compute unit (1024 of them:
// 53.6 us instead of 49.7, their parts of dw are twice as many).
int64_t backward_blocks(int64_t rows, int width) {
  const int64_t all = blocks_of(backward_shape(width), rows);
  return all < 512 ? all : 512;
}

template <int P, int THREADS, int LPR = 64>
void launch_backward_kernel(const NormArgs& a, dim3 grid, int waves, hipStream_t s) {
  const dim3 block(waves > 4 ? 64 * waves : 256);
  if (a.stream_f32) hipLaunchKernelGGL((rms_norm_backward_kernel<true, P, THREADS, LPR>), grid, block, 0, s, a, waves);
  else hipLaunchKernelGGL((rms_norm_backward_kernel<false, P, THREADS, LPR>), grid, block, 0, s, a, waves);
}

}  // namespace

int64_t rms_norm_threads(int64_t rows, int32_t width, bool stream_f32, int kind) {
  const Shape sh = shape_of(width, forward_unit(stream_f32), forward_lanes(stream_f32, kind));
  return blocks_of(sh, rows) * threads_of(sh);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (a.x_f32) return launch_norm_types<true, true>(a, s);
  return a.stream_f32 ? launch_norm_types<false, true>(a, s) : launch_norm_types<false, false>(a, s);
}

int64_t rms_norm_backward_workspace(int64_t rows, int32_t width) { return backward_blocks(rows, width) * width * 4; }

hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s) {
  const int64_t blocks = backward_blocks(a.rows, a.width);
  if (blocks > 0) {
    const Shape sh = backward_shape(a.width);
    const dim3 grid(static_cast<unsigned>(blocks));
    const hipError_t e = by_pieces(sh.p, [&](auto p) {
      constexpr int P = decltype(p)::value < 4 ? decltype(p)::value : 4;
      if constexpr (P == 1) {
        if (sh.lanes == 8) launch_backward_kernel<P, 256, 8>(a, grid, sh.waves, s);
        else if (sh.lanes == 16) launch_backward_kernel<P, 256, 16>(a, grid, sh.waves, s);
        else if (sh.lanes == 32) launch_backward_kernel<P, 256, 32>(a, grid, sh.waves, s);
        if (sh.lanes < 64) return hipGetLastError();
      }
      // (more than one wave takes two pieces a lane, more than 16384 columns four)
      if constexpr (P == 4) launch_backward_kernel<P, 1024>(a, grid, sh.waves, s);
      else if (sh.waves <= 4) launch_backward_kernel<P, 256>(a, grid, sh.waves, s);
      else if constexpr (P == 2) launch_backward_kernel<P, 1024>(a, grid, sh.waves, s);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!a.dw) return hipSuccess;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((a.width + 15) / 16), dim3(256), 0, s, a.partial, a.dw, a.width,
                     static_cast<int>(blocks));
  return hipGetLastError();
}

}  // namespace moegg
