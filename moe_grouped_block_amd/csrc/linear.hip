// Matrix product with bias, activation and residual in its epilogue, dense or
// grouped by expert, and its gradients (BF16 operands, fp32 sums).
//
//   forward    z = x w_g^T + b_g (c = bf16(z)), y = act(z) + residual
//   backward   dz = dy act'(c), rounded to bf16 as the operand of both products
//              dx = dz w_g, dw_g = dz^T x over the group's rows, db_g = column
//              sums of the unrounded dz
//
// Group g owns rows [offsets[g-1], offsets[g]) (any numbers, no alignment);
// without offsets there is one group of all rows.
#include <cstring>
#include <type_traits>

#include "linear_gemm.h"

namespace moegg {
namespace {

// ---------------------------------------------------------------------------
// few rows: the weights are read once and nothing else matters
// ---------------------------------------------------------------------------
//
// One workgroup computes 16 NT columns n for up to 16 rows of a group at a
// time.  Its NW waves share r: each streams its part of the weight rows from
// global memory into registers (16 bytes a lane, U steps of 32 r in flight)
// and multiplies it with the rows of x by 16 x 16 x 32 MFMAs; the partial sums
// meet in LDS.  The rows of x come from L2, as many bytes a workgroup as one
// of its NT weight tiles where there are 16 of them.
constexpr int kFewRows = 16;

template <int NT, int NW, int U>
__global__ __launch_bounds__(64 * NW) void linear_few_rows_kernel(LinearArgs a) {
  typedef float v4f4 __attribute__((ext_vector_type(4)));
  __shared__ float part[NW][NT][16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int g = blockIdx.y;
  int64_t begin, end;
  group_rows(a, g, begin, end);
  const bool pair = a.act == LIN_SWIGLU;
  // column of index i of tile t: SwiGLU tiles are 8 linear columns and their 8 gates
  auto column = [&](int t, int i) {
    const int tile = blockIdx.x * NT + t;
    if (!pair) return tile * 16 + i;
    const int j = tile * 8 + (i & 7);                       // output column
    return (j >> 5) * 64 + (j & 31) + (i & 8) * 4;
  };
  const uint16_t* wrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    wrow[t] = a.w + (static_cast<int64_t>(g) * a.n + min(column(t, l16), a.n - 1)) * a.k + q * 8;
  const int steps = (a.k + 31) / 32, whole = a.k / 32;
  const int s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
  const int n_out = pair ? a.n / 2 : a.n;
  for (int64_t m0 = begin; m0 < end; m0 += kFewRows) {
    const int rows = static_cast<int>(min(end - m0, int64_t{kFewRows}));
    const uint16_t* const xrow = a.x + (m0 + min(l16, rows - 1)) * a.k + q * 8;
    v4f4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = v4f4{};
    for (int s = s0; s < s1; s += U) {
      v4u vw[NT][U], vx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        vx[u] = v4u{};
#pragma unroll
        for (int t = 0; t < NT; ++t) vw[t][u] = v4u{};
        if (s + u < s1 && (s + u < whole || (s + u) * 32 + q * 8 < a.k)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            vw[t][u] = *reinterpret_cast<const v4u*>(wrow[t] + (s + u) * 32);
          vx[u] = *reinterpret_cast<const v4u*>(xrow + (s + u) * 32);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, vw[t][u]), __builtin_bit_cast(v8bf, vx[u]),
                                                           acc[t], 0, 0, 0);
    }
    // lane: row l16, weight rows 4 q + [0, 4)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][t][l16][4 * q + e] = acc[t][e];
    __syncthreads();
    for (int at = threadIdx.x; at < NT * 256; at += 64 * NW) {
      const int i = at & 15, row = (at >> 4) & 15, t = at >> 8;
      const int n = column(t, i);
      if (row < rows && n < a.n) {
        const int64_t m = m0 + row;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) z += part[w][t][row][i];
        if (a.bias) z += a.bias[static_cast<int64_t>(g) * a.n + n];
        if (a.c) a.c[m * a.n + n] = static_cast<uint16_t>(bf16x2(z, 0.0f));
        float y = z;
        bool store = true;
        int ycol = n;
        if (pair) {
          float gate = 0.0f;
          const int ng = n + 32;
          store = i < 8;
          if (store) {
#pragma unroll
            for (int w = 0; w < NW; ++w) gate += part[w][t][row][i + 8];
            if (a.bias) gate += a.bias[static_cast<int64_t>(g) * a.n + ng];
          }
          y = z * (gate * sigmoid_f(gate));
          ycol = (blockIdx.x * NT + t) * 8 + i;
        } else if (a.act == LIN_GELU) {
          y = gelu_f(z);
        } else if (a.act == LIN_SRELU) {
          const float v = relu_f(z);
          y = v * v;
        }
        if (store) {
          if (a.residual) y += bf_lo(a.residual[m * n_out + ycol]);
          if (a.out_f32) static_cast<float*>(a.y)[m * n_out + ycol] = y;
          else static_cast<uint16_t*>(a.y)[m * n_out + ycol] = static_cast<uint16_t>(bf16x2(y, 0.0f));
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// joins of a split r
// ---------------------------------------------------------------------------

__device__ __forceinline__ void store4(void* base, bool f32, int64_t i, v4f v) {
  if (f32) *reinterpret_cast<v4f*>(static_cast<float*>(base) + i) = v;
  else *reinterpret_cast<v2u*>(static_cast<uint16_t*>(base) + i) = v2u{bf16x2(v.x, v.y), bf16x2(v.z, v.w)};
}

// Four columns of z (c's columns at, ...), kept in 8 bits: 8 neighbouring
// threads have a block of 32.
template <int KIND>
__device__ __forceinline__ void save4(const LinearArgs& a, int64_t row, int col, v4f z) {
  const float f[4] = {z.x, z.y, z.z, z.w};
  uint32_t amax = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) amax = max(amax, __float_as_uint(f[e]) & 0x7FFFFFFFu);
  amax = max(amax, dpp_u<0xB1>(amax));
  amax = max(amax, dpp_u<0x4E>(amax));
  amax = max(amax, dpp_u<0x141>(amax));
  const uint32_t byte = mx_block_byte<KIND>(amax);
  *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(a.c) + row * a.n + col) =
      byte == 255u ? 0u : mx_codes<KIND>(f, mx_factor(byte));
  if ((col & 31) == 0) a.c_sf[row * (a.n >> 5) + (col >> 5)] = static_cast<uint8_t>(byte);
}

// The parts of tiles [first, tiles), added in their order: 4 columns of the
// output a thread (and, of a SwiGLU pair, their 4 gates).
template <int MODE, int BP, int BQ>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a, TilePlan plan) {
  constexpr int PER = BP * BQ / 4 / 256;         // workgroups per tile
  const int lane = threadIdx.x & 63;
  const int split = plan.tiles - plan.first, i = blockIdx.x / PER;
  const int at = (blockIdx.x - i * PER) * 256 + threadIdx.x;
  const int row = at / (BQ / 4), col = (at - row * (BQ / 4)) * 4;
  LinearTile t;
  const int row_tiles = static_cast<int>(((MODE == MODE_DW ? a.n : a.m) + BP - 1) / BP);
  if (!place<MODE, BP, BQ>(a, plan.first + i, row_tiles, lane, t)) return;
  const int64_t r = t.row0 + row;
  const int c = t.col0 + col, cols = out_columns<MODE>(a);
  if (r >= t.row_end || c >= cols) return;
  const float* const base = partials<MODE>(a) + static_cast<int64_t>(i) * (BP * BQ) + row * BQ + col;
  const int64_t stride = static_cast<int64_t>(split) * (BP * BQ);
  auto sum = [&](int off) __attribute__((always_inline)) {
    v4f v = *reinterpret_cast<const v4f*>(base + off);
    for (int q = 1; q < plan.parts; ++q) v += *reinterpret_cast<const v4f*>(base + q * stride + off);
    return v;
  };
  if constexpr (MODE != MODE_FORWARD) {
    store4(MODE == MODE_DX ? static_cast<void*>(a.dx) : a.dw, MODE == MODE_DW && a.out_f32,
           (MODE == MODE_DW ? static_cast<int64_t>(t.g) * a.n + r : r) * cols + c, sum(0));
  } else {
    const bool pair = a.act == LIN_SWIGLU;
    if (pair && (c & 32)) return;                // a pair's gates are handled with its linear half
    auto z_of = [&](int off) __attribute__((always_inline)) {
      v4f z = sum(off);
      if (a.bias) z += *reinterpret_cast<const v4f_any*>(a.bias + c + off);
      if (a.c && a.c_kind == ROW_E4M3) save4<ROW_E4M3>(a, r, c + off, z);
      else if (a.c && a.c_kind == ROW_E5M2) save4<ROW_E5M2>(a, r, c + off, z);
      else if (a.c) store4(a.c, false, r * a.n + c + off, z);
      return z;
    };
    v4f z = z_of(0);
    if (pair) {
      const v4f gate = z_of(32);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = z[e] * (gate[e] * sigmoid_f(gate[e]));
    } else if (a.act == LIN_GELU) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = gelu_f(z[e]);
    } else if (a.act == LIN_SRELU) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = relu_f(z[e]);
        z[e] = v * v;
      }
    }
    const int n_out = pair ? a.n / 2 : a.n;
    const int64_t o = r * n_out + (pair ? (c >> 6) * 32 + (c & 31) : c);
    if (a.residual) {
      const v2u u = *reinterpret_cast<const v2u*>(a.residual + o);
      z += v4f{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
    }
    store4(a.y, a.out_f32, o, z);
  }
}

// ---------------------------------------------------------------------------
// dz and db
// ---------------------------------------------------------------------------
//
// One pass over dy and c: dz in bf16, and the column sums of the unrounded
// dz over tiles of dz_rows() rows of one group, summed per group afterwards.
// An x in 8 bits becomes BF16 in the same launch (it is an operand of dw as dz
// is): its workgroups run beside the others.
// dz is the operand of both products: kept in two bf16 parts it would double
// their work.  With its one rounding dx and dw are 0.0023 off the 64-bit values
// (root mean square, 16384 x 2816 x 2048 with SwiGLU), where the rounding of the
// results alone is 0.0017.
__device__ __forceinline__ void unpack8(v4u u, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(u[i]);
    f[2 * i + 1] = bf_hi(u[i]);
  }
}
__device__ __forceinline__ v4u pack8(const float* f) {
  return v4u{bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7])};
}

// Eight columns of a row of c: BF16, or codes and their block's scale byte.
template <int CK>
struct EightOfC {
  v2u codes;
  uint32_t byte;
  __device__ __forceinline__ void clear() {
    codes = v2u{};
    byte = 0;
  }
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t row, int n) {
    codes = *reinterpret_cast<const v2u*>(reinterpret_cast<const uint8_t*>(a.c) + row * a.n + n);
    byte = a.c_sf[row * (a.n >> 5) + (n >> 5)];
  }
  __device__ __forceinline__ void get(float* z) const {
    const float f = mx_scale_value(byte);
    mx_four<CK>(codes.x, f, z);
    mx_four<CK>(codes.y, f, z + 4);
  }
};
template <>
struct EightOfC<ROW_BF16> {
  v4u u;
  __device__ __forceinline__ void clear() { u = v4u{}; }
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t row, int n) {
    u = *reinterpret_cast<const v4u*>(a.c + row * a.n + n);
  }
  __device__ __forceinline__ void get(float* z) const { unpack8(u, z); }
};

// One row's 8 columns of dy (and of c, or of both halves of a pair) -> dz.
template <int ACT, int CK>
__device__ __forceinline__ void dz_of(const float* d, const EightOfC<CK>& c0, const EightOfC<CK>& c1, float* v, float* w) {
  if constexpr (ACT == LIN_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d[i];
  } else if constexpr (ACT == LIN_SWIGLU) {
    float x[8], q[8];
    c0.get(x);
    c1.get(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_f(q[i]);
      v[i] = d[i] * (q[i] * s);
      w[i] = d[i] * (x[i] * s) * (1.0f + q[i] * (1.0f - s));
    }
  } else {
    float z[8];
    c0.get(z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (ACT == LIN_SRELU) {
        const float t = d[i] * relu_f(z[i]);           // (2 z may overflow where 2 d z does not)
        v[i] = t + t;
      } else {
        // past 30 s is 0 or 1: keeps 0 times z^3 from becoming NaN (comparisons, so that a NaN stays one)
        const float c = z[i] > 30.0f ? 30.0f : z[i] < -30.0f ? -30.0f : z[i];
        const float s = sigmoid_f(2.0f * kGeluC * c * (1.0f + kGeluA * c * c));
        v[i] = d[i] * (s + c * s * (1.0f - s) * (2.0f * kGeluC) * (1.0f + 3.0f * kGeluA * c * c));
      }
    }
  }
}

// Rows and columns of dy that a workgroup of linear_dz_kernel takes, and the
// rest of its launch.
struct DzPlan {
  uint16_t* dz;             // or null
  float* sums;              // or null
  uint16_t* x;              // where an x in 8 bits goes, or null: by the workgroups from y = cols on
  int rows, cols;           // rows of a tile, workgroups along the columns
};

// 32 threads run along 256 columns of dy, 8 rows at a time; four of a
// thread's rows are in flight at once.
template <int ACT, int CK, bool X8>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearArgs a, DzPlan plan) {
  if constexpr (X8) {
    if (static_cast<int>(blockIdx.y) >= plan.cols) {
      const int64_t chunk = static_cast<int64_t>(blockIdx.y - plan.cols) * gridDim.x + blockIdx.x;
      if (a.x8.kind == ROW_E4M3) dequantise_chunk<ROW_E4M3, false>(a.x8, plan.x, a.m, a.k, chunk);
      else dequantise_chunk<ROW_E5M2, false>(a.x8, plan.x, a.m, a.k, chunk);
      return;
    }
  }
  uint16_t* const dz = plan.dz;
  float* const sums = plan.sums;
  constexpr bool PAIR = ACT == LIN_SWIGLU;
  constexpr int S = PAIR ? 16 : 8, U = 4;
  __shared__ float red[8][32][S + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, lane = threadIdx.x & 63;
  int g;
  int64_t row0, end;
  if (!find_row_tile(a, plan.rows, blockIdx.x, lane, g, row0, end)) return;
  const int n_out = PAIR ? a.n / 2 : a.n;
  const int col = (blockIdx.y * 32 + tx) * 8;                  // of dy
  const int n = PAIR ? (col >> 5) * 64 + (col & 31) : col;     // of dz (and n + 32 of a pair)
  float s[S];
#pragma unroll
  for (int i = 0; i < S; ++i) s[i] = 0.0f;
  const int rows = static_cast<int>(min(end - row0, int64_t{plan.rows}));
  if (col < n_out) {
    for (int r = ty; r < rows; r += 8 * U) {
      v4u d[U];
      EightOfC<CK> c0[U], c1[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = row0 + min(r + 8 * u, rows - 1);     // (rows past the end: read, not used)
        d[u] = *reinterpret_cast<const v4u*>(a.dy + m * n_out + col);
        c0[u].clear();
        c1[u].clear();
        if constexpr (ACT != LIN_NONE) c0[u].load(a, m, n);
        if constexpr (PAIR) c1[u].load(a, m, n + 32);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + 8 * u >= rows) break;
        const int64_t m = row0 + r + 8 * u;
        float f[8], v[8], w[8];
        unpack8(d[u], f);
        dz_of<ACT, CK>(f, c0[u], c1[u], v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[i] += v[i];
          if constexpr (PAIR) s[8 + i] += w[i];
        }
        if (dz) {
          *reinterpret_cast<v4u*>(dz + m * a.n + n) = pack8(v);
          if constexpr (PAIR) *reinterpret_cast<v4u*>(dz + m * a.n + n + 32) = pack8(w);
        }
      }
    }
  }
  if (!sums) return;
#pragma unroll
  for (int i = 0; i < S; ++i) red[ty][tx][i] = s[i];
  __syncthreads();
  // 32 x S sums, S / 8 a thread
#pragma unroll
  for (int h = 0; h < S / 8; ++h) {
    const int i = (threadIdx.x & 7) + 8 * h, t = threadIdx.x >> 3;
    const int c = (blockIdx.y * 32 + t) * 8;
    if (c >= n_out) continue;
    float v = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += red[y][t][i];
    const int at = PAIR ? (c >> 5) * 64 + (c & 31) + (i & 7) + 32 * h : c + i;
    sums[static_cast<int64_t>(blockIdx.x) * a.n + at] = v;
  }
}

template <int Q>
__global__ __launch_bounds__(512) void linear_db_kernel(LinearArgs a, DbPlan p) {
  __shared__ float red[kDbWords];
  db_columns<Q>(a, p, blockIdx.x, blockIdx.y, red);
}

// ---------------------------------------------------------------------------
// choices
// ---------------------------------------------------------------------------

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return div_up(a, b) * b; }

// Row tiles of all groups at most.
int64_t row_tiles(const LinearArgs& a, int bm) { return most_row_tiles(a, bm); }

// Workgroups of linear_dz_kernel along the columns, and rows of a tile: 128, or
// 32 where that leaves most of the chip empty (129 x 512, GELU: 13.7 us with
// 128, 5.5 with 32).
int dz_cols(const LinearArgs& a) { return static_cast<int>(div_up(a.act == LIN_SWIGLU ? a.n / 2 : a.n, 256)); }
int dz_rows(const LinearArgs& a) { return row_tiles(a, 128) * dz_cols(a) < 512 ? 32 : 128; }

// Tile shapes: how many workgroups the chip holds at once, and what they take,
// in microseconds: a step of 64 r where few of them are there, where half of
// them are and where more are, and everything outside the steps.  Per product:
// forward, dx, dw.  Fitted to sweeps of shapes and parts over 30 problems of 40
// to 16384 rows; what was chosen was the best or within 10 % of it.
enum Shape : int { SHAPE_256 = 0, SHAPE_128 = 1, SHAPE_64 = 2 };
struct ShapeCost {
  int bp, bq, slots;
  double few, half, step, rest;
};
constexpr ShapeCost kShapes[3][3] = {
    {{256, 256, 256, 1.00, 1.20, 1.55, 8.0}, {128, 128, 512, 0.42, 0.58, 1.10, 5.0}, {64, 64, 256, 0.17, 0.22, 0.25, 4.0}},
    {{256, 256, 256, 1.00, 1.10, 1.40, 8.0}, {128, 128, 512, 0.38, 0.53, 0.90, 4.8}, {64, 64, 256, 0.17, 0.22, 0.25, 4.0}},
    {{256, 256, 256, 0.95, 1.05, 1.35, 8.0}, {128, 128, 512, 0.38, 0.53, 0.90, 4.8}, {64, 64, 256, 0.20, 0.25, 0.25, 4.0}}};

struct Plan {
  Shape shape;
  TilePlan tiles;
  int64_t workgroups;
  int64_t partial_bytes;
  double cost;                // microseconds, by kShapes
};

// Which tile, and which tiles share their r among several workgroups: the
// cheapest by rounds of workgroups, where a last round that leaves most of the
// chip empty (or the only one) may be split, against the bytes of its parts,
// written and read at about 4 TB/s, and a join's launch.
// `tiles(s)`: tiles of shape s at most, of which `likely(s)` are taken to be
// there; `r`: length of the sum; `known`: the tiles are these, and may be split.
template <typename F, typename G>
Plan choose(LinearMode mode, F&& tiles, G&& likely, int64_t r, bool known) {
  Plan best{};
  double least = 0.0;
  const int64_t steps = div_up(r > 0 ? r : 1, kR);
  for (int s = 0; s < 3; ++s) {
    const ShapeCost& c = kShapes[mode][s];
    const int64_t total = tiles(c);
    auto rounds = [&](int64_t n, int64_t st) {
      const int64_t left = n % c.slots;
      return static_cast<double>(n / c.slots) * (st * c.step + c.rest) +
             (left ? st * (left <= c.slots / 2 ? c.few + (c.half - c.few) * 2 * left / c.slots : c.step) + c.rest : 0.0);
    };
    auto take = [&](double cost, int64_t first, int parts) {
      if (least != 0.0 && cost >= least) return;
      least = best.cost = cost;
      best.shape = static_cast<Shape>(s);
      best.tiles = {known ? static_cast<int>(total) : -1, static_cast<int>(first), parts};
      best.workgroups = first + (total - first) * parts;
      best.partial_bytes = parts > 1 ? (total - first) * parts * c.bp * c.bq * 4 : 0;
    };
    take(rounds(likely(c), steps), total, 1);
    if (!known) continue;
    for (int64_t first : {int64_t{0}, total / c.slots * c.slots}) {
      if (first == total || (first == 0 && total > 2 * c.slots)) continue;
      for (int parts = 2; parts <= 16 && parts * 2 <= steps; ++parts) {
        const double bytes = static_cast<double>((total - first) * parts) * c.bp * c.bq * 4;
        take((first ? rounds(first, steps) : 0.0) + rounds((total - first) * parts, div_up(steps, parts)) + 4.0 + 2.0 * bytes / 4e6,
             first, parts);
      }
    }
  }
  return best;
}

// Split only without offsets, where the host knows the tiles.  (The workspace
// is sized without knowing the offsets, so never too small.)
Plan plan_rows(const LinearArgs& a, LinearMode mode) {
  const int64_t cols = mode == MODE_FORWARD ? a.n : a.k, r = mode == MODE_FORWARD ? a.k : a.n;
  const auto tiles = [&](const ShapeCost& c) { return row_tiles(a, c.bp) * div_up(cols, c.bq); };
  // half a tile of every group is not full, but a group with rows has one
  const auto likely = [&](const ShapeCost& c) {
    const int64_t most = row_tiles(a, c.bp), filled = a.m < a.groups ? a.m : a.groups, ragged = a.m / c.bp + a.groups / 2;
    return (a.groups == 1 ? most : ragged < filled ? filled : ragged < most ? ragged : most) * div_up(cols, c.bq);
  };
  return choose(mode, tiles, likely, r, a.groups == 1 && !a.offsets);
}
Plan plan_dw(const LinearArgs& a) {
  // a group's share of the rows; groups whose rows the host does not know are not split
  const auto tiles = [&](const ShapeCost& c) { return a.groups * div_up(a.n, c.bp) * div_up(a.k, c.bq); };
  return choose(MODE_DW, tiles, tiles, div_up(a.m, a.groups), a.groups == 1);
}
// The kernel for few rows reads a group's weights once for every 16 of its
// rows, so the rows must be few even where most of them are one group's.
// Measured, against tiles, 64 groups of 2048 x 1408: 32 rows 27 / 28 us, 64
// rows 37 / 51, 128 rows 59 / 61, 256 rows 68 / 64; with all rows in one
// group 128 rows 39 / 18, 512 rows 155 / 18.
// Its columns are spread over workgroups, so it does not keep c in 8 bits,
// whose blocks are 32 columns: tiles do.
bool few_rows(const LinearArgs& a) {
  if (a.c_kind != ROW_BF16) return false;
  return a.m <= kFewRows || (a.m <= 2 * static_cast<int64_t>(a.groups) && a.m <= 8 * kFewRows);
}

// The forward's tiles, of all rows but the last `few`: a handful of rows past
// whole tiles would cost a row of tiles (often a round of its own, or a split
// and a join), the kernel for few rows a launch and a pass over the weights.
// Measured: 4099 x 2048 x 2816 64.3 -> 63.0 us, 2050 x 2048 x 2048 37.7 -> 30.0,
// 8200 x 4096 x 4096 244 -> 230, 16390 x 64 x 2048 28.4 -> 24.0.
struct ForwardPlan {
  Plan tiles;
  int64_t few;                // all of them: no tiles
};
ForwardPlan plan_forward(const LinearArgs& a) {
  if (a.m == 0 || few_rows(a)) return {Plan{}, a.m};
  ForwardPlan f{plan_rows(a, MODE_FORWARD), 0};
  const int64_t few = a.m % 128;
  if (a.c_kind == ROW_BF16 && a.groups == 1 && !a.offsets && few && few <= kFewRows && few < a.m) {
    LinearArgs b = a;
    b.m -= few;
    const Plan p = plan_rows(b, MODE_FORWARD);
    if (p.cost + 5.0 + 2.0 * a.n * a.k / 5e6 < f.tiles.cost) f = {p, few};
  }
  return f;
}

template <int MODE, int BP, int BQ>
void launch_join(const LinearArgs& a, const Plan& p, hipStream_t s) {
  if (p.tiles.parts > 1)
    hipLaunchKernelGGL((linear_join_kernel<MODE, BP, BQ>),
                       dim3(static_cast<unsigned>((p.tiles.tiles - p.tiles.first) * (BP * BQ / 1024))), dim3(256), 0, s, a, p.tiles);
}
// dw's tiles are the host's in any case (tiles < 0 means counted on the device).
TilePlan dw_tiles(const Plan& p) {
  return p.tiles.tiles < 0 ? TilePlan{static_cast<int>(p.workgroups), static_cast<int>(p.workgroups), 1} : p.tiles;
}

template <int MODE>
hipError_t launch_tiles(const LinearArgs& a, const Plan& p, hipStream_t s) {
  const TilePlan t = MODE == MODE_DW ? dw_tiles(p) : p.tiles;
  const dim3 grid(static_cast<unsigned>(p.workgroups));
  switch (p.shape) {
    case SHAPE_256:
      if constexpr (MODE == MODE_DW) {
        if (a.x8.kind == ROW_E4M3) {
          hipLaunchKernelGGL((linear_pingpong_kernel<MODE, ROW_E4M3>), grid, dim3(512), 0, s, a, t);
          launch_join<MODE, 256, 256>(a, p, s);
          break;
        }
        if (a.x8.kind == ROW_E5M2) {
          hipLaunchKernelGGL((linear_pingpong_kernel<MODE, ROW_E5M2>), grid, dim3(512), 0, s, a, t);
          launch_join<MODE, 256, 256>(a, p, s);
          break;
        }
      }
      hipLaunchKernelGGL((linear_pingpong_kernel<MODE>), grid, dim3(512), 0, s, a, t);
      launch_join<MODE, 256, 256>(a, p, s);
      break;
    case SHAPE_128:
      if constexpr (MODE == MODE_FORWARD) {
        if (p.workgroups > 256) hipLaunchKernelGGL((linear_tile_kernel<128, 128, 2, 2>), grid, dim3(256), 0, s, a, t);
        else hipLaunchKernelGGL((linear_ring_kernel<MODE, 128, 128, 2, 2>), grid, dim3(256), 0, s, a, t);
      } else {
        hipLaunchKernelGGL((linear_ring_kernel<MODE, 128, 128, 2, 2>), grid, dim3(256), 0, s, a, t);
      }
      launch_join<MODE, 128, 128>(a, p, s);
      break;
    case SHAPE_64:
      hipLaunchKernelGGL((linear_narrow_kernel<MODE>), grid, dim3(512), 0, s, a, t);
      launch_join<MODE, 64, 64>(a, p, s);
      break;
  }
  return hipGetLastError();
}

// db, dx and dw in one launch where both products have the same tiles, of 256 x
// 256 or 64 x 64: dx's tiles fill what dw's last round leaves empty, and db's
// few workgroups are beside them.  Measured against launches of their own: 64
// groups of 2048 x 1408, 24571 rows, 565 -> 514 us (fp32 dw), 456 -> 422 (BF16
// dw); dense 16384 x 2816 x 2048 and 4096^3, 1 to 2 % less.  (The tiles of the
// two spread over each other took 546 instead of 516 us in the first case.  256
// workgroups that take tile after tile from counters, with the next tile's loads
// ahead of this one's stores, took 465 instead of 436 us, 64 groups of 1408 x
// 2048 from 8 bits: the registers do not hold both tiles.)
// 129 rows of 512 x 512 from 8 bits: 25 -> 17 us.
bool both(const LinearArgs& a, const Plan& dx, const Plan& dw) {
  return a.m && dx.shape == dw.shape && dx.shape != SHAPE_128 &&
         (dx.workgroups + dw.workgroups + div_up(a.n, 32) * a.groups + 16) * 512 <= kLaunchThreads;
}
hipError_t launch_both(const LinearArgs& a, const Plan& dx, const Plan& dw, const DbPlan& db, hipStream_t s) {
  BothPlan p{};
  p.dx = dx.tiles;
  p.dw = dw_tiles(dw);
  p.db = db;
  p.db_eights = static_cast<int>(div_up(int64_t{db.cols} * db.groups, 8));
  p.dw_eights = static_cast<int>(div_up(dw.workgroups, 8));
  const dim3 grid(static_cast<unsigned>(8 * (p.db_eights + p.dw_eights) + dx.workgroups)), block(512);
  if (dx.shape == SHAPE_256) {
    switch (a.x8.kind) {
      case ROW_E4M3: hipLaunchKernelGGL((linear_both_kernel<ROW_E4M3>), grid, block, 0, s, a, p); break;
      case ROW_E5M2: hipLaunchKernelGGL((linear_both_kernel<ROW_E5M2>), grid, block, 0, s, a, p); break;
      default: hipLaunchKernelGGL((linear_both_kernel<ROW_BF16>), grid, block, 0, s, a, p); break;
    }
    launch_join<MODE_DX, 256, 256>(a, dx, s);
    launch_join<MODE_DW, 256, 256>(a, dw, s);
  } else {
    hipLaunchKernelGGL(linear_narrow_both_kernel, grid, block, 0, s, a, p);
    launch_join<MODE_DX, 64, 64>(a, dx, s);
    launch_join<MODE_DW, 64, 64>(a, dw, s);
  }
  return hipGetLastError();
}

// Whether an x in 8 bits is brought to BF16 in the workspace: the 256 x 256 tile
// of dw reads the codes itself (64 groups of 1408 x 2048, 24571 rows: 454 -> 434
// to 440 us, 16384 x 2816 x 2048 378 -> 376, and no copy of x in memory); the
// others are fed by direct loads alone.
bool x_by_workspace(const LinearArgs& a, const Plan& dw) { return a.x8.kind != ROW_BF16 && dw.shape != SHAPE_256; }

// The backward's tiles, and the places in its workspace of dz, the column sums
// of the row tiles, the parts of dx and of dw, and x in BF16 where it is kept in 8
// bits.
struct BackwardPlan {
  Plan dx, dw;
  int64_t dz_at, sums_at, dx_at, dw_at, x_at, total;
};
BackwardPlan plan_backward(const LinearArgs& a, bool dx, bool dw, bool db) {
  BackwardPlan p{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  if (dx && a.m) p.dx = plan_rows(a, MODE_DX);
  if (dw) p.dw = plan_dw(a);
  p.dz_at = take(a.act != LIN_NONE && (dx || dw) ? a.m * a.n * 2 : 0);
  p.sums_at = take(db ? row_tiles(a, dz_rows(a)) * a.n * 4 : 0);
  p.dx_at = take(p.dx.partial_bytes);
  p.dw_at = take(p.dw.partial_bytes);
  p.x_at = take(dw && x_by_workspace(a, p.dw) ? a.m * a.k * 2 : 0);
  p.total = at;
  return p;
}

template <typename T>
LinearPlan packed(const T& t, int64_t workspace) {
  static_assert(sizeof(T) <= sizeof(LinearPlan::detail) && std::is_trivially_copyable_v<T>, "the form that callers pass on");
  LinearPlan p{workspace, {}};
  memcpy(p.detail, &t, sizeof(T));
  return p;
}
template <typename T>
T unpacked(const LinearPlan& p) {
  T t;
  memcpy(&t, p.detail, sizeof(T));
  return t;
}

}  // namespace

LinearPlan plan_linear(const LinearArgs& a) {
  const ForwardPlan f = plan_forward(a);
  return packed(f, f.tiles.partial_bytes);
}
LinearPlan plan_linear_backward(const LinearArgs& a, bool dx, bool dw, bool db) {
  const BackwardPlan p = plan_backward(a, dx, dw, db);
  return packed(p, p.total);
}

// Many workgroups (groups): small ones of 4 waves and 32 columns, four to a
// compute unit; few: 8 waves share a narrow tile, which reads fewer rows of
// weights but deeper.  Measured, 64 groups of 2048 x 1408, 96 rows: 87 us
// with 8 waves, 76 (4.8 TB/s of weights) with 4; one group of 8192 x 8192,
// one row: 26 us (5.1 TB/s) with 8 waves, 34 with 4; 2816 x 2048 from the
// last-level cache: 5.2 and 7.7 us.
hipError_t launch_few_rows(const LinearArgs& a, hipStream_t s) {
  const int64_t tiles = div_up(a.n, 16);
  if (tiles * a.groups >= 2048)
    hipLaunchKernelGGL((linear_few_rows_kernel<2, 4, 4>), dim3(static_cast<unsigned>(div_up(tiles, 2)), static_cast<unsigned>(a.groups)),
                       dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((linear_few_rows_kernel<1, 8, 8>), dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.groups)), dim3(512), 0,
                       s, a);
  return hipGetLastError();
}

hipError_t launch_linear(const LinearArgs& args, const LinearPlan& plan, hipStream_t s) {
  LinearArgs a = args;
  const ForwardPlan p = unpacked<ForwardPlan>(plan);
  if (a.m == 0) return hipSuccess;
  if (p.few == a.m) return launch_few_rows(a, s);
  a.dx_partial = static_cast<float*>(a.workspace);
  a.m -= p.few;
  const hipError_t e = launch_tiles<MODE_FORWARD>(a, p.tiles, s);
  if (e != hipSuccess || !p.few) return e;
  const int64_t n_out = a.act == LIN_SWIGLU ? a.n / 2 : a.n, m = a.m;
  a.m = p.few;
  a.x += m * a.k;
  a.y = static_cast<uint8_t*>(a.y) + m * n_out * (a.out_f32 ? 4 : 2);
  if (a.c) a.c += m * a.n;
  if (a.residual) a.residual += m * n_out;
  return launch_few_rows(a, s);
}

namespace {
template <int CK, bool X8>
void launch_dz(const LinearArgs& a, const DzPlan& p, dim3 grid, hipStream_t s) {
  switch (a.act) {
    case LIN_SWIGLU: hipLaunchKernelGGL((linear_dz_kernel<LIN_SWIGLU, CK, X8>), grid, dim3(256), 0, s, a, p); break;
    case LIN_SRELU: hipLaunchKernelGGL((linear_dz_kernel<LIN_SRELU, CK, X8>), grid, dim3(256), 0, s, a, p); break;
    case LIN_GELU: hipLaunchKernelGGL((linear_dz_kernel<LIN_GELU, CK, X8>), grid, dim3(256), 0, s, a, p); break;
    default: hipLaunchKernelGGL((linear_dz_kernel<LIN_NONE, ROW_BF16, X8>), grid, dim3(256), 0, s, a, p); break;
  }
}
template <bool X8>
void launch_dz_kind(const LinearArgs& a, const DzPlan& p, dim3 grid, hipStream_t s) {
  switch (a.c_kind) {
    case ROW_E4M3: launch_dz<ROW_E4M3, X8>(a, p, grid, s); break;
    case ROW_E5M2: launch_dz<ROW_E5M2, X8>(a, p, grid, s); break;
    default: launch_dz<ROW_BF16, X8>(a, p, grid, s); break;
  }
}
}  // namespace

hipError_t launch_linear_backward(const LinearArgs& args, const LinearPlan& plan, hipStream_t s) {
  LinearArgs a = args;
  const BackwardPlan w = unpacked<BackwardPlan>(plan);
  uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
  const bool make_dz = a.act != LIN_NONE && (a.dx || a.dw) && a.m;
  const bool x8 = a.dw && x_by_workspace(a, w.dw);
  uint16_t* const dz = make_dz ? reinterpret_cast<uint16_t*>(ws + w.dz_at) : nullptr;
  float* const sums = a.db ? reinterpret_cast<float*>(ws + w.sums_at) : nullptr;
  uint16_t* const x = x8 ? reinterpret_cast<uint16_t*>(ws + w.x_at) : nullptr;
  const int rows = dz_rows(a);
  a.dz = make_dz ? dz : a.dy;
  a.dx_partial = reinterpret_cast<float*>(ws + w.dx_at);
  a.dw_partial = reinterpret_cast<float*>(ws + w.dw_at);
  hipError_t e = hipSuccess;
  if ((make_dz || a.db) && a.m) {
    const int64_t tiles = row_tiles(a, rows);
    const DzPlan p{dz, sums, x, rows, dz_cols(a)};
    dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(p.cols));
    if (x8) {
      grid.y += static_cast<unsigned>(div_up(div_up(a.m * a.k, kSavedChunk), tiles));
      launch_dz_kind<true>(a, p, grid, s);
    } else {
      launch_dz_kind<false>(a, p, grid, s);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else if (x8 && a.m && (e = launch_dequantise(a.x8, x, false, a.m, a.k, s)) != hipSuccess) {
    return e;
  }
  if (x8) {
    a.x = x;
    a.x8.kind = ROW_BF16;
  }
  // db by few row tiles a group: few threads a column, or most of them only wait
  // (64 groups of 2048 columns, 4 tiles each: 15 us with 16 threads, 5 with 2)
  DbPlan db{};
  if (a.db) {
    const int q = row_tiles(a, rows) <= 16 * static_cast<int64_t>(a.groups) ? 2 : 16;
    db = {sums, rows, q, static_cast<int>(div_up(a.n, 512 / q)), a.groups};
  }
  if (a.dx && a.dw && both(a, w.dx, w.dw)) return launch_both(a, w.dx, w.dw, db, s);
  if (a.db) {
    const dim3 grid(static_cast<unsigned>(db.cols), static_cast<unsigned>(db.groups));
    if (db.q == 2) hipLaunchKernelGGL((linear_db_kernel<2>), grid, dim3(512), 0, s, a, db);
    else hipLaunchKernelGGL((linear_db_kernel<16>), grid, dim3(512), 0, s, a, db);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.dx && a.m && (e = launch_tiles<MODE_DX>(a, w.dx, s)) != hipSuccess) return e;
  if (a.dw && (e = launch_tiles<MODE_DW>(a, w.dw, s)) != hipSuccess) return e;
  return e;
}

}  // namespace moegg
