// The tile kernel of linear and its gradients (BF16 operands, fp32 sums).
//
//   out(p, q) = sum over r of P(p, r) Q(q, r)
//
//   forward   P = x rows (m),   Q = w rows (n),    r = k   both contiguous along r
//   dx        P = dz rows (m),  Q = w columns (k), r = n   Q contiguous along q
//   dw        P = dz columns (n), Q = x columns (k), r = m   both contiguous along p / q
//
// One workgroup computes a BP x BQ tile in steps of 64 r through two stages of
// LDS, or of 32 r through four.  Each step's two operand tiles come into LDS by
// direct global -> LDS loads of 16 bytes a lane.  An operand contiguous along r
// lies in LDS as rows of the step's r (128 or 64 bytes) and is read with 16-byte
// reads; one contiguous along its rows lies as lines of its rows, one for every
// r, and is read with the transposing 8-byte reads (ds_read_b64_tr_b16: 16 lanes
// read 4 lines of 16 elements, and each gets one column's 4), so no operand is
// ever transposed in memory.  Both images are swizzled in 16-byte chunks so that
// a read's lanes meet all banks once.
//
// The Q tile is the matrix instruction's first operand: a lane then holds
// one row p of the output and runs of 4 contiguous columns.
#pragma once

#include "grouped_gemm.h"
#include "layer_internal.h"

namespace moegg {
namespace {

constexpr int kR = 64;                 // r per step of the kernels with two stages, and unit of the parts of r
constexpr int kRingR = 32;             // r per step of those with a ring of four

// What a lane reads past the end of r: zeros.
__device__ const uint32_t kZeros[4] = {0, 0, 0, 0};

// Swizzle of line r of an image whose lines hold CH 16-byte chunks: the slot
// of chunk c is c ^ line_swizzle(r).  A transposing read covers 4 lines of 64
// bytes in 32 lanes; lines are 256 bytes or more apart in multiples of the 64
// banks (CH >= 16), or half of that (CH = 8).
template <int CH>
__device__ __forceinline__ int line_swizzle(int r) {
  return (CH >= 16 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) ^ (((r >> 3) & 1) << 1);
}

// One operand's tile of ROWS rows and R of r: staging and fragments.
template <bool ALONG_R, int ROWS, int R, int NW>
struct TileOperand {
  static constexpr int BYTES = ROWS * R * 2;
  static constexpr int RC = R / 8;                 // chunks per row (along r)
  static constexpr int NI = BYTES / 1024 / NW;     // 1 KB loads per wave and step
  static constexpr int CH = ROWS / 8;              // chunks per line (rows contiguous)
  static_assert(NI * NW * 1024 == BYTES, "tile split over the waves");
  const uint8_t* base;                             // wave-uniform: the step's first byte
  uint32_t off[NI];                                // per lane
  int64_t advance;                                 // bytes per step

  // Image row (ALONG_R) or line of load j, and its source chunk.
  __device__ static __forceinline__ int image_row(int wave, int j, int lane) {
    return ((wave * NI + j) * 64 + lane) / (ALONG_R ? RC : CH);
  }
  // Slot of chunk c of a row of r: rows of 128 (64) bytes fill the 64 banks in
  // pairs (fours), and a read takes one chunk of 16 consecutive rows.
  __device__ static __forceinline__ int row_swizzle(int row) { return R == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
  __device__ static __forceinline__ int image_chunk(int wave, int j, int lane) {
    const int r = image_row(wave, j, lane);
    return ALONG_R ? (lane % RC) ^ row_swizzle(r) : (lane % CH) ^ line_swizzle<CH>(r);
  }
  // Tile of rows from i0 on (up to n), from r0 on; rows past the last one
  // repeat it (their results are not stored).
  __device__ __forceinline__ void init(const uint16_t* src, int64_t ld, int64_t i0, int64_t n, int64_t r0, int wave,
                                       int lane) {
    if constexpr (ALONG_R) {
      base = reinterpret_cast<const uint8_t*>(src + i0 * ld + r0);
      advance = R * 2;
      const int last = static_cast<int>(min(n - i0, int64_t{256})) - 1;
#pragma unroll
      for (int j = 0; j < NI; ++j)
        off[j] = static_cast<uint32_t>(min(image_row(wave, j, lane), last)) * static_cast<uint32_t>(ld * 2) +
                 image_chunk(wave, j, lane) * 16;
    } else {
      base = reinterpret_cast<const uint8_t*>(src + r0 * ld + i0);
      advance = R * ld * 2;
      const int last = static_cast<int>(min(n - i0, int64_t{256})) - 8;
#pragma unroll
      for (int j = 0; j < NI; ++j)
        off[j] = static_cast<uint32_t>(image_row(wave, j, lane)) * static_cast<uint32_t>(ld * 2) +
                 min(image_chunk(wave, j, lane) * 8, last) * 2;
    }
  }
  __device__ __forceinline__ void load(uint8_t* lds, int wave, int j) const {
    dma16(at(base, off[j]), lds + (wave * NI + j) * 1024);
  }
  // The last step of a ragged r: `left` of its r exist.
  __device__ __forceinline__ void load_tail(uint8_t* lds, int wave, int lane, int j, int left) const {
    const int r = ALONG_R ? image_chunk(wave, j, lane) * 8 : image_row(wave, j, lane);
    const uint8_t* src = r < left ? at(base, off[j]) : reinterpret_cast<const uint8_t*>(kZeros);
    dma16(src, lds + (wave * NI + j) * 1024);
  }

  // Per-lane byte offsets of the fragments of B blocks of 32 rows from tb on,
  // B a power of two and tb a multiple of 32 B.  Along r an offset belongs to a
  // window of 16 r and the block is a constant more; along the rows it is the
  // other way round (the swizzle does not move with the window).
  template <int B>
  struct Frags {
    static constexpr int N = ALONG_R ? R / 16 : B;
    uint32_t off[N];
    __device__ __forceinline__ void init(int tb, int lane) {
      if constexpr (ALONG_R) {
        const int row = tb + (lane & 31), sw = row_swizzle(row);
#pragma unroll
        for (int k = 0; k < N; ++k) off[k] = row * (R * 2) + (((2 * k + (lane >> 5)) ^ sw) * 16);
      } else {
        const int q = lane >> 4, line = (q >> 1) * 8 + ((lane >> 2) & 3);
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int chunk = tb / 8 + 4 * b + (q & 1) * 2 + ((lane & 3) >> 1);
          off[b] = line * (ROWS * 2) + (chunk ^ line_swizzle<CH>(line)) * 16 + (lane & 1) * 8;
        }
      }
    }
    // computed once, not again at every use
    __device__ __forceinline__ void keep() {
#pragma unroll
      for (int i = 0; i < N; ++i) asm volatile("" : "+v"(off[i]));
    }
    // Block b, window k: lane l holds row tb + 32 b + l % 32, r 16 k + 8 (l / 32) + [0, 8).
    __device__ __forceinline__ v4u read(const uint8_t* lds, int b, int k) const {
      if constexpr (ALONG_R) {
        return *reinterpret_cast<const v4u*>(lds + off[k] + b * (32 * R * 2));
      } else {
        typedef short v4s __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4s lds4;
        lds4* const p = (lds4*)(lds + off[b] + k * (16 * ROWS * 2));
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + ROWS);     // 4 lines on (8 bytes a step)
        return __builtin_bit_cast(v4u, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  };
};

enum LinearMode : int { MODE_FORWARD = 0, MODE_DX = 1, MODE_DW = 2 };

// Rows [begin, end) of group g, inside [0, m] whatever the offsets hold.
__device__ __forceinline__ void group_rows(const LinearArgs& a, int g, int64_t& begin, int64_t& end) {
  begin = 0;
  end = a.m;
  if (a.offsets) {
    begin = g ? a.offsets[g - 1] : 0;
    end = a.offsets[g];
    begin = min(max(begin, int64_t{0}), a.m);
    end = min(max(end, begin), a.m);
  }
}

// Row tiles of all groups at most (and exactly, without offsets).
template <int BM>
__host__ __device__ __forceinline__ int64_t most_row_tiles(const LinearArgs& a) {
  return (a.m + BM - 1) / BM + (a.groups > 1 ? a.groups - 1 : 0);
}

// Tiles of BM rows of every group (a tile holds rows of one group); the
// groups run along the lanes, 64 at a time.  Offsets that decrease name rows
// several times: the tiles that the launch has no place for are left out.
template <int BM>
__device__ __forceinline__ int count_row_tiles(const LinearArgs& a, int lane) {
  if (!a.offsets) return static_cast<int>(most_row_tiles<BM>(a));
  int64_t sum = 0;
  for (int g = lane; g < a.groups; g += 64) {
    int64_t b, e;
    group_rows(a, g, b, e);
    sum += (e - b + BM - 1) / BM;
  }
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  return __builtin_amdgcn_readfirstlane(static_cast<int>(min(sum, most_row_tiles<BM>(a))));
}
// Row tile mt: its group, first row and the end of the group's rows.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const LinearArgs& a, int mt, int lane, int& g, int64_t& row0, int64_t& end) {
  if (!a.offsets) {
    g = 0;
    row0 = static_cast<int64_t>(mt) * BM;
    end = a.m;
    return row0 < end;
  }
  int before = 0;
  for (int g0 = 0; g0 < a.groups; g0 += 64) {
    int64_t b = 0, e = 0;
    if (g0 + lane < a.groups) group_rows(a, g0 + lane, b, e);
    const int tiles = static_cast<int>((e - b + BM - 1) / BM);
    int scan = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(scan, d);
      if (lane >= d) scan += y;
    }
    const uint64_t past = __ballot(before + scan > mt);
    if (past) {
      const int l = __builtin_ctzll(past);
      g = __builtin_amdgcn_readfirstlane(g0 + l);
      const int first = before + __builtin_amdgcn_readlane(scan, l) - __builtin_amdgcn_readlane(tiles, l);
      const int bl = __builtin_amdgcn_readlane(static_cast<int>(b), l);
      row0 = bl + static_cast<int64_t>(mt - first) * BM;
      end = __builtin_amdgcn_readlane(static_cast<int>(e), l);
      return true;
    }
    before += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

// Workgroup w of `total` tiles -> tile.  Workgroups go round-robin over the 8
// XCDs (each with its own L2), so each pass of 256 gives every XCD 32
// consecutive tiles (the last pass an eighth of what is left).
__device__ __forceinline__ int tile_of_workgroup(int w, int total) {
  const int pass = w & ~255, rem = min(total - pass, 256), i = w - pass;
  const int xcd = i & 7, j = i >> 3;
  return pass + xcd * (rem >> 3) + min(xcd, rem & 7) + j;
}
// Tile -> (row tile, column tile): bands of 8 row tiles, rows fastest, so that
// consecutive tiles share operands.
__device__ __forceinline__ void tile_position(int t, int rows, int cols, int& rt, int& ct) {
  const int band = t / (8 * cols), in = t - band * 8 * cols;
  const int height = min(8, rows - 8 * band);
  ct = in / height;
  rt = 8 * band + in - ct * height;
}

// 16-byte aligned or not, 4 floats.
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));

// Rows of a 32-row block of output through the wave's LDS scratch, in whole
// W-byte segments: lane (row l32, half hi) holds bytes [32 b + 16 hi, + 16) of
// its row in q[b].  Rows from `rows` on and bytes from `valid` on are not stored.
template <int W>
__device__ __forceinline__ void store_block(uint8_t* base, int64_t pitch, const v4u* q, uint8_t* lds, int lane, int rows,
                                            int valid) {
  constexpr int CPR = W / 16;
  auto slot = [](int r, int c) __attribute__((always_inline)) {
    return W == 128 ? c ^ ((r >> 1) & 7) : c ^ ((r >> 2) & 3);
  };
  const int l32 = lane & 31, hi = lane >> 5;
  wave_sync_lds();
#pragma unroll
  for (int b = 0; b < W / 32; ++b) *reinterpret_cast<v4u*>(lds + l32 * W + slot(l32, 2 * b + hi) * 16) = q[b];
  wave_sync_lds();
  const int c = lane % CPR;
  v4u v[W / 32];
#pragma unroll
  for (int k = 0; k < W / 32; ++k) {
    const int r = k * (64 / CPR) + lane / CPR;
    v[k] = *reinterpret_cast<const v4u*>(lds + r * W + slot(r, c) * 16);
  }
#pragma unroll
  for (int k = 0; k < W / 32; ++k) {
    const int r = k * (64 / CPR) + lane / CPR;
    if (r < rows && c * 16 < valid) *reinterpret_cast<v4u*>(base + r * pitch + c * 16) = v[k];
  }
  wave_sync_lds();
}

// gelu(z) = z / 2 (1 + tanh u) = z sigmoid(2 u), u = c (z + a z^3)
constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
__device__ __forceinline__ float gelu_f(float z) {
  return z * sigmoid_f(2.0f * kGeluC * z * (1.0f + kGeluA * z * z));
}
// relu(z), where a NaN stays one (fmaxf(z, 0) is 0 for it)
__device__ __forceinline__ float relu_f(float z) { return z < 0.0f ? 0.0f : z; }
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// How a launch covers the tiles (tile counts on the host, see choose()).
// Tiles [0, first) have a workgroup each; each later one has `parts`, which
// share r and leave their sums in the workspace, (parts, tiles - first, BP,
// BQ) fp32, for a join.  With groups whose rows the host does not know
// (tiles < 0) there is a workgroup for every tile there may be.
struct TilePlan {
  int tiles, first, parts;
};

// What a workgroup computes: rows [row0, row_end) (up to its tile's), columns
// from col0 on, r in [r0, r1), of group g; `slot`: where its part goes, or -1.
struct LinearTile {
  int g, col0, slot;
  int64_t row0, row_end, r0, r1;
};

template <int MODE>
__device__ __forceinline__ int out_columns(const LinearArgs& a) { return MODE == MODE_FORWARD ? a.n : a.k; }

// Where the parts of a product go.
template <int MODE>
__device__ __forceinline__ float* partials(const LinearArgs& a) { return MODE == MODE_DW ? a.dw_partial : a.dx_partial; }

// Group, rows and columns of tile i.
template <int MODE, int BP, int BQ>
__device__ __forceinline__ bool place(const LinearArgs& a, int i, int row_tiles, int lane, LinearTile& t) {
  const int col_tiles = (out_columns<MODE>(a) + BQ - 1) / BQ;
  int rt, ct;
  if constexpr (MODE == MODE_DW) {
    t.g = i / (row_tiles * col_tiles);
    tile_position(i - t.g * row_tiles * col_tiles, row_tiles, col_tiles, rt, ct);
    t.row0 = static_cast<int64_t>(rt) * BP;
    t.row_end = a.n;
  } else {
    tile_position(i, row_tiles, col_tiles, rt, ct);
    if (!find_row_tile<BP>(a, rt, lane, t.g, t.row0, t.row_end)) return false;
  }
  t.col0 = ct * BQ;
  return true;
}

template <int MODE, int BP, int BQ>
__device__ __forceinline__ bool locate(const LinearArgs& a, const TilePlan& p, int w, int lane, LinearTile& t) {
  const int row_tiles = MODE == MODE_DW ? (a.n + BP - 1) / BP : count_row_tiles<BP>(a, lane);
  int i = w, part = -1;
  if (p.tiles < 0) {
    const int total = row_tiles * ((out_columns<MODE>(a) + BQ - 1) / BQ);
    if (w >= total) return false;
    i = tile_of_workgroup(w, total);
  } else if (w < p.first) {
    i = tile_of_workgroup(w, p.first);
  } else {
    const int split = p.tiles - p.first, j = w - p.first;
    part = j / split;
    i = p.first + tile_of_workgroup(j - part * split, split);
  }
  t.slot = part < 0 ? -1 : part * (p.tiles - p.first) + i - p.first;
  if (!place<MODE, BP, BQ>(a, i, row_tiles, lane, t)) return false;
  t.r0 = 0;
  t.r1 = MODE == MODE_FORWARD ? a.k : a.n;
  if constexpr (MODE == MODE_DW) group_rows(a, t.g, t.r0, t.r1);
  if (part >= 0) {
    const int64_t steps = (t.r1 - t.r0 + kR - 1) / kR;
    const int64_t lo = steps * part / p.parts, hi = steps * (part + 1) / p.parts;
    t.r1 = min(t.r1, t.r0 + hi * kR);
    t.r0 = min(t.r1, t.r0 + lo * kR);
  }
  return true;
}

// A wave's accumulators to its place in the workspace: 32 TM rows from row on
// of the tile, 64 columns from col on.
template <int BP, int BQ, int TM, int TN>
__device__ __forceinline__ void store_part(float* partial, v16f (&acc)[TM][TN], int slot, int row, int col,
                                           uint8_t* scratch, int lane) {
  float* const base = partial + static_cast<int64_t>(slot) * (BP * BQ) + row * BQ + col;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      v4u v[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        v[b] = v4u{__float_as_uint(acc[i][j][4 * b]), __float_as_uint(acc[i][j][4 * b + 1]),
                   __float_as_uint(acc[i][j][4 * b + 2]), __float_as_uint(acc[i][j][4 * b + 3])};
      store_block<128>(reinterpret_cast<uint8_t*>(base + i * 32 * BQ + 32 * j), BQ * 4, v, scratch, lane, 32, 128);
    }
}

// A wave's accumulators to memory: rows [row, row + 32 TM) of group g up to
// row_end, 64 columns from ncol on, through 4 KB of LDS scratch.
template <int MODE, int TM, int TN>
__device__ __forceinline__ void store_output(const LinearArgs& a, v16f (&acc)[TM][TN], int g, int64_t row, int64_t row_end,
                                             int ncol, uint8_t* scratch, int lane) {
  const int l32 = lane & 31, hi = lane >> 5;
  const int cols = out_columns<MODE>(a);
  if (ncol >= cols) return;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t rb = row + i * 32;                        // first row of the block
    const int rows = static_cast<int>(min(row_end - rb, int64_t{32}));
    if (rows <= 0) break;
    if constexpr (MODE != MODE_FORWARD) {
      const int64_t r = (MODE == MODE_DW ? static_cast<int64_t>(g) * a.n : 0) + rb;
      if (MODE == MODE_DW && a.out_f32) {
        float* const base = static_cast<float*>(a.dw) + r * cols + ncol;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          v4u v[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v[b] = v4u{__float_as_uint(acc[i][j][4 * b]), __float_as_uint(acc[i][j][4 * b + 1]),
                       __float_as_uint(acc[i][j][4 * b + 2]), __float_as_uint(acc[i][j][4 * b + 3])};
          store_block<128>(reinterpret_cast<uint8_t*>(base + 32 * j), static_cast<int64_t>(cols) * 4, v, scratch, lane, rows,
                           (cols - ncol - 32 * j) * 4);
        }
      } else {
        uint16_t* const base = (MODE == MODE_DW ? static_cast<uint16_t*>(a.dw) : a.dx) + r * cols + ncol;
        v4u v[4];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = acc[i][j][e];
          bf16_pieces(f, v + 2 * j);
        }
        store_block<128>(reinterpret_cast<uint8_t*>(base), static_cast<int64_t>(cols) * 2, v, scratch, lane, rows,
                         (cols - ncol) * 2);
      }
    } else {
      // z = sum + bias, c = bf16(z)
      float z[TN][16];
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int n = ncol + 32 * j + 8 * b + 4 * hi;
          v4f_any v{};
          if (a.bias && n < a.n) v = *reinterpret_cast<const v4f_any*>(a.bias + static_cast<int64_t>(g) * a.n + n);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[j][4 * b + e] = acc[i][j][4 * b + e] + v[e];
        }
      if (a.c) {
        v4u v[4];
#pragma unroll
        for (int j = 0; j < TN; ++j) bf16_pieces(z[j], v + 2 * j);
        store_block<128>(reinterpret_cast<uint8_t*>(a.c + rb * a.n + ncol), static_cast<int64_t>(a.n) * 2, v, scratch, lane,
                         rows, (a.n - ncol) * 2);
      }
      // y = act(z): TO blocks of 32 columns from column ycol on
      const bool pair = a.act == LIN_SWIGLU;
      const int n_out = pair ? a.n / 2 : a.n, ycol = pair ? ncol / 2 : ncol;
      if (pair) {
#pragma unroll
        for (int e = 0; e < 16; ++e) z[0][e] = z[0][e] * (z[1][e] * sigmoid_f(z[1][e]));
      } else if (a.act == LIN_GELU) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) z[j][e] = gelu_f(z[j][e]);
      } else if (a.act == LIN_SRELU) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v = relu_f(z[j][e]);
            z[j][e] = v * v;
          }
      }
      if (a.residual) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          if (j && pair) break;
          v4u u[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int n = ycol + 32 * j + 16 * b + 8 * hi;
            u[b] = v4u{};
            if (n < n_out && l32 < rows) u[b] = *reinterpret_cast<const v4u*>(a.residual + (rb + l32) * n_out + n);
          }
          v2u w[4];
          unpack_bf16(u, w);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            z[j][4 * b] += bf_lo(w[b].x);
            z[j][4 * b + 1] += bf_hi(w[b].x);
            z[j][4 * b + 2] += bf_lo(w[b].y);
            z[j][4 * b + 3] += bf_hi(w[b].y);
          }
        }
      }
      if (a.out_f32) {
        float* const base = static_cast<float*>(a.y) + rb * n_out + ycol;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          if (j && pair) break;
          v4u v[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v[b] = v4u{__float_as_uint(z[j][4 * b]), __float_as_uint(z[j][4 * b + 1]), __float_as_uint(z[j][4 * b + 2]),
                       __float_as_uint(z[j][4 * b + 3])};
          store_block<128>(reinterpret_cast<uint8_t*>(base + 32 * j), static_cast<int64_t>(n_out) * 4, v, scratch, lane, rows,
                           (n_out - ycol - 32 * j) * 4);
        }
      } else {
        uint8_t* const base = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(a.y) + rb * n_out + ycol);
        v4u v[4];
        bf16_pieces(z[0], v);
        if (pair) {
          store_block<64>(base, static_cast<int64_t>(n_out) * 2, v, scratch, lane, rows, 64);
        } else {
          bf16_pieces(z[1], v + 2);
          store_block<128>(base, static_cast<int64_t>(n_out) * 2, v, scratch, lane, rows, (n_out - ycol) * 2);
        }
      }
    }
  }
}

// The forward's 128 x 128 tile, two stages of 64 r (see linear_ring_kernel).
template <int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ, 2) void linear_tile_kernel(LinearArgs a, TilePlan plan) {
  constexpr int NW = WP * WQ, TM = BP / WP / 32, TN = BQ / WQ / 32;
  using TP = TileOperand<true, BP, kR, NW>;
  using TQ = TileOperand<true, BQ, kR, NW>;
  static_assert(TN == 2, "a wave's columns are one pair of 32-column blocks");
  // one array per stage and operand: the compiler then sees that a stage's
  // loads do not touch what is being read
  __shared__ __attribute__((aligned(16))) uint8_t sP0[TP::BYTES], sP1[TP::BYTES], sQ0[TQ::BYTES], sQ1[TQ::BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;

  LinearTile t;
  if (!locate<MODE_FORWARD, BP, BQ>(a, plan, blockIdx.x, lane, t)) return;
  const int64_t wg = static_cast<int64_t>(t.g) * a.n * a.k;
  TP p;
  TQ q;
  p.init(a.x, a.k, t.row0, t.row_end, t.r0, wave, lane);
  q.init(a.w + wg, a.k, t.col0, a.n, t.r0, wave, lane);
  typename TP::template Frags<TM> fp;
  typename TQ::template Frags<TN> fq;
  fp.init(wp * (TM * 32), lane);
  fq.init(wq * (TN * 32), lane);

  // ---- the sum ----
  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v16f{};
  const int64_t span = t.r1 - t.r0;
  const int steps = static_cast<int>((span + kR - 1) / kR);
  const int tail = static_cast<int>(span - static_cast<int64_t>(steps - 1) * kR);   // r of the last step
  auto issue = [&](int s, uint8_t* lp, uint8_t* lq) __attribute__((always_inline)) {
    if (s >= steps - 1 && (s >= steps || tail < kR)) {
      const int left = s < steps ? tail : 0;
#pragma unroll
      for (int j = 0; j < TP::NI; ++j) p.load_tail(lp, wave, lane, j, left);
#pragma unroll
      for (int j = 0; j < TQ::NI; ++j) q.load_tail(lq, wave, lane, j, left);
    } else {
#pragma unroll
      for (int j = 0; j < TP::NI; ++j) p.load(lp, wave, j);
#pragma unroll
      for (int j = 0; j < TQ::NI; ++j) q.load(lq, wave, j);
    }
    p.base += p.advance;
    q.base += q.advance;
  };
  auto compute = [&](const uint8_t* lp, const uint8_t* lq) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < kR / 16; ++kk) {
      v8bf vq[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) vq[j] = __builtin_bit_cast(v8bf, fq.read(lq, j, kk));
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const v8bf vp = __builtin_bit_cast(v8bf, fp.read(lp, i, kk));
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vq[j], vp, acc[i][j], 0, 0, 0);
      }
    }
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    wait_vmcnt<0>();
    __syncthreads();
  };
  // Steps go in pairs, so that the loop has one exit and names its buffers
  // statically; an odd last step is followed by one of zeros.
  if (steps > 0) {
    issue(0, sP0, sQ0);
    arrive();
    for (int s = 0; s < steps; s += 2) {
      issue(s + 1, sP1, sQ1);
      compute(sP0, sQ0);
      arrive();
      if (s + 2 < steps) issue(s + 2, sP0, sQ0);
      compute(sP1, sQ1);
      arrive();
    }
  }

  // ---- the output ----
  uint8_t* const scratch = (wave & 1 ? sP1 : sP0) + (wave >> 1) * 4096;
  static_assert(TP::BYTES >= (NW + 1) / 2 * 4096, "scratch of the waves");
  if (t.slot >= 0) store_part<BP, BQ>(partials<MODE_FORWARD>(a), acc, t.slot, wp * (TM * 32), wq * 64, scratch, lane);
  else store_output<MODE_FORWARD>(a, acc, t.g, t.row0 + wp * (TM * 32), t.row_end, t.col0 + wq * 64, scratch, lane);
}

// The same tile in steps of 32 r through a ring of four stages: three stages
// are in flight, and a step has one barrier (behind it every wave has read the
// stage before, whose place stage s + 3 takes).  Measured against two stages
// of 64 r, 256 tiles of 2048^3: 28.7 -> 22 to 23.5 us; dw 2816 x 2048 over 4099
// rows (352 tiles) 70 -> 60; but the forward with 512 tiles, two workgroups to
// a compute unit, 55 -> 63: there both operands come in 64-byte pieces, and
// two workgroups hide the latency well enough.
template <int MODE, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ, 2) void linear_ring_kernel(LinearArgs a, TilePlan plan) {
  constexpr int NW = WP * WQ, TM = BP / WP / 32, TN = BQ / WQ / 32, R = kRingR;
  using TP = TileOperand<MODE != MODE_DW, BP, R, NW>;
  using TQ = TileOperand<MODE == MODE_FORWARD, BQ, R, NW>;
  constexpr int N = TP::NI + TQ::NI;
  static_assert(TN == 2, "a wave's columns are one pair of 32-column blocks");
  __shared__ __attribute__((aligned(16))) uint8_t sP0[TP::BYTES], sP1[TP::BYTES], sP2[TP::BYTES], sP3[TP::BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t sQ0[TQ::BYTES], sQ1[TQ::BYTES], sQ2[TQ::BYTES], sQ3[TQ::BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;

  LinearTile t;
  if (!locate<MODE, BP, BQ>(a, plan, blockIdx.x, lane, t)) return;
  const int64_t wg = static_cast<int64_t>(t.g) * a.n * a.k;
  TP p;
  TQ q;
  p.init(MODE == MODE_FORWARD ? a.x : a.dz, MODE == MODE_FORWARD ? a.k : a.n, t.row0, MODE == MODE_DW ? a.n : t.row_end, t.r0,
         wave, lane);
  q.init(MODE == MODE_DW ? a.x : a.w + wg, a.k, t.col0, MODE == MODE_FORWARD ? a.n : a.k, t.r0, wave, lane);
  typename TP::template Frags<TM> fp;
  typename TQ::template Frags<TN> fq;
  fp.init(wp * (TM * 32), lane);
  fq.init(wq * (TN * 32), lane);
  fp.keep();
  fq.keep();
  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v16f{};
  const int span = static_cast<int>(t.r1 - t.r0), full = span / R;
  // ANY: a stage that is ragged or past the end (zeros)
  auto issue = [&](auto any, int s, uint8_t* lp, uint8_t* lq) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TP::NI; ++j)
      if constexpr (decltype(any)::value) p.load_tail(lp, wave, lane, j, span - s * R);
      else p.load(lp, wave, j);
#pragma unroll
    for (int j = 0; j < TQ::NI; ++j)
      if constexpr (decltype(any)::value) q.load_tail(lq, wave, lane, j, span - s * R);
      else q.load(lq, wave, j);
    p.base += p.advance;
    q.base += q.advance;
  };
  auto step = [&](auto any, int s, const uint8_t* lp, const uint8_t* lq, uint8_t* next_p, uint8_t* next_q)
      __attribute__((always_inline)) {
    wait_vmcnt<2 * N>();                           // stage s (s + 1 and s + 2 are on their way)
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(any, s + 3, next_p, next_q);
#pragma unroll
    for (int kk = 0; kk < R / 16; ++kk) {
      v8bf vq[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) vq[j] = __builtin_bit_cast(v8bf, fq.read(lq, j, kk));
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const v8bf vp = __builtin_bit_cast(v8bf, fp.read(lp, i, kk));
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vq[j], vp, acc[i][j], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);            // this stage read before the next barrier
  };
  if (span > 0) {
    const std::true_type any{};
    const std::false_type plain{};
    auto four = [&](auto any, int s) __attribute__((always_inline)) {
      step(any, s, sP0, sQ0, sP3, sQ3);
      step(any, s + 1, sP1, sQ1, sP0, sQ0);
      step(any, s + 2, sP2, sQ2, sP1, sQ1);
      step(any, s + 3, sP3, sQ3, sP2, sQ2);
    };
    issue(any, 0, sP0, sQ0);
    issue(any, 1, sP1, sQ1);
    issue(any, 2, sP2, sQ2);
    int s = 0;
    for (; s + 6 < full; s += 4) four(plain, s);
    for (; s * R < span; s += 4) four(any, s);
    wait_vmcnt<0>();
    __syncthreads();
  }
  uint8_t* const scratch = (wave & 1 ? sP1 : sP0) + (wave >> 1) * 4096;
  static_assert(TP::BYTES >= (NW + 1) / 2 * 4096, "scratch of the waves");
  if (t.slot >= 0) store_part<BP, BQ>(partials<MODE>(a), acc, t.slot, wp * (TM * 32), wq * 64, scratch, lane);
  else store_output<MODE>(a, acc, t.g, t.row0 + wp * (TM * 32), t.row_end, t.col0 + wq * 64, scratch, lane);
}

// The 64 x 64 tile of small outputs (a router's product, some hundred rows):
// what counts is that every compute unit has a workgroup and each of them many
// bytes in flight.  Four pairs of waves share the tile's r, each with two
// stages of its own, and their sums meet in LDS: a quarter of the steps and no
// join.  Measured against 128 x 128 tiles (with their best parts of r): 256 x
// 2048 x 2048 15.0 -> 10.2 us, 1000 x 512 x 512 8.3 -> 6.1, 951 rows of 15
// groups of 392 x 2144 27.0 -> 17.9; with more tiles than compute units 128 x
// 128 wins (3311 x 288 x 1008, 260 tiles: 11.7 against 14.4).
template <int MODE>
__global__ __launch_bounds__(512, 2) void linear_narrow_kernel(LinearArgs a, TilePlan plan) {
  constexpr int G = 4, NW = 2;
  using TP = TileOperand<MODE != MODE_DW, 64, kR, NW>;
  using TQ = TileOperand<MODE == MODE_FORWARD, 64, kR, NW>;
  __shared__ __attribute__((aligned(16))) uint8_t sP0[G * TP::BYTES], sP1[G * TP::BYTES], sQ0[G * TQ::BYTES], sQ1[G * TQ::BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wave / NW, wp = wave % NW;

  LinearTile t;
  if (!locate<MODE, 64, 64>(a, plan, blockIdx.x, lane, t)) return;
  const int64_t wg = static_cast<int64_t>(t.g) * a.n * a.k;
  const int64_t steps = (t.r1 - t.r0 + kR - 1) / kR;
  const int64_t r0 = min(t.r1, t.r0 + steps * grp / G * kR), r1 = min(t.r1, t.r0 + steps * (grp + 1) / G * kR);
  const int span = static_cast<int>(r1 - r0), full = span / kR, most = static_cast<int>((steps + G - 1) / G);
  TP p;
  TQ q;
  p.init(MODE == MODE_FORWARD ? a.x : a.dz, MODE == MODE_FORWARD ? a.k : a.n, t.row0, MODE == MODE_DW ? a.n : t.row_end, r0, wp,
         lane);
  q.init(MODE == MODE_DW ? a.x : a.w + wg, a.k, t.col0, MODE == MODE_FORWARD ? a.n : a.k, r0, wp, lane);
  typename TP::template Frags<1> fp;
  typename TQ::template Frags<2> fq;
  fp.init(wp * 32, lane);
  fq.init(0, lane);
  v16f acc[1][2];
  acc[0][0] = acc[0][1] = v16f{};
  auto issue = [&](int s, uint8_t* lp, uint8_t* lq) __attribute__((always_inline)) {
    lp += grp * TP::BYTES;
    lq += grp * TQ::BYTES;
    if (s < full) {
#pragma unroll
      for (int j = 0; j < TP::NI; ++j) p.load(lp, wp, j);
#pragma unroll
      for (int j = 0; j < TQ::NI; ++j) q.load(lq, wp, j);
    } else {
#pragma unroll
      for (int j = 0; j < TP::NI; ++j) p.load_tail(lp, wp, lane, j, span - s * kR);
#pragma unroll
      for (int j = 0; j < TQ::NI; ++j) q.load_tail(lq, wp, lane, j, span - s * kR);
    }
    p.base += p.advance;
    q.base += q.advance;
  };
  auto compute = [&](const uint8_t* lp, const uint8_t* lq) __attribute__((always_inline)) {
    lp += grp * TP::BYTES;
    lq += grp * TQ::BYTES;
#pragma unroll
    for (int k = 0; k < kR / 16; ++k) {
      const v8bf vp = __builtin_bit_cast(v8bf, fp.read(lp, 0, k));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[0][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fq.read(lq, j, k)), vp, acc[0][j], 0, 0, 0);
    }
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    wait_vmcnt<0>();
    __syncthreads();
  };
  // steps in pairs, as in linear_tile_kernel; all pairs of waves take `most` of them
  if (most > 0) {
    issue(0, sP0, sQ0);
    arrive();
    for (int s = 0; s < most; s += 2) {
      issue(s + 1, sP1, sQ1);
      compute(sP0, sQ0);
      arrive();
      if (s + 2 < most) issue(s + 2, sP0, sQ0);
      compute(sP1, sQ1);
      arrive();
    }
  }
  // sums of pairs 1, 2, 3 to pair 0, added in that order
  static_assert(G * TP::BYTES >= 2 * NW * 8192, "two pairs' sums in each P image");
  auto place_of = [&](int from) { return (from < 3 ? sP0 + (from - 1) * (NW * 8192) : sP1) + wp * 8192 + lane * 16; };
  if (grp > 0) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<v4f*>(place_of(grp) + (j * 4 + b) * 1024) =
            v4f{acc[0][j][4 * b], acc[0][j][4 * b + 1], acc[0][j][4 * b + 2], acc[0][j][4 * b + 3]};
  }
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int from = 1; from < G; ++from)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const v4f v = *reinterpret_cast<const v4f*>(place_of(from) + (j * 4 + b) * 1024);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][j][4 * b + e] += v[e];
      }
  uint8_t* const scratch = sQ0 + wp * 4096;
  if (t.slot >= 0) store_part<64, 64>(partials<MODE>(a), acc, t.slot, wp * 32, 0, scratch, lane);
  else store_output<MODE>(a, acc, t.g, t.row0 + wp * 32, t.row_end, t.col0, scratch, lane);
}

// The 256 x 256 tile: 8 waves, 2 along p x 4 along q, each 128 x 64, on the
// ping-pong schedule of the grouped product.  A step of 32 r is two clusters:
// M reads the step's 12 fragments from LDS, C runs its 16 MFMAs.  The two
// waves of a SIMD (w and w + 4) run one cluster apart, so one issues MFMAs
// while the other reads.  Four stages of 32 KB ring through LDS: stage s + 3 is
// issued during C(s), into the place of stage s - 1, which both groups have
// read by then, and is waited for at the end of M(s + 2), four clusters later.
// Steps past the last read zeros, so the steps go in fours with one exit and
// every wave has the same loads in flight.
constexpr int kRingBytes = 256 * kRingR * 2;      // one operand, one stage
template <int MODE>
__device__ __forceinline__ void pingpong_tile(const LinearArgs& a, const TilePlan& plan, int w, uint8_t* const (&sp)[4],
                                              uint8_t* const (&sq)[4]) {
  constexpr int R = kRingR;
  using TP = TileOperand<MODE != MODE_DW, 256, R, 8>;
  using TQ = TileOperand<MODE == MODE_FORWARD, 256, R, 8>;
  constexpr int N = TP::NI + TQ::NI;
  static_assert(TP::NI == 2 && TQ::NI == 2 && TP::BYTES == kRingBytes && TQ::BYTES == kRingBytes, "loads per wave and stage");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave >> 2, wq = wave & 3;

  LinearTile t;
  if (!locate<MODE, 256, 256>(a, plan, w, lane, t)) return;
  const int64_t wg = static_cast<int64_t>(t.g) * a.n * a.k;
  TP p;
  TQ q;
  p.init(MODE == MODE_FORWARD ? a.x : a.dz, MODE == MODE_FORWARD ? a.k : a.n, t.row0, MODE == MODE_DW ? a.n : t.row_end, t.r0,
         wave, lane);
  q.init(MODE == MODE_DW ? a.x : a.w + wg, a.k, t.col0, MODE == MODE_FORWARD ? a.n : a.k, t.r0, wave, lane);
  typename TP::template Frags<4> ap;
  typename TQ::template Frags<2> aq;
  ap.init(wp * 128, lane);
  aq.init(wq * 64, lane);
  ap.keep();
  aq.keep();
  v16f acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v16f{};

  const int span = static_cast<int>(t.r1 - t.r0);
  const int full = span / R;
  struct Stage {
    uint8_t *p, *q;
  };
  const Stage st[4] = {{sp[0], sq[0]}, {sp[1], sq[1]}, {sp[2], sq[2]}, {sp[3], sq[3]}};
  // load j (0..3) of stage s (the bases run along); ANY: a stage that is
  // ragged or past the end
  auto issue = [&](auto any, int s, const Stage& d, int j) __attribute__((always_inline)) {
    if (j < TP::NI) {
      if constexpr (decltype(any)::value) p.load_tail(d.p, wave, lane, j, span - s * R);
      else p.load(d.p, wave, j);
      if (j == TP::NI - 1) p.base += p.advance;
    } else {
      if constexpr (decltype(any)::value) q.load_tail(d.q, wave, lane, j - TP::NI, span - s * R);
      else q.load(d.q, wave, j - TP::NI);
      if (j == N - 1) q.base += q.advance;
    }
  };
  auto sync = []() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](auto any, int s, const Stage& now, const Stage& next3) __attribute__((always_inline)) {
    v4u fq[2][2], fp[4][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) fq[j][k] = aq.read(now.q, j, k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) fp[i][k] = ap.read(now.p, i, k);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(fq[j][k]));
#pragma unroll
      for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(fp[i][k]));
    }
    wait_vmcnt<N>();                             // stage s + 1
    sync();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fq[j][k]),
                                                              __builtin_bit_cast(v8bf, fp[i][k]), acc[i][j], 0, 0, 0);
          const int m = k * 8 + i * 2 + j;
          if (m % 4 == 0) issue(any, s + 3, next3, m / 4);
        }
    // the MFMAs stay in their cluster
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[i][j]));
    sync();
  };
  if (span > 0) {
    const std::true_type any{};
    const std::false_type plain{};
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int j = 0; j < N; ++j) issue(any, s, st[s], j);
    wait_vmcnt<2 * N>();
    sync();
    if (wp) sync();
    int s = 0;
    for (; s + 6 < full; s += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) step(plain, s + i, st[i], st[(i + 3) & 3]);
    }
    for (; s * R < span; s += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) step(any, s + i, st[i], st[(i + 3) & 3]);
    }
    wait_vmcnt<0>();
    if (!wp) sync();
    sync();
  }
  uint8_t* const scratch = (wave < 4 ? sp[0] : sp[1]) + (wave & 3) * 4096;
  if (t.slot >= 0) store_part<256, 256>(partials<MODE>(a), acc, t.slot, wp * 128, wq * 64, scratch, lane);
  else store_output<MODE>(a, acc, t.g, t.row0 + wp * 128, t.row_end, t.col0 + wq * 64, scratch, lane);
}

// One LDS array per stage and operand (see linear_tile_kernel).
#define MOEGG_RING_STAGES                                                                                     \
  __shared__ __attribute__((aligned(16))) uint8_t sP0[kRingBytes], sP1[kRingBytes], sP2[kRingBytes], sP3[kRingBytes]; \
  __shared__ __attribute__((aligned(16))) uint8_t sQ0[kRingBytes], sQ1[kRingBytes], sQ2[kRingBytes], sQ3[kRingBytes]; \
  uint8_t* const sp[4] = {sP0, sP1, sP2, sP3};                                                                \
  uint8_t* const sq[4] = {sQ0, sQ1, sQ2, sQ3}

template <int MODE>
__global__ __launch_bounds__(512, 1) void linear_pingpong_kernel(LinearArgs a, TilePlan plan) {
  MOEGG_RING_STAGES;
  pingpong_tile<MODE>(a, plan, blockIdx.x, sp, sq);
}

// The tiles of dw and then of dx in one launch.  dw's workgroups are counted in
// eights (a workgroup's number modulo 8 stays its XCD).
struct BothPlan {
  TilePlan dx, dw;
  int dw_eights;
};
__global__ __launch_bounds__(512, 1) void linear_both_kernel(LinearArgs a, BothPlan p) {
  MOEGG_RING_STAGES;
  const int first_dx = 8 * p.dw_eights;
  const bool dw = static_cast<int>(blockIdx.x) < first_dx;
  const int w = blockIdx.x - (dw ? 0 : first_dx);
  if (dw) {
    if (w < p.dw.first + (p.dw.tiles - p.dw.first) * p.dw.parts) pingpong_tile<MODE_DW>(a, p.dw, w, sp, sq);
  } else if (p.dx.tiles < 0 || w < p.dx.first + (p.dx.tiles - p.dx.first) * p.dx.parts) {
    pingpong_tile<MODE_DX>(a, p.dx, w, sp, sq);
  }
}

}  // namespace
}  // namespace moegg
