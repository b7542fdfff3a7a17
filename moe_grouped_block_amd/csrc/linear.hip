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
#include <hip/hip_runtime.h>

#include "layer_internal.h"

namespace moegg {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float(static_cast<uint32_t>(u) << 16); }
__device__ __forceinline__ uint16_t to_bf(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// gelu(z) = z / 2 (1 + tanh u) = z sigmoid(2 u), u = c (z + a z^3)
__device__ __forceinline__ float act1(float z, int act) {
  if (act == LIN_SRELU) {
    const float r = fmaxf(z, 0.0f);
    return r * r;
  }
  if (act == LIN_GELU) return z * sigmoid(2.0f * kGeluC * z * (1.0f + kGeluA * z * z));
  return z;
}
__device__ __forceinline__ float dact1(float z, int act) {
  if (act == LIN_SRELU) return 2.0f * fmaxf(z, 0.0f);
  if (act == LIN_GELU) {
    z = fminf(fmaxf(z, -30.0f), 30.0f);          // s is 0 or 1 there: keeps 0 times z^3 from becoming NaN
    const float s = sigmoid(2.0f * kGeluC * z * (1.0f + kGeluA * z * z));
    return s + z * s * (1.0f - s) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
  }
  return 1.0f;
}

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

// Row tile `mt` of the groups' tiles of BM rows (a tile holds rows of one
// group): group, first row, end of the group's rows; false past the last.
template <int BM>
__device__ __forceinline__ bool find_tile(const LinearArgs& a, int64_t mt, int& g, int64_t& row0, int64_t& end) {
  if (!a.offsets) {
    g = 0;
    row0 = mt * BM;
    end = a.m;
    return row0 < end;
  }
  int64_t before = 0;
  for (g = 0; g < a.groups; ++g) {
    int64_t b;
    group_rows(a, g, b, end);
    const int64_t tiles = (end - b + BM - 1) / BM;
    if (mt < before + tiles) {
      row0 = b + (mt - before) * BM;
      return true;
    }
    before += tiles;
  }
  return false;
}

// acc[j] += P(p0 + wave's 32 rows, r) Q(q0 + 32 j + row, r) over r in [r0, r1).
// An operand is contiguous along r (element (i, r) at i ld + r) or along i
// (at r ld + i); rows from `n` on and r from r1 on count as zero.
constexpr int kBM = 128, kBN = 64, kBK = 32, kPitch = kBK + 8;
template <bool ALONG_I, int ROWS>
__device__ __forceinline__ void stage(uint16_t (*lds)[kPitch], const uint16_t* src, int64_t ld, int64_t i0, int64_t n,
                                      int64_t r0, int64_t r1) {
  if constexpr (!ALONG_I) {
    for (int p = threadIdx.x; p < ROWS * (kBK / 8); p += 256) {
      const int i = p / (kBK / 8), c = p % (kBK / 8) * 8;
      v4u u{};
      if (i0 + i < n && r0 + c < r1) u = *reinterpret_cast<const v4u*>(src + (i0 + i) * ld + r0 + c);
      *reinterpret_cast<v4u*>(&lds[i][c]) = u;
    }
  } else {
    for (int p = threadIdx.x; p < kBK * (ROWS / 8); p += 256) {
      const int r = p / (ROWS / 8), c = p % (ROWS / 8) * 8;
      v4u u{};
      if (r0 + r < r1 && i0 + c < n) u = *reinterpret_cast<const v4u*>(src + (r0 + r) * ld + i0 + c);
      for (int q = 0; q < 8; ++q) lds[c + q][r] = static_cast<uint16_t>(u[q / 2] >> (16 * (q & 1)));
    }
  }
}
template <bool P_ALONG_I, bool Q_ALONG_I>
__device__ __forceinline__ void product(const uint16_t* p, int64_t ldp, int64_t p0, int64_t np, const uint16_t* q,
                                        int64_t ldq, int64_t q0, int64_t nq, int64_t r0, int64_t r1, v16f* acc) {
  __shared__ __attribute__((aligned(16))) uint16_t sp[kBM][kPitch], sq[kBN][kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, hi = lane >> 5;
  for (int64_t r = r0; r < r1; r += kBK) {
    __syncthreads();
    stage<P_ALONG_I, kBM>(sp, p, ldp, p0, np, r, r1);
    stage<Q_ALONG_I, kBN>(sq, q, ldq, q0, nq, r, r1);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kBK; kk += 16) {
      const v8bf fp = *reinterpret_cast<const v8bf*>(&sp[wave * 32 + l32][kk + 8 * hi]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v8bf fq = *reinterpret_cast<const v8bf*>(&sq[32 * j + l32][kk + 8 * hi]);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fq, fp, acc[j], 0, 0, 0);
      }
    }
  }
}
// Accumulator element v of lane l: P row l % 32, Q row 8 (v / 4) + 4 (l / 32) + v % 4.
__device__ __forceinline__ int q_row(int v) { return 8 * (v / 4) + 4 * ((threadIdx.x >> 5) & 1) + v % 4; }

__global__ __launch_bounds__(256) void linear_kernel(LinearArgs a) {
  int g;
  int64_t row0, end;
  if (!find_tile<kBM>(a, blockIdx.y, g, row0, end)) return;
  const int n0 = blockIdx.x * kBN;
  v16f acc[2] = {};
  product<false, false>(a.x, a.k, row0, end, a.w + static_cast<int64_t>(g) * a.n * a.k, a.k, n0, a.n, 0, a.k, acc);
  const int64_t m = row0 + (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
  if (m >= end) return;
  const int n_out = a.act == LIN_SWIGLU ? a.n / 2 : a.n;
  for (int j = 0; j < 2; ++j)
    for (int v = 0; v < 16; ++v) {
      const int n = n0 + 32 * j + q_row(v);
      if (n >= a.n) continue;
      if (a.bias) acc[j][v] += a.bias[static_cast<int64_t>(g) * a.n + n];
      if (a.c) a.c[m * a.n + n] = to_bf(acc[j][v]);
    }
  for (int j = 0; j < 2; ++j)
    for (int v = 0; v < 16; ++v) {
      int n = n0 + 32 * j + q_row(v);
      if (n >= a.n) continue;
      float y;
      if (a.act == LIN_SWIGLU) {
        if (j) continue;
        y = acc[0][v] * (acc[1][v] * sigmoid(acc[1][v]));
        n = n0 / 2 + q_row(v);
      } else {
        y = act1(acc[j][v], a.act);
      }
      if (a.residual) y += bf(a.residual[m * n_out + n]);
      if (a.out_f32) static_cast<float*>(a.y)[m * n_out + n] = y;
      else static_cast<uint16_t*>(a.y)[m * n_out + n] = to_bf(y);
    }
}

// dz of row m, column n, in fp32.
__device__ __forceinline__ float dz_at(const LinearArgs& a, int64_t m, int n) {
  if (a.act == LIN_NONE) return bf(a.dy[m * a.n + n]);
  if (a.act == LIN_SWIGLU) {
    const int pair = n / 64, i = n % 32;
    const float d = bf(a.dy[m * (a.n / 2) + pair * 32 + i]);
    const float x = bf(a.c[m * a.n + pair * 64 + i]), q = bf(a.c[m * a.n + pair * 64 + 32 + i]);
    const float s = sigmoid(q);
    return n % 64 < 32 ? d * (q * s) : d * (x * s) * (1.0f + q * (1.0f - s));
  }
  return bf(a.dy[m * a.n + n]) * dact1(bf(a.c[m * a.n + n]), a.act);
}
__global__ __launch_bounds__(256) void dz_kernel(LinearArgs a, uint16_t* dz) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < a.m * a.n) dz[i] = to_bf(dz_at(a, i / a.n, static_cast<int>(i % a.n)));
}
__global__ __launch_bounds__(256) void db_kernel(LinearArgs a) {
  __shared__ float part[4][64];
  const int n = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6, g = blockIdx.y;
  int64_t begin, end;
  group_rows(a, g, begin, end);
  float sum = 0.0f;
  if (n < a.n)
    for (int64_t m = begin + q; m < end; m += 4) sum += dz_at(a, m, n);
  part[q][threadIdx.x & 63] = sum;
  __syncthreads();
  if (q == 0 && n < a.n) a.db[static_cast<int64_t>(g) * a.n + n] = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}
__global__ __launch_bounds__(256) void dx_kernel(LinearArgs a, const uint16_t* dz) {
  int g;
  int64_t row0, end;
  if (!find_tile<kBM>(a, blockIdx.y, g, row0, end)) return;
  const int k0 = blockIdx.x * kBN;
  v16f acc[2] = {};
  product<false, true>(dz, a.n, row0, end, a.w + static_cast<int64_t>(g) * a.n * a.k, a.k, k0, a.k, 0, a.n, acc);
  const int64_t m = row0 + (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
  if (m >= end) return;
  for (int j = 0; j < 2; ++j)
    for (int v = 0; v < 16; ++v) {
      const int k = k0 + 32 * j + q_row(v);
      if (k < a.k) a.dx[m * a.k + k] = to_bf(acc[j][v]);
    }
}
__global__ __launch_bounds__(256) void dw_kernel(LinearArgs a, const uint16_t* dz) {
  const int g = blockIdx.z;
  int64_t begin, end;
  group_rows(a, g, begin, end);
  const int n0 = blockIdx.y * kBM, k0 = blockIdx.x * kBN;
  v16f acc[2] = {};
  product<true, true>(dz, a.n, n0, a.n, a.x, a.k, k0, a.k, begin, end, acc);
  const int n = n0 + (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
  if (n >= a.n) return;
  for (int j = 0; j < 2; ++j)
    for (int v = 0; v < 16; ++v) {
      const int k = k0 + 32 * j + q_row(v);
      if (k >= a.k) continue;
      const int64_t at = (static_cast<int64_t>(g) * a.n + n) * a.k + k;
      if (a.out_f32) static_cast<float*>(a.dw)[at] = acc[j][v];
      else static_cast<uint16_t*>(a.dw)[at] = to_bf(acc[j][v]);
    }
}

unsigned div_up(int64_t a, int64_t b) { return static_cast<unsigned>((a + b - 1) / b); }
unsigned row_tiles(const LinearArgs& a) { return div_up(a.m, kBM) + (a.offsets ? a.groups : 0); }

}  // namespace

int64_t linear_workspace(const LinearArgs&) { return 0; }
int64_t linear_backward_workspace(const LinearArgs& a, bool dx, bool dw, bool) {
  return a.act != LIN_NONE && (dx || dw) ? a.m * a.n * 2 : 0;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  if (a.m == 0) return hipSuccess;
  hipLaunchKernelGGL(linear_kernel, dim3(div_up(a.n, kBN), row_tiles(a)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear_backward(const LinearArgs& a, hipStream_t s) {
  const uint16_t* dz = a.dy;
  if (a.act != LIN_NONE && a.m && (a.dx || a.dw)) {
    dz = static_cast<uint16_t*>(a.workspace);
    hipLaunchKernelGGL(dz_kernel, dim3(div_up(a.m * a.n, 256)), dim3(256), 0, s, a, static_cast<uint16_t*>(a.workspace));
  }
  if (a.db) hipLaunchKernelGGL(db_kernel, dim3(div_up(a.n, 64), a.groups), dim3(256), 0, s, a);
  if (a.dx && a.m) hipLaunchKernelGGL(dx_kernel, dim3(div_up(a.k, kBN), row_tiles(a)), dim3(256), 0, s, a, dz);
  if (a.dw) hipLaunchKernelGGL(dw_kernel, dim3(div_up(a.k, kBN), div_up(a.n, kBM), a.groups), dim3(256), 0, s, a, dz);
  return hipGetLastError();
}

}  // namespace moegg
