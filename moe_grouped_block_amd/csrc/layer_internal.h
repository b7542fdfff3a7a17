// Internal interface between the C-ABI front of the layer operators
// (layer_api.cpp) and their HIP kernels (route.hip, exchange.hip,
// linear.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moegg.h"

namespace moegg {

// The calling thread's last error (moegg_last_error), kept in moegg_api.cpp.
__attribute__((format(printf, 2, 3))) moegg_status set_error(moegg_status st, const char* fmt, ...);
void clear_error();

// ---- route -----------------------------------------------------------------

constexpr int kMaxExperts = 1024;   // as the grouped product's num_groups
constexpr int kMaxTopK = 32;

struct RouteArgs {
  const void* logits;      // (T, E) fp32 or bf16
  const float* bias;       // (E) or null
  const float* dweights;   // (T, k)            [backward]
  int32_t* ids;            // (T, k)            read by the backward
  float* weights;          // (T, k)
  void* dlogits;           // (T, E)            [backward]
  int64_t tokens;
  int32_t experts;
  int32_t top_k;
  bool bf16;
  bool softmax;
  bool renormalise;
  float scale;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

// ---- exchange --------------------------------------------------------------

struct SortArgs {
  const int32_t* ids;       // (slots)
  const float* weights;     // (slots) or null
  int32_t* padded_offsets;  // (E)
  int32_t* row_of;          // (slots)
  int32_t* slot_of;         // (rows)
  float* prob;              // (rows) or null
  int32_t* hist;            // workspace: (blocks, E)
  int64_t slots;
  int64_t rows;
  int32_t experts;
  int32_t m_aligned;
  int32_t blocks;           // sort_blocks(slots)
  int32_t chunk;            // slots per block
};
// Slots per block and block count of the sort: one block (and one launch) up
// to kSortOne slots, then blocks of kSortChunk, and longer ones past 256 blocks
// (each block sums the counts of all blocks).
constexpr int kSortThreads = 512;
constexpr int kSortOne = 4096;
constexpr int kSortChunk = 1024;
constexpr int kSortMaxBlocks = 256;
inline int32_t sort_chunk(int64_t slots) {
  const int64_t even = slots <= kSortOne ? slots : (slots + kSortMaxBlocks - 1) / kSortMaxBlocks;
  const int64_t least = slots <= kSortOne ? 1 : kSortChunk;
  return static_cast<int32_t>(((even > least ? even : least) + kSortThreads - 1) / kSortThreads * kSortThreads);
}
inline int32_t sort_blocks(int64_t slots) {
  const int64_t c = sort_chunk(slots);
  return slots > c ? static_cast<int32_t>((slots + c - 1) / c) : 1;
}
hipError_t launch_sort(const SortArgs& a, hipStream_t s);

// A launch counts its threads in 32 bits; what would need more is refused.
constexpr int64_t kLaunchThreads = (int64_t{1} << 32) - 1024;
constexpr int kPadRows = 16;        // padding rows of one wave, see zero_padding()
// Waves of the largest of the exchange's launches.
inline int64_t exchange_waves(int64_t tokens, int64_t rows, int32_t width) {
  return tokens * ((width + 511) / 512) + (rows + kPadRows - 1) / kPadRows;
}

// Format of the sorted rows.
enum RowKind : int { ROW_BF16 = 0, ROW_E4M3 = 1, ROW_E5M2 = 2, ROW_E2M1 = 3 };

struct ExchangeArgs {
  const uint16_t* x;        // (T, H) bf16: x, dy
  const uint16_t* rows_in;  // (rows, H) bf16: the experts' outputs
  const float* weights;     // (T, k) or null
  const uint16_t* residual; // (T, H) or null
  const int32_t* row_of;    // (T, k)
  const int32_t* slot_of;   // (rows)
  const int32_t* offsets;   // (E)
  uint8_t* rows_out;        // (rows, H) in `kind`
  uint8_t* scales;          // MX kinds
  uint16_t* y;              // (T, H) bf16
  float* dweights;          // (T, k) or null
  int64_t tokens;
  int64_t rows;
  int32_t experts;
  int32_t top_k;
  int32_t width;
  int32_t kind;
  bool kplanes;
};
hipError_t launch_dispatch(const ExchangeArgs& a, hipStream_t s);
hipError_t launch_combine(const ExchangeArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t s);
// values[slot] = rows[row_of[slot]] (0 for a dropped slot)
hipError_t launch_unsort(const float* rows, const int32_t* row_of, float* values, int64_t slots, int64_t n_rows,
                         hipStream_t s);

// ---- linear ----------------------------------------------------------------

enum LinearAct : int { LIN_NONE = 0, LIN_SWIGLU = 1, LIN_SRELU = 2, LIN_GELU = 3 };

struct LinearArgs {
  const uint16_t* x;        // (M, K) bf16
  const uint16_t* w;        // (L, N, K) bf16
  const float* bias;        // (L, N) or null
  const uint16_t* residual; // (M, N_out) bf16 or null
  const int32_t* offsets;   // (L) group ends or null (one group: all rows)
  void* y;                  // (M, N_out) bf16 or fp32
  uint16_t* c;              // (M, N) bf16: written by the forward (or null), read by the backward
  const uint16_t* dy;       // (M, N_out) bf16   [backward]
  uint16_t* dx;             // (M, K) bf16 or null
  void* dw;                 // (L, N, K) bf16 or fp32, or null
  float* db;                // (L, N) or null
  void* workspace;
  int64_t workspace_bytes;
  const uint16_t* dz;       // (M, N) bf16: dy, or in the workspace    [set by the launchers]
  float* dx_partial;        // fp32 sums of the parts of r, in the workspace: of y or dx,
  float* dw_partial;        // and of dw
  int64_t m;
  int32_t n;
  int32_t k;
  int32_t groups;
  int32_t act;              // LinearAct
  bool out_f32;             // y (forward) or dw (backward) in fp32
};
// Bytes of workspace (pointers in `a` only say what is asked for).
int64_t linear_workspace(const LinearArgs& a);
int64_t linear_backward_workspace(const LinearArgs& a, bool dx, bool dw, bool db);
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_backward(const LinearArgs& a, hipStream_t s);

}  // namespace moegg
