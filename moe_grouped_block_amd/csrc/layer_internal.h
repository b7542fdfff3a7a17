// Internal interface between the C-ABI front of the layer operators
// (layer_api.cpp) and their HIP kernels (route.hip, exchange.hip,
// linear.hip, norm.hip, saved.hip).  Not installed, not part of the ABI.
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
constexpr int kMaxGroups = 64;

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
  int32_t groups;          // 1: none
  int32_t top_groups;
  bool group_sums;         // a group's score: its two largest keys added, else its largest
  uint32_t group_magic;    // expert e is in group (e magic) >> 22
  int32_t group_lanes;     // a group is so many whole lanes, or 0       [set by the launchers]
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

// ---- norm ------------------------------------------------------------------

constexpr int kMaxNormWidth = 32768;  // 16 waves of 4 pieces of 8 columns a lane

struct NormArgs {
  const void* x;            // (T, H) bf16 or fp32
  const void* residual;     // (T, H) in the stream's type, or null
  const float* weight;      // (H)
  void* h;                  // (T, H) in the stream's type: with a residual
  uint16_t* y;              // (T, H) bf16 or null
  uint8_t* codes;           // (T, H) in `kind`, MX kinds
  uint8_t* scales;
  const uint16_t* dy;       // (T, H) bf16                     [backward]
  const void* stored;       // (T, H) in the stream's type: h  [backward]
  const void* dh;           // the same, or null               [backward]
  void* dx;                 // the same, or null               [backward]
  float* dw;                // (H) or null                     [backward]
  float* partial;           // workspace (with dw): rows of dw's parts
  int64_t rows;
  int32_t width;
  int32_t kind;             // RowKind of the codes (ROW_BF16: y alone)
  bool x_f32;
  bool stream_f32;
  bool kplanes;
  double eps;
  double inverse_width;
};
int64_t rms_norm_threads(int64_t rows, int32_t width, bool stream_f32, int kind);
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
int64_t rms_norm_backward_workspace(int64_t rows, int32_t width);
hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s);

// ---- rows kept in 8 bits -----------------------------------------------------

struct SavedRows {
  const uint8_t* codes;     // (rows, width) E4M3 or E5M2
  const uint8_t* scales;    // (rows, width / 32), or (width / 128, rows, 4) planes
  int32_t kind;             // ROW_E4M3 | ROW_E5M2
  bool kplanes;
};
// codes and scales of x (bf16 or fp32); out (bf16 or fp32) of codes and scales
hipError_t launch_quantise(const void* x, bool x_f32, uint8_t* codes, uint8_t* scales, int kind, bool kplanes, int64_t rows,
                           int32_t width, hipStream_t s);
hipError_t launch_dequantise(const SavedRows& q, void* out, bool out_f32, int64_t rows, int32_t width, hipStream_t s);

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
  int32_t c_kind;           // RowKind of c: ROW_BF16, or 8 bits (c holds codes)
  uint8_t* c_sf;            // scales of an 8-bit c, (M, N / 32)
  SavedRows x8;             // x in 8 bits (kind ROW_BF16: none)    [backward]
};
// A call's workspace in bytes, and its tiles in linear.hip's own form: made once
// for the check of the workspace and the launch (a plan is 0.3 us, a small call 8).
struct LinearPlan {
  int64_t workspace;
  int64_t detail[20];
};
// They read the sizes, the types and whether there are offsets; no pointer is followed.
LinearPlan plan_linear(const LinearArgs& a);
LinearPlan plan_linear_backward(const LinearArgs& a, bool dx, bool dw, bool db);
hipError_t launch_linear(const LinearArgs& a, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_backward(const LinearArgs& a, const LinearPlan& plan, hipStream_t s);

}  // namespace moegg
