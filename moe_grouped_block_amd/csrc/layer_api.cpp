// C-ABI front of the layer operators (route, sort / dispatch / combine,
// linear): host-side validation and dispatch.  As in moegg_api.cpp every rule
// is checked before any HIP call, so a rejected call enqueues nothing.
#include "layer_internal.h"

#include <cmath>

using moegg::clear_error;
using moegg::set_error;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Null / misaligned among required and optional pointers.
struct Pointer {
  const char* name;
  const void* p;
  uintptr_t align;
  bool required;
};
template <int N>
moegg_status check_pointers(const Pointer (&ps)[N]) {
  for (const Pointer& q : ps)
    if (q.required && !q.p) return set_error(MOEGG_ERROR_INVALID_VALUE, "%s is required", q.name);
  for (const Pointer& q : ps)
    if (!aligned(q.p, q.align))
      return set_error(MOEGG_ERROR_MISALIGNED, "%s (%p) not %d-byte aligned", q.name, q.p, static_cast<int>(q.align));
  return MOEGG_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte (no byte, none shared).
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// No output shares a byte with an input or with another output.
struct Span {
  const char* name;
  const void* p;
  int64_t bytes;
};
template <int NI, int NO>
moegg_status check_apart(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Span& q : in)
      if (overlap(q.p, q.bytes, out[i].p, out[i].bytes))
        return set_error(MOEGG_ERROR_INVALID_VALUE, "%s and %s overlap", q.name, out[i].name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[j].p, out[j].bytes, out[i].p, out[i].bytes))
        return set_error(MOEGG_ERROR_INVALID_VALUE, "%s and %s overlap", out[j].name, out[i].name);
  }
  return MOEGG_OK;
}

moegg_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return set_error(MOEGG_ERROR_LAUNCH, "%s: %s", what, hipGetErrorString(e));
  clear_error();
  return MOEGG_OK;
}

// ---- route -------------------------------------------------------------------

moegg_status check_route(const moegg_route_problem* pp) {
  if (!pp) return set_error(MOEGG_ERROR_INVALID_VALUE, "problem must be non-NULL");
  const moegg_route_problem& p = *pp;
  if (p.num_tokens < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "num_tokens=%lld negative", (long long)p.num_tokens);
  if (p.num_experts < 1 || p.num_experts > moegg::kMaxExperts)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_experts=%d outside 1..%d", p.num_experts, moegg::kMaxExperts);
  if (p.top_k < 1 || p.top_k > p.num_experts)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "top_k=%d outside 1..num_experts=%d", p.top_k, p.num_experts);
  if (p.top_k > moegg::kMaxTopK)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "top_k=%d above %d", p.top_k, moegg::kMaxTopK);
  if (p.num_tokens > INT32_MAX / p.top_k)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_tokens=%lld x top_k=%d above 2^31-1", (long long)p.num_tokens, p.top_k);
  if (p.num_tokens * (p.num_experts > 256 ? 64 : 16) > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_tokens=%lld: more threads than a launch holds", (long long)p.num_tokens);
  if (p.dtype != MOEGG_DT_BF16 && p.dtype != MOEGG_DT_F32)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dtype=%d must be BF16 or F32", p.dtype);
  if (p.score != MOEGG_SCORE_SOFTMAX && p.score != MOEGG_SCORE_SIGMOID)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "score=%d must be SOFTMAX or SIGMOID", p.score);
  if (p.renormalise != 0 && p.renormalise != 1)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "renormalise=%d must be 0 or 1", p.renormalise);
  if (!std::isfinite(p.scale)) return set_error(MOEGG_ERROR_INVALID_VALUE, "scale must be finite");
  return MOEGG_OK;
}

int64_t logits_bytes(const moegg_route_problem& p) {
  return p.num_tokens * p.num_experts * (p.dtype == MOEGG_DT_BF16 ? 2 : 4);
}

moegg::RouteArgs route_args(const moegg_route_problem& p) {
  moegg::RouteArgs a{};
  a.tokens = p.num_tokens;
  a.experts = p.num_experts;
  a.top_k = p.top_k;
  a.bf16 = p.dtype == MOEGG_DT_BF16;
  a.softmax = p.score == MOEGG_SCORE_SOFTMAX;
  a.renormalise = p.renormalise != 0;
  a.scale = p.scale;
  return a;
}

// ---- sort and exchange ---------------------------------------------------------

moegg_status check_sort(const moegg_sort_problem* pp, int64_t* capacity) {
  if (!pp) return set_error(MOEGG_ERROR_INVALID_VALUE, "problem must be non-NULL");
  const moegg_sort_problem& p = *pp;
  if (p.num_tokens < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "num_tokens=%lld negative", (long long)p.num_tokens);
  if (p.num_experts < 1 || p.num_experts > moegg::kMaxExperts)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_experts=%d outside 1..%d", p.num_experts, moegg::kMaxExperts);
  if (p.top_k < 1) return set_error(MOEGG_ERROR_INVALID_VALUE, "top_k=%d must be positive", p.top_k);
  if (p.top_k > moegg::kMaxTopK)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "top_k=%d above %d", p.top_k, moegg::kMaxTopK);
  if (p.m_aligned < 1 || p.m_aligned > 65536)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "m_aligned=%d outside 1..65536", p.m_aligned);
  if (p.num_tokens > INT32_MAX / p.top_k)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_tokens=%lld x top_k=%d above 2^31-1", (long long)p.num_tokens, p.top_k);
  const int64_t slots = p.num_tokens * p.top_k;
  const int64_t filled = slots < p.num_experts ? slots : p.num_experts;    // experts with a row at most
  const int64_t rows = (slots + filled * (p.m_aligned - 1)) / p.m_aligned * p.m_aligned;
  if (rows > INT32_MAX)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "%lld padded rows: above 2^31-1", (long long)rows);
  *capacity = rows;
  return MOEGG_OK;
}

int64_t sort_workspace_bytes(const moegg_sort_problem& p) {
  const int32_t blocks = moegg::sort_blocks(p.num_tokens * p.top_k);
  return blocks > 1 ? static_cast<int64_t>(blocks) * p.num_experts * 4 : 0;
}

int row_kind(int dtype) {
  switch (dtype) {
    case MOEGG_DT_BF16: return moegg::ROW_BF16;
    case MOEGG_DT_E4M3: return moegg::ROW_E4M3;
    case MOEGG_DT_E5M2: return moegg::ROW_E5M2;
    case MOEGG_DT_E2M1X2: return moegg::ROW_E2M1;
    default: return -1;
  }
}

moegg_status check_exchange(const moegg_exchange_problem* pp) {
  if (!pp) return set_error(MOEGG_ERROR_INVALID_VALUE, "problem must be non-NULL");
  const moegg_exchange_problem& p = *pp;
  if (p.num_tokens < 0 || p.rows < 0)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_tokens=%lld rows=%lld negative", (long long)p.num_tokens, (long long)p.rows);
  if (p.top_k < 1) return set_error(MOEGG_ERROR_INVALID_VALUE, "top_k=%d must be positive", p.top_k);
  if (p.top_k > moegg::kMaxTopK)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "top_k=%d above %d", p.top_k, moegg::kMaxTopK);
  if (p.num_experts < 1 || p.num_experts > moegg::kMaxExperts)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_experts=%d outside 1..%d", p.num_experts, moegg::kMaxExperts);
  if (p.rows > INT32_MAX || p.num_tokens > INT32_MAX / p.top_k)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_tokens=%lld rows=%lld above 2^31-1", (long long)p.num_tokens, (long long)p.rows);
  const int kind = row_kind(p.dtype);
  if (kind < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "dtype=%d must be BF16, E4M3, E5M2 or E2M1X2", p.dtype);
  const int step = kind == moegg::ROW_BF16 ? 8 : kind == moegg::ROW_E2M1 ? 256 : 128;
  if (p.width < 1 || p.width % step != 0)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d: a positive multiple of %d needed for this row type", p.width, step);
  if (p.width > (1 << 20)) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d above 2^20", p.width);
  if (moegg::exchange_waves(p.num_tokens, p.rows, p.width) * 64 > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_tokens=%lld rows=%lld width=%d: more threads than a launch holds",
                     (long long)p.num_tokens, (long long)p.rows, p.width);
  if (p.sf_layout != MOEGG_SF_ROW_MAJOR && p.sf_layout != MOEGG_SF_KPLANES)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "sf_layout=%d must be ROW_MAJOR or KPLANES", p.sf_layout);
  return MOEGG_OK;
}

moegg::ExchangeArgs exchange_args(const moegg_exchange_problem& p) {
  moegg::ExchangeArgs a{};
  a.tokens = p.num_tokens;
  a.rows = p.rows;
  a.experts = p.num_experts;
  a.top_k = p.top_k;
  a.width = p.width;
  a.kind = row_kind(p.dtype);
  a.kplanes = p.sf_layout == MOEGG_SF_KPLANES;
  return a;
}

// Bytes of the rows in their type, and of their scales.
int64_t row_bytes(const moegg_exchange_problem& p) {
  const int64_t n = p.rows * p.width;
  return p.dtype == MOEGG_DT_BF16 ? 2 * n : p.dtype == MOEGG_DT_E2M1X2 ? n / 2 : n;
}

int64_t scale_bytes(const moegg_exchange_problem& p) { return p.rows * (p.width / 32); }
int64_t slot_bytes(const moegg_exchange_problem& p) { return p.num_tokens * p.top_k * 4; }

moegg_status check_scales(const moegg_exchange_problem& p, const uint8_t* sf) {
  const bool mx = p.dtype != MOEGG_DT_BF16;
  if (mx && !sf) return set_error(MOEGG_ERROR_INVALID_VALUE, "MX rows need sf");
  if (!mx && sf) return set_error(MOEGG_ERROR_INVALID_VALUE, "BF16 rows take no sf");
  return MOEGG_OK;
}

// ---- linear ----------------------------------------------------------------------

moegg_status check_linear(const moegg_linear_problem* pp) {
  if (!pp) return set_error(MOEGG_ERROR_INVALID_VALUE, "problem must be non-NULL");
  const moegg_linear_problem& p = *pp;
  if (p.m < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "m=%lld negative", (long long)p.m);
  // (the kernels count r, which may be m, in 32 bits up to two steps past its end)
  if (p.m > INT32_MAX - 1023) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "m=%lld above 2^31-1024", (long long)p.m);
  if (p.n <= 0 || p.k <= 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "n=%d k=%d must be positive", p.n, p.k);
  if (p.num_groups < 1 || p.num_groups > moegg::kMaxExperts)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_groups=%d outside 1..%d", p.num_groups, moegg::kMaxExperts);
  if (p.act != MOEGG_ACT_NONE && p.act != MOEGG_ACT_SWIGLU && p.act != MOEGG_ACT_SRELU && p.act != MOEGG_ACT_GELU)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "act=%d must be NONE, SWIGLU, SRELU or GELU", p.act);
  if (p.dtype != MOEGG_DT_BF16 && p.dtype != MOEGG_DT_F32)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dtype=%d must be BF16 or F32", p.dtype);
  if (p.act == MOEGG_ACT_SWIGLU && p.n % 64 != 0)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "SwiGLU needs n %% 64 == 0 (32-column pairs), n=%d", p.n);
  if (p.n % 8 != 0 || p.k % 8 != 0)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "n=%d k=%d: multiples of 8 needed", p.n, p.k);
  if (p.n > (1 << 20) || p.k > (1 << 20))
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "n=%d k=%d above 2^20", p.n, p.k);
  // Threads of the tiles of y, dx and dw: 512 for 64 x 64 (at most 64 columns),
  // else 256 for 128 x 128 at most
  const auto threads = [](int64_t row_tiles64, int64_t row_tiles128, int64_t cols) {
    return cols <= 64 ? row_tiles64 * 512 : row_tiles128 * (cols / 128 + 1) * 256;
  };
  const int64_t rows64 = p.m / 64 + p.num_groups + 1, rows128 = p.m / 128 + p.num_groups + 1;
  const int64_t dw64 = p.num_groups * int64_t{p.n / 64 + 1}, dw128 = p.num_groups * int64_t{p.n / 128 + 1};
  if (threads(rows64, rows128, p.n) > moegg::kLaunchThreads || threads(rows64, rows128, p.k) > moegg::kLaunchThreads ||
      threads(dw64, dw128, p.k) > moegg::kLaunchThreads || rows128 * 256 > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "m=%lld n=%d k=%d num_groups=%d: more threads than a launch holds",
                     (long long)p.m, p.n, p.k, p.num_groups);
  return MOEGG_OK;
}

moegg::LinearArgs linear_args(const moegg_linear_problem& p, const moegg_linear_args* pa) {
  moegg::LinearArgs a{};
  a.m = p.m;
  a.n = p.n;
  a.k = p.k;
  a.groups = p.num_groups;
  a.act = p.act == MOEGG_ACT_SWIGLU  ? moegg::LIN_SWIGLU
          : p.act == MOEGG_ACT_SRELU ? moegg::LIN_SRELU
          : p.act == MOEGG_ACT_GELU  ? moegg::LIN_GELU
                                     : moegg::LIN_NONE;
  a.out_f32 = p.dtype == MOEGG_DT_F32;
  if (pa) {
    a.x = static_cast<const uint16_t*>(pa->x);
    a.w = static_cast<const uint16_t*>(pa->w);
    a.bias = pa->bias;
    a.residual = static_cast<const uint16_t*>(pa->residual);
    a.offsets = pa->offsets;
    a.y = pa->y;
    a.c = static_cast<uint16_t*>(pa->c);
    a.dy = static_cast<const uint16_t*>(pa->dy);
    a.dx = static_cast<uint16_t*>(pa->dx);
    a.dw = pa->dw;
    a.db = pa->db;
    a.workspace = pa->workspace;
    a.workspace_bytes = pa->workspace_bytes;
  }
  return a;
}

int64_t w_bytes(const moegg_linear_problem& p) { return int64_t{p.num_groups} * p.n * p.k * 2; }

moegg_status check_linear_pointers(const moegg_linear_problem& p, const moegg_linear_args& a, int64_t workspace) {
  const Pointer ps[] = {{"x", a.x, 16, false},   {"w", a.w, 16, false},     {"residual", a.residual, 16, false},
                        {"y", a.y, 16, false},   {"c", a.c, 16, false},     {"dy", a.dy, 16, false},
                        {"dx", a.dx, 16, false}, {"dw", a.dw, 16, false},   {"workspace", a.workspace, 16, false},
                        {"bias", a.bias, 4, false}, {"offsets", a.offsets, 4, false}, {"db", a.db, 4, false}};
  const moegg_status st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (!a.offsets && p.num_groups != 1)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_groups=%d needs offsets", p.num_groups);
  if (workspace > 0 && (!a.workspace || a.workspace_bytes < workspace))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "workspace of %lld bytes needed, %lld given", (long long)workspace,
                     (long long)(a.workspace ? a.workspace_bytes : 0));
  return MOEGG_OK;
}

}  // namespace

extern "C" {

moegg_status moegg_route(const moegg_route_problem* problem, const void* logits, const float* bias, int32_t* ids,
                         float* weights, void* stream) {
  moegg_status st = check_route(problem);
  if (st != MOEGG_OK) return st;
  const bool any = problem->num_tokens > 0;
  const Pointer ps[] = {{"logits", logits, 16, any}, {"ids", ids, 4, any}, {"weights", weights, 4, any}, {"bias", bias, 4, false}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "route");
  const int64_t chosen = problem->num_tokens * problem->top_k * 4;
  const Span in[] = {{"logits", logits, logits_bytes(*problem)}, {"bias", bias, int64_t{problem->num_experts} * 4}};
  const Span out[] = {{"ids", ids, chosen}, {"weights", weights, chosen}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  moegg::RouteArgs a = route_args(*problem);
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  return launched(moegg::launch_route(a, static_cast<hipStream_t>(stream)), "route kernel");
}

moegg_status moegg_route_backward(const moegg_route_problem* problem, const void* logits, const int32_t* ids,
                                  const float* dweights, void* dlogits, void* stream) {
  moegg_status st = check_route(problem);
  if (st != MOEGG_OK) return st;
  const bool any = problem->num_tokens > 0;
  const Pointer ps[] = {{"logits", logits, 16, any}, {"dlogits", dlogits, 16, any}, {"ids", ids, 4, any}, {"dweights", dweights, 4, any}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "route");
  const int64_t chosen = problem->num_tokens * problem->top_k * 4;
  const Span in[] = {{"logits", logits, logits_bytes(*problem)}, {"ids", ids, chosen}, {"dweights", dweights, chosen}};
  const Span out[] = {{"dlogits", dlogits, logits_bytes(*problem)}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  moegg::RouteArgs a = route_args(*problem);
  a.logits = logits;
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  return launched(moegg::launch_route_backward(a, static_cast<hipStream_t>(stream)), "route backward kernel");
}

int64_t moegg_sort_rows(const moegg_sort_problem* problem) {
  int64_t rows = 0;
  return check_sort(problem, &rows) == MOEGG_OK ? rows : -1;
}

int64_t moegg_sort_workspace(const moegg_sort_problem* problem) {
  int64_t rows = 0;
  return check_sort(problem, &rows) == MOEGG_OK ? sort_workspace_bytes(*problem) : -1;
}

moegg_status moegg_sort(const moegg_sort_problem* problem, const int32_t* ids, const float* weights,
                        int32_t* padded_offsets, int32_t* row_of, int32_t* slot_of, float* prob, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  int64_t capacity = 0;
  moegg_status st = check_sort(problem, &capacity);
  if (st != MOEGG_OK) return st;
  const moegg_sort_problem& p = *problem;
  if (p.rows < capacity || p.rows > INT32_MAX)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "rows=%lld outside %lld..2^31-1", (long long)p.rows, (long long)capacity);
  const bool any = p.num_tokens > 0;
  const Pointer ps[] = {{"padded_offsets", padded_offsets, 4, true}, {"ids", ids, 4, any}, {"row_of", row_of, 4, any},
                        {"slot_of", slot_of, 4, p.rows > 0}, {"weights", weights, 4, false}, {"prob", prob, 4, false},
                        {"workspace", workspace, 16, false}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (any && (weights != nullptr) != (prob != nullptr))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "weights and prob come together");
  const int64_t need = sort_workspace_bytes(p);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "workspace of %lld bytes needed", (long long)need);
  const int64_t slot_bytes = p.num_tokens * p.top_k * 4;
  const Span in[] = {{"ids", ids, slot_bytes}, {"weights", weights, slot_bytes}};
  const Span out[] = {{"padded_offsets", padded_offsets, int64_t{p.num_experts} * 4}, {"row_of", row_of, slot_bytes},
                      {"slot_of", slot_of, p.rows * 4}, {"prob", prob, p.rows * 4}, {"workspace", workspace, need}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  moegg::SortArgs a{};
  a.ids = ids;
  a.weights = weights;
  a.padded_offsets = padded_offsets;
  a.row_of = row_of;
  a.slot_of = slot_of;
  a.prob = prob;
  a.hist = static_cast<int32_t*>(workspace);
  a.slots = p.num_tokens * p.top_k;
  a.rows = p.rows;
  a.experts = p.num_experts;
  a.m_aligned = p.m_aligned;
  a.blocks = moegg::sort_blocks(a.slots);
  a.chunk = moegg::sort_chunk(a.slots);
  return launched(moegg::launch_sort(a, static_cast<hipStream_t>(stream)), "sort kernel");
}

moegg_status moegg_dispatch(const moegg_exchange_problem* problem, const void* x, const int32_t* row_of,
                            const int32_t* slot_of, const int32_t* padded_offsets, void* out, uint8_t* sf,
                            void* stream) {
  moegg_status st = check_exchange(problem);
  if (st != MOEGG_OK) return st;
  const moegg_exchange_problem& p = *problem;
  const bool any = p.num_tokens > 0 && p.rows > 0;
  const Pointer ps[] = {{"x", x, 16, any}, {"out", out, 16, any}, {"sf", sf, 16, false}, {"row_of", row_of, 4, any},
                        {"slot_of", slot_of, 4, any}, {"padded_offsets", padded_offsets, 4, any}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (any && (st = check_scales(p, sf)) != MOEGG_OK) return st;
  const Span in[] = {{"x", x, p.num_tokens * p.width * 2}, {"row_of", row_of, slot_bytes(p)}, {"slot_of", slot_of, p.rows * 4},
                     {"padded_offsets", padded_offsets, int64_t{p.num_experts} * 4}};
  const Span outs[] = {{"out", out, row_bytes(p)}, {"sf", sf, scale_bytes(p)}};
  if (any && (st = check_apart(in, outs)) != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "dispatch");
  moegg::ExchangeArgs a = exchange_args(p);
  a.x = static_cast<const uint16_t*>(x);
  a.row_of = row_of;
  a.slot_of = slot_of;
  a.offsets = padded_offsets;
  a.rows_out = static_cast<uint8_t*>(out);
  a.scales = sf;
  return launched(moegg::launch_dispatch(a, static_cast<hipStream_t>(stream)), "dispatch kernel");
}

moegg_status moegg_combine(const moegg_exchange_problem* problem, const void* rows_in, const int32_t* row_of,
                           const float* weights, const void* residual, void* y, void* stream) {
  moegg_status st = check_exchange(problem);
  if (st != MOEGG_OK) return st;
  const moegg_exchange_problem& p = *problem;
  if (p.dtype != MOEGG_DT_BF16) return set_error(MOEGG_ERROR_INVALID_VALUE, "combine reads BF16 rows");
  const bool any = p.num_tokens > 0;
  const Pointer ps[] = {{"rows_in", rows_in, 16, any && p.rows > 0}, {"y", y, 16, any}, {"residual", residual, 16, false},
                        {"row_of", row_of, 4, any}, {"weights", weights, 4, false}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  const int64_t y_bytes = p.num_tokens * p.width * 2;
  const Span in[] = {{"rows_in", rows_in, row_bytes(p)}, {"row_of", row_of, slot_bytes(p)}, {"weights", weights, slot_bytes(p)}};
  const Span out[] = {{"y", y, y_bytes}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (residual != y && overlap(residual, y_bytes, y, y_bytes))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and y overlap without being the same tensor");
  if (!any) return launched(hipSuccess, "combine");
  moegg::ExchangeArgs a = exchange_args(p);
  a.rows_in = static_cast<const uint16_t*>(rows_in);
  a.row_of = row_of;
  a.weights = weights;
  a.residual = static_cast<const uint16_t*>(residual);
  a.y = static_cast<uint16_t*>(y);
  return launched(moegg::launch_combine(a, static_cast<hipStream_t>(stream)), "combine kernel");
}

moegg_status moegg_combine_backward(const moegg_exchange_problem* problem, const void* dy, const int32_t* row_of,
                                    const int32_t* slot_of, const int32_t* padded_offsets, const void* rows_in,
                                    const float* weights, void* out, uint8_t* sf, float* dweights, void* stream) {
  moegg_status st = check_exchange(problem);
  if (st != MOEGG_OK) return st;
  const moegg_exchange_problem& p = *problem;
  // (without rows every slot is a dropped one: dweights is still written)
  const bool rows = p.num_tokens > 0 && p.rows > 0, any = rows || (p.num_tokens > 0 && dweights);
  const Pointer ps[] = {{"dy", dy, 16, any}, {"out", out, 16, rows}, {"sf", sf, 16, false}, {"rows_in", rows_in, 16, false},
                        {"row_of", row_of, 4, any}, {"slot_of", slot_of, 4, rows},
                        {"padded_offsets", padded_offsets, 4, rows}, {"weights", weights, 4, false},
                        {"dweights", dweights, 4, false}};
  st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (rows && (st = check_scales(p, sf)) != MOEGG_OK) return st;
  if (rows && (rows_in != nullptr) != (dweights != nullptr))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "rows_in and dweights come together");
  const Span in[] = {{"dy", dy, p.num_tokens * p.width * 2}, {"row_of", row_of, slot_bytes(p)}, {"slot_of", slot_of, p.rows * 4},
                     {"padded_offsets", padded_offsets, int64_t{p.num_experts} * 4},
                     {"rows_in", rows_in, p.rows * p.width * 2}, {"weights", weights, slot_bytes(p)}};
  const Span outs[] = {{"out", out, row_bytes(p)}, {"sf", sf, scale_bytes(p)}, {"dweights", dweights, slot_bytes(p)}};
  if (any && (st = check_apart(in, outs)) != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "combine backward");
  moegg::ExchangeArgs a = exchange_args(p);
  a.x = static_cast<const uint16_t*>(dy);
  a.rows_in = static_cast<const uint16_t*>(rows_in);
  a.weights = weights;
  a.row_of = row_of;
  a.slot_of = slot_of;
  a.offsets = padded_offsets;
  a.rows_out = static_cast<uint8_t*>(out);
  a.scales = sf;
  a.dweights = dweights;
  return launched(moegg::launch_combine_backward(a, static_cast<hipStream_t>(stream)), "combine backward kernel");
}

moegg_status moegg_unsort(const float* rows_values, const int32_t* row_of, float* values, int64_t num_slots,
                          int64_t rows, void* stream) {
  if (num_slots < 0 || rows < 0 || num_slots > INT32_MAX || rows > INT32_MAX)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_slots=%lld rows=%lld outside 0..2^31-1", (long long)num_slots, (long long)rows);
  const bool any = num_slots > 0;
  const Pointer ps[] = {{"rows_values", rows_values, 4, any && rows > 0}, {"row_of", row_of, 4, any}, {"values", values, 4, any}};
  moegg_status st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  const Span in[] = {{"rows_values", rows_values, rows * 4}, {"row_of", row_of, num_slots * 4}};
  const Span out[] = {{"values", values, num_slots * 4}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "unsort");
  return launched(moegg::launch_unsort(rows_values, row_of, values, num_slots, rows, static_cast<hipStream_t>(stream)),
                  "unsort kernel");
}

int64_t moegg_linear_workspace(const moegg_linear_problem* problem) {
  if (check_linear(problem) != MOEGG_OK) return -1;
  return moegg::linear_workspace(linear_args(*problem, nullptr));
}

int64_t moegg_linear_backward_workspace(const moegg_linear_problem* problem, int32_t want) {
  if (check_linear(problem) != MOEGG_OK) return -1;
  return moegg::linear_backward_workspace(linear_args(*problem, nullptr), want & 1, want & 2, want & 4);
}

moegg_status moegg_linear(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream) {
  moegg_status st = check_linear(problem);
  if (st != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_linear_problem& p = *problem;
  const moegg::LinearArgs a = linear_args(p, args);
  const bool any = p.m > 0;
  if (any && (!a.x || !a.w || !a.y)) return set_error(MOEGG_ERROR_INVALID_VALUE, "x, w and y are required");
  if (a.dy || a.dx || a.dw || a.db)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dy, dx, dw and db are for moegg_linear_backward");
  const int64_t workspace = moegg::linear_workspace(a);
  st = check_linear_pointers(p, *args, workspace);
  if (st != MOEGG_OK) return st;
  const int64_t n_out = p.act == MOEGG_ACT_SWIGLU ? p.n / 2 : p.n;
  const int64_t y_bytes = p.m * n_out * (a.out_f32 ? 4 : 2);
  const int64_t c_bytes = p.m * p.n * 2;
  const Span in[] = {{"x", a.x, p.m * p.k * 2}, {"w", a.w, w_bytes(p)}, {"bias", a.bias, int64_t{p.num_groups} * p.n * 4},
                     {"offsets", a.offsets, int64_t{p.num_groups} * 4}};
  const Span out[] = {{"y", a.y, y_bytes}, {"c", a.c, c_bytes}, {"workspace", a.workspace, workspace}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (overlap(a.residual, p.m * n_out * 2, a.c, c_bytes) || overlap(a.residual, p.m * n_out * 2, a.workspace, workspace))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and c or the workspace overlap");
  if (overlap(a.residual, p.m * n_out * 2, a.y, y_bytes) && (a.out_f32 || static_cast<const void*>(a.residual) != a.y))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and y overlap without being the same BF16 tensor");
  if (!any) return launched(hipSuccess, "linear");
  return launched(moegg::launch_linear(a, static_cast<hipStream_t>(stream)), "linear kernel");
}

moegg_status moegg_linear_backward(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream) {
  moegg_status st = check_linear(problem);
  if (st != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_linear_problem& p = *problem;
  const moegg::LinearArgs a = linear_args(p, args);
  const bool any = p.m > 0;
  if (a.bias || a.residual || a.y)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "bias, residual and y are for moegg_linear");
  // (without rows dx has no elements, and its pointer may be NULL)
  const bool none = !a.dx && !a.dw && !a.db;
  if (any && none) return set_error(MOEGG_ERROR_INVALID_VALUE, "one of dx, dw and db is required");
  if (any && !a.dy) return set_error(MOEGG_ERROR_INVALID_VALUE, "dy is required");
  if (any && a.act != moegg::LIN_NONE && !a.c) return set_error(MOEGG_ERROR_INVALID_VALUE, "this activation's gradient needs c");
  if (any && a.dx && !a.w) return set_error(MOEGG_ERROR_INVALID_VALUE, "dx needs w");
  if (any && a.dw && !a.x) return set_error(MOEGG_ERROR_INVALID_VALUE, "dw needs x");
  const int64_t workspace = moegg::linear_backward_workspace(a, a.dx, a.dw, a.db);
  st = check_linear_pointers(p, *args, workspace);
  if (st != MOEGG_OK) return st;
  const int64_t n_out = p.act == MOEGG_ACT_SWIGLU ? p.n / 2 : p.n;
  const Span in[] = {{"x", a.x, p.m * p.k * 2}, {"w", a.w, w_bytes(p)}, {"dy", a.dy, p.m * n_out * 2}, {"c", a.c, p.m * p.n * 2},
                     {"offsets", a.offsets, int64_t{p.num_groups} * 4}};
  const Span out[] = {{"dx", a.dx, p.m * p.k * 2}, {"dw", a.dw, w_bytes(p) * (a.out_f32 ? 2 : 1)},
                      {"db", a.db, int64_t{p.num_groups} * p.n * 4}, {"workspace", a.workspace, workspace}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (none) return launched(hipSuccess, "linear backward");
  return launched(moegg::launch_linear_backward(a, static_cast<hipStream_t>(stream)), "linear backward kernel");
}

}  // extern "C"
