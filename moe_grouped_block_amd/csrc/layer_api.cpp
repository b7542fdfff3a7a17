// C-ABI front of the layer operators (route, sort / dispatch / combine,
// linear, norm, rows kept in 8 bits): host-side validation and dispatch.  As in moegg_api.cpp every rule
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
  a.groups = 1;
  return a;
}

moegg_status check_groups(const moegg_route_problem& p, const moegg_route_groups* pg) {
  if (!pg) return set_error(MOEGG_ERROR_INVALID_VALUE, "groups must be non-NULL");
  const moegg_route_groups& g = *pg;
  if (g.num_groups < 1 || p.num_experts % g.num_groups != 0)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_groups=%d does not divide num_experts=%d", g.num_groups, p.num_experts);
  if (g.num_groups > moegg::kMaxGroups)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "num_groups=%d above %d", g.num_groups, moegg::kMaxGroups);
  if (g.top_groups < 1 || g.top_groups > g.num_groups)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "top_groups=%d outside 1..num_groups=%d", g.top_groups, g.num_groups);
  if (g.best != 1 && g.best != 2) return set_error(MOEGG_ERROR_INVALID_VALUE, "best=%d must be 1 or 2", g.best);
  if (p.top_k > g.top_groups * (p.num_experts / g.num_groups))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "top_k=%d above the %d experts of %d groups", p.top_k,
                     g.top_groups * (p.num_experts / g.num_groups), g.top_groups);
  return MOEGG_OK;
}

moegg_status run_route(const moegg_route_problem* problem, const moegg_route_groups* groups, bool grouped, const void* logits,
                       const float* bias, int32_t* ids, float* weights, void* stream) {
  moegg_status st = check_route(problem);
  if (st != MOEGG_OK) return st;
  if (grouped && (st = check_groups(*problem, groups)) != MOEGG_OK) return st;
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
  if (grouped && groups->top_groups < groups->num_groups) {    // (of all groups: no choice)
    a.groups = groups->num_groups;
    a.top_groups = groups->top_groups;
    a.group_sums = groups->best == 2;
    // (e magic) >> 22 = e / size for every e < 1024: e size < 2^22
    a.group_magic = (1u << 22) / static_cast<uint32_t>(problem->num_experts / groups->num_groups) + 1;
  }
  return launched(moegg::launch_route(a, static_cast<hipStream_t>(stream)), "route kernel");
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

moegg::LinearArgs linear_args(const moegg_linear_problem& p, const moegg_linear_args* pa,
                              const moegg_linear_saved* saved = nullptr) {
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
  if (saved) {
    a.c_kind = row_kind(saved->c_dtype);
    a.c_sf = saved->c_sf;
    a.x8 = {static_cast<const uint8_t*>(pa ? pa->x : nullptr), saved->x_sf, row_kind(saved->x_dtype),
            saved->x_sf_layout == MOEGG_SF_KPLANES};
  }
  return a;
}

int64_t w_bytes(const moegg_linear_problem& p) { return int64_t{p.num_groups} * p.n * p.k * 2; }

// 8 bits, or BF16 (-1: neither).
int kept_kind(int dtype) {
  const int kind = row_kind(dtype);
  return kind == moegg::ROW_E2M1 ? -1 : kind;
}
int64_t kept_bytes(int kind, int64_t n) { return kind == moegg::ROW_BF16 ? 2 * n : n; }

moegg_status check_saved(const moegg_linear_problem& p, const moegg_linear_saved& s) {
  if (kept_kind(s.x_dtype) < 0 || kept_kind(s.c_dtype) < 0)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "x_dtype=%d c_dtype=%d must be BF16, E4M3 or E5M2", s.x_dtype, s.c_dtype);
  if (s.x_sf_layout != MOEGG_SF_ROW_MAJOR && s.x_sf_layout != MOEGG_SF_KPLANES)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "x_sf_layout=%d must be ROW_MAJOR or KPLANES", s.x_sf_layout);
  if (s.reserved != 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "reserved=%d must be 0", s.reserved);
  const bool x8 = s.x_dtype != MOEGG_DT_BF16, c8 = s.c_dtype != MOEGG_DT_BF16;
  const int step = s.x_sf_layout == MOEGG_SF_KPLANES ? 128 : 32;
  if (x8 && p.k % step != 0)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "k=%d: a multiple of %d needed for x in 8 bits", p.k, step);
  if (c8 && p.n % 32 != 0) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "n=%d: a multiple of 32 needed for c in 8 bits", p.n);
  if (!x8 && s.x_sf) return set_error(MOEGG_ERROR_INVALID_VALUE, "a BF16 x takes no x_sf");
  if (!c8 && s.c_sf) return set_error(MOEGG_ERROR_INVALID_VALUE, "a BF16 c takes no c_sf");
  // (x's way to BF16 shares a launch with dz)
  const int64_t dz = (p.m / 128 + p.num_groups + 1) * int64_t{p.n / 256 + 2} * 256;
  if (x8 && (p.m * p.k + 4095) / 4096 * 256 + dz > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "m=%lld k=%d: more threads than a launch holds", (long long)p.m, p.k);
  return MOEGG_OK;
}

moegg_status check_linear_pointers(const moegg_linear_problem& p, const moegg_linear_args& a, const moegg_linear_saved* saved,
                                   int64_t workspace) {
  const Pointer ps[] = {{"x", a.x, 16, false},   {"w", a.w, 16, false},     {"residual", a.residual, 16, false},
                        {"y", a.y, 16, false},   {"c", a.c, 16, false},     {"dy", a.dy, 16, false},
                        {"dx", a.dx, 16, false}, {"dw", a.dw, 16, false},   {"workspace", a.workspace, 16, false},
                        {"bias", a.bias, 4, false}, {"offsets", a.offsets, 4, false}, {"db", a.db, 4, false}};
  moegg_status st = check_pointers(ps);
  if (st != MOEGG_OK) return st;
  if (saved) {
    const Pointer sf[] = {{"x_sf", saved->x_sf, 16, false}, {"c_sf", saved->c_sf, 16, false}};
    if ((st = check_pointers(sf)) != MOEGG_OK) return st;
  }
  if (!a.offsets && p.num_groups != 1)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "num_groups=%d needs offsets", p.num_groups);
  if (workspace > 0 && (!a.workspace || a.workspace_bytes < workspace))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "workspace of %lld bytes needed, %lld given", (long long)workspace,
                     (long long)(a.workspace ? a.workspace_bytes : 0));
  return MOEGG_OK;
}

// Forward; `saved`: which of the tensors are in 8 bits, or null.
moegg_status run_linear(const moegg_linear_problem* problem, const moegg_linear_args* args, const moegg_linear_saved* saved,
                        void* stream) {
  moegg_status st = check_linear(problem);
  if (st != MOEGG_OK) return st;
  if (saved && (st = check_saved(*problem, *saved)) != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_linear_problem& p = *problem;
  const moegg::LinearArgs a = linear_args(p, args, saved);
  const bool any = p.m > 0;
  if (any && (!a.x || !a.w || !a.y)) return set_error(MOEGG_ERROR_INVALID_VALUE, "x, w and y are required");
  if (a.dy || a.dx || a.dw || a.db)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dy, dx, dw and db are for moegg_linear_backward");
  if (a.x8.kind != moegg::ROW_BF16) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "x_dtype: the forward reads a BF16 x");
  if (any && a.c_kind != moegg::ROW_BF16 && (!a.c || !a.c_sf))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "c and c_sf are required with c_dtype");
  const moegg::LinearPlan plan = moegg::plan_linear(a);
  const int64_t workspace = plan.workspace;
  st = check_linear_pointers(p, *args, saved, workspace);
  if (st != MOEGG_OK) return st;
  const int64_t n_out = p.act == MOEGG_ACT_SWIGLU ? p.n / 2 : p.n;
  const int64_t y_bytes = p.m * n_out * (a.out_f32 ? 4 : 2);
  const int64_t c_bytes = kept_bytes(a.c_kind, p.m * p.n), sf_bytes = p.m * (p.n / 32);
  const Span in[] = {{"x", a.x, p.m * p.k * 2}, {"w", a.w, w_bytes(p)}, {"bias", a.bias, int64_t{p.num_groups} * p.n * 4},
                     {"offsets", a.offsets, int64_t{p.num_groups} * 4}};
  const Span out[] = {{"y", a.y, y_bytes}, {"c", a.c, c_bytes}, {"c_sf", a.c_sf, sf_bytes},
                      {"workspace", a.workspace, workspace}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (overlap(a.residual, p.m * n_out * 2, a.c, c_bytes) || overlap(a.residual, p.m * n_out * 2, a.c_sf, sf_bytes) ||
      overlap(a.residual, p.m * n_out * 2, a.workspace, workspace))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and c, c_sf or the workspace overlap");
  if (overlap(a.residual, p.m * n_out * 2, a.y, y_bytes) && (a.out_f32 || static_cast<const void*>(a.residual) != a.y))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and y overlap without being the same BF16 tensor");
  if (!any) return launched(hipSuccess, "linear");
  return launched(moegg::launch_linear(a, plan, static_cast<hipStream_t>(stream)), "linear kernel");
}

moegg_status run_linear_backward(const moegg_linear_problem* problem, const moegg_linear_args* args,
                                 const moegg_linear_saved* saved, void* stream) {
  moegg_status st = check_linear(problem);
  if (st != MOEGG_OK) return st;
  if (saved && (st = check_saved(*problem, *saved)) != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_linear_problem& p = *problem;
  const moegg::LinearArgs a = linear_args(p, args, saved);
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
  if (any && a.c && a.c_kind != moegg::ROW_BF16 && !a.c_sf) return set_error(MOEGG_ERROR_INVALID_VALUE, "c in 8 bits needs c_sf");
  if (any && a.dw && a.x8.kind != moegg::ROW_BF16 && !a.x8.scales)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "x in 8 bits needs x_sf");
  const moegg::LinearPlan plan = moegg::plan_linear_backward(a, a.dx, a.dw, a.db);
  const int64_t workspace = plan.workspace;
  st = check_linear_pointers(p, *args, saved, workspace);
  if (st != MOEGG_OK) return st;
  const int64_t n_out = p.act == MOEGG_ACT_SWIGLU ? p.n / 2 : p.n;
  const Span in[] = {{"x", args->x, kept_bytes(a.x8.kind, p.m * p.k)}, {"w", a.w, w_bytes(p)}, {"dy", a.dy, p.m * n_out * 2},
                     {"c", a.c, kept_bytes(a.c_kind, p.m * p.n)}, {"offsets", a.offsets, int64_t{p.num_groups} * 4},
                     {"x_sf", a.x8.scales, p.m * (p.k / 32)}, {"c_sf", a.c_sf, p.m * (p.n / 32)}};
  const Span out[] = {{"dx", a.dx, p.m * p.k * 2}, {"dw", a.dw, w_bytes(p) * (a.out_f32 ? 2 : 1)},
                      {"db", a.db, int64_t{p.num_groups} * p.n * 4}, {"workspace", a.workspace, workspace}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (none) return launched(hipSuccess, "linear backward");
  return launched(moegg::launch_linear_backward(a, plan, static_cast<hipStream_t>(stream)), "linear backward kernel");
}

// ---- norm, rows kept in 8 bits -----------------------------------------------------

int norm_kind(const moegg_norm_problem& p) { return p.mx_dtype == MOEGG_DT_NONE ? moegg::ROW_BF16 : row_kind(p.mx_dtype); }

moegg_status check_norm(const moegg_norm_problem* pp, bool backward) {
  if (!pp) return set_error(MOEGG_ERROR_INVALID_VALUE, "problem must be non-NULL");
  const moegg_norm_problem& p = *pp;
  if (p.rows < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "rows=%lld negative", (long long)p.rows);
  if (p.rows > INT32_MAX) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "rows=%lld above 2^31-1", (long long)p.rows);
  if (p.stream_dtype != MOEGG_DT_BF16 && p.stream_dtype != MOEGG_DT_F32)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "stream_dtype=%d must be BF16 or F32", p.stream_dtype);
  if (!(p.eps > 0.0f) || !std::isfinite(p.eps)) return set_error(MOEGG_ERROR_INVALID_VALUE, "eps must be positive and finite");
  int step = 8;
  if (!backward) {
    if (p.x_dtype != MOEGG_DT_BF16 && p.x_dtype != MOEGG_DT_F32)
      return set_error(MOEGG_ERROR_INVALID_VALUE, "x_dtype=%d must be BF16 or F32", p.x_dtype);
    if (p.x_dtype == MOEGG_DT_F32 && p.stream_dtype != MOEGG_DT_F32)
      return set_error(MOEGG_ERROR_NOT_SUPPORTED, "an F32 x goes with an F32 stream");
    if (p.mx_dtype != MOEGG_DT_NONE && (row_kind(p.mx_dtype) < 0 || p.mx_dtype == MOEGG_DT_BF16))
      return set_error(MOEGG_ERROR_INVALID_VALUE, "mx_dtype=%d must be NONE, E4M3, E5M2 or E2M1X2", p.mx_dtype);
    if (p.sf_layout != MOEGG_SF_ROW_MAJOR && p.sf_layout != MOEGG_SF_KPLANES)
      return set_error(MOEGG_ERROR_INVALID_VALUE, "sf_layout=%d must be ROW_MAJOR or KPLANES", p.sf_layout);
    step = p.mx_dtype == MOEGG_DT_NONE ? 8 : p.mx_dtype == MOEGG_DT_E2M1X2 ? 256 : 128;
  }
  if (p.width < 1 || p.width % step != 0)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d: a positive multiple of %d needed", p.width, step);
  if (p.width > moegg::kMaxNormWidth)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d above %d", p.width, moegg::kMaxNormWidth);
  // (the backward's grid is bounded)
  if (!backward && moegg::rms_norm_threads(p.rows, p.width, p.stream_dtype == MOEGG_DT_F32, norm_kind(p)) > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "rows=%lld width=%d: more threads than a launch holds", (long long)p.rows, p.width);
  return MOEGG_OK;
}

moegg::NormArgs norm_args(const moegg_norm_problem& p, const moegg_norm_args& q, bool backward) {
  moegg::NormArgs a{};
  a.weight = q.weight;
  if (backward) {
    a.dy = static_cast<const uint16_t*>(q.dy);
    a.stored = q.h;
    a.dh = q.dh;
    a.dx = q.dx;
    a.dw = q.dweight;
    a.partial = q.dweight ? static_cast<float*>(q.workspace) : nullptr;
  } else {
    a.x = q.x;
    a.residual = q.residual;
    a.h = q.h;
    a.y = static_cast<uint16_t*>(q.y);
    a.codes = q.codes;
    a.scales = q.sf;
    a.kind = norm_kind(p);
    a.x_f32 = p.x_dtype == MOEGG_DT_F32;
    a.kplanes = p.sf_layout == MOEGG_SF_KPLANES;
  }
  a.rows = p.rows;
  a.width = p.width;
  a.stream_f32 = p.stream_dtype == MOEGG_DT_F32;
  a.eps = p.eps;
  a.inverse_width = 1.0 / p.width;
  return a;
}

// Sizes and types of rows and their 8 bits.
moegg_status check_kept_rows(int32_t x_dtype, int64_t rows, int32_t width, int32_t dtype, int32_t sf_layout) {
  if (x_dtype != MOEGG_DT_BF16 && x_dtype != MOEGG_DT_F32)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "x_dtype=%d must be BF16 or F32", x_dtype);
  if (dtype != MOEGG_DT_E4M3 && dtype != MOEGG_DT_E5M2)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dtype=%d must be E4M3 or E5M2", dtype);
  if (sf_layout != MOEGG_SF_ROW_MAJOR && sf_layout != MOEGG_SF_KPLANES)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "sf_layout=%d must be ROW_MAJOR or KPLANES", sf_layout);
  if (rows < 0) return set_error(MOEGG_ERROR_INVALID_VALUE, "rows=%lld negative", (long long)rows);
  if (rows > INT32_MAX) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "rows=%lld above 2^31-1", (long long)rows);
  const int step = sf_layout == MOEGG_SF_KPLANES ? 128 : 32;
  if (width < 1 || width % step != 0)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d: a positive multiple of %d needed", width, step);
  if (width > (1 << 20)) return set_error(MOEGG_ERROR_NOT_SUPPORTED, "width=%d above 2^20", width);
  if ((rows * width + 4095) / 4096 * 256 > moegg::kLaunchThreads)
    return set_error(MOEGG_ERROR_NOT_SUPPORTED, "rows=%lld width=%d: more threads than a launch holds", (long long)rows, width);
  return MOEGG_OK;
}

}  // namespace

extern "C" {

moegg_status moegg_route(const moegg_route_problem* problem, const void* logits, const float* bias, int32_t* ids,
                         float* weights, void* stream) {
  return run_route(problem, nullptr, false, logits, bias, ids, weights, stream);
}

moegg_status moegg_route_grouped(const moegg_route_problem* problem, const moegg_route_groups* groups, const void* logits,
                                 const float* bias, int32_t* ids, float* weights, void* stream) {
  return run_route(problem, groups, true, logits, bias, ids, weights, stream);
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
  return moegg::plan_linear(linear_args(*problem, nullptr)).workspace;
}

int64_t moegg_linear_backward_workspace(const moegg_linear_problem* problem, int32_t want) {
  if (check_linear(problem) != MOEGG_OK) return -1;
  return moegg::plan_linear_backward(linear_args(*problem, nullptr), want & 1, want & 2, want & 4).workspace;
}

int64_t moegg_linear_saving_workspace(const moegg_linear_problem* problem, const moegg_linear_saved* saved) {
  if (check_linear(problem) != MOEGG_OK || (saved && check_saved(*problem, *saved) != MOEGG_OK)) return -1;
  return moegg::plan_linear(linear_args(*problem, nullptr, saved)).workspace;
}

int64_t moegg_linear_saved_backward_workspace(const moegg_linear_problem* problem, const moegg_linear_saved* saved,
                                              int32_t want) {
  if (check_linear(problem) != MOEGG_OK || (saved && check_saved(*problem, *saved) != MOEGG_OK)) return -1;
  return moegg::plan_linear_backward(linear_args(*problem, nullptr, saved), want & 1, want & 2, want & 4).workspace;
}

moegg_status moegg_linear(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream) {
  return run_linear(problem, args, nullptr, stream);
}

moegg_status moegg_linear_backward(const moegg_linear_problem* problem, const moegg_linear_args* args, void* stream) {
  return run_linear_backward(problem, args, nullptr, stream);
}

moegg_status moegg_linear_saving(const moegg_linear_problem* problem, const moegg_linear_args* args,
                                 const moegg_linear_saved* saved, void* stream) {
  return run_linear(problem, args, saved, stream);
}

moegg_status moegg_linear_saved_backward(const moegg_linear_problem* problem, const moegg_linear_args* args,
                                         const moegg_linear_saved* saved, void* stream) {
  return run_linear_backward(problem, args, saved, stream);
}

moegg_status moegg_quantise(const void* x, int32_t x_dtype, int64_t rows, int32_t width, int32_t dtype, int32_t sf_layout,
                            uint8_t* codes, uint8_t* sf, void* stream) {
  moegg_status st = check_kept_rows(x_dtype, rows, width, dtype, sf_layout);
  if (st != MOEGG_OK) return st;
  const bool any = rows > 0;
  const Pointer ps[] = {{"x", x, 16, any}, {"codes", codes, 16, any}, {"sf", sf, 16, any}};
  if ((st = check_pointers(ps)) != MOEGG_OK) return st;
  const Span in[] = {{"x", x, rows * width * (x_dtype == MOEGG_DT_F32 ? 4 : 2)}};
  const Span out[] = {{"codes", codes, rows * width}, {"sf", sf, rows * (width / 32)}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "quantise");
  return launched(moegg::launch_quantise(x, x_dtype == MOEGG_DT_F32, codes, sf, row_kind(dtype), sf_layout == MOEGG_SF_KPLANES,
                                         rows, width, static_cast<hipStream_t>(stream)),
                  "quantise kernel");
}

moegg_status moegg_dequantise(const uint8_t* codes, const uint8_t* sf, int64_t rows, int32_t width, int32_t dtype,
                              int32_t sf_layout, void* x, int32_t x_dtype, void* stream) {
  moegg_status st = check_kept_rows(x_dtype, rows, width, dtype, sf_layout);
  if (st != MOEGG_OK) return st;
  const bool any = rows > 0;
  const Pointer ps[] = {{"x", x, 16, any}, {"codes", codes, 16, any}, {"sf", sf, 16, any}};
  if ((st = check_pointers(ps)) != MOEGG_OK) return st;
  const Span in[] = {{"codes", codes, rows * width}, {"sf", sf, rows * (width / 32)}};
  const Span out[] = {{"x", x, rows * width * (x_dtype == MOEGG_DT_F32 ? 4 : 2)}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  if (!any) return launched(hipSuccess, "dequantise");
  const moegg::SavedRows q{codes, sf, row_kind(dtype), sf_layout == MOEGG_SF_KPLANES};
  return launched(moegg::launch_dequantise(q, x, x_dtype == MOEGG_DT_F32, rows, width, static_cast<hipStream_t>(stream)),
                  "dequantise kernel");
}

moegg_status moegg_rms_norm(const moegg_norm_problem* problem, const moegg_norm_args* args, void* stream) {
  moegg_status st = check_norm(problem, false);
  if (st != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_norm_problem& p = *problem;
  const moegg_norm_args& q = *args;
  const bool any = p.rows > 0, mx = p.mx_dtype != MOEGG_DT_NONE;
  const Pointer ps[] = {{"x", q.x, 16, any}, {"weight", q.weight, 4, any}, {"residual", q.residual, 16, false},
                        {"h", q.h, 16, any && q.residual}, {"y", q.y, 16, any && !mx}, {"codes", q.codes, 16, any && mx},
                        {"sf", q.sf, 16, any && mx}};
  if ((st = check_pointers(ps)) != MOEGG_OK) return st;
  if (q.dy || q.dh || q.dx || q.dweight)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "dy, dh, dx and dweight are for moegg_rms_norm_backward");
  if (any && !q.residual && q.h) return set_error(MOEGG_ERROR_INVALID_VALUE, "h without a residual is x");
  if (any && !q.residual && p.x_dtype != p.stream_dtype)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "without a residual x has the stream's type");
  if (!mx && (q.codes || q.sf)) return set_error(MOEGG_ERROR_INVALID_VALUE, "codes and sf need mx_dtype");
  const int64_t n = p.rows * p.width, stream_bytes = n * (p.stream_dtype == MOEGG_DT_F32 ? 4 : 2);
  const Span in[] = {{"x", q.x, n * (p.x_dtype == MOEGG_DT_F32 ? 4 : 2)}, {"weight", q.weight, int64_t{p.width} * 4}};
  const Span out[] = {{"h", q.h, stream_bytes}, {"y", q.y, n * 2}, {"codes", q.codes, p.mx_dtype == MOEGG_DT_E2M1X2 ? n / 2 : n},
                      {"sf", q.sf, p.rows * (p.width / 32)}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  for (const Span& o : out)
    if (overlap(q.residual, stream_bytes, o.p, o.bytes) && (o.p != q.h || q.residual != q.h))
      return set_error(MOEGG_ERROR_INVALID_VALUE, "residual and %s overlap", o.name);
  if (!any) return launched(hipSuccess, "rms_norm");
  return launched(moegg::launch_rms_norm(norm_args(p, q, false), static_cast<hipStream_t>(stream)), "rms_norm kernel");
}

int64_t moegg_rms_norm_backward_workspace(const moegg_norm_problem* problem) {
  if (check_norm(problem, true) != MOEGG_OK) return -1;
  return moegg::rms_norm_backward_workspace(problem->rows, problem->width);
}

moegg_status moegg_rms_norm_backward(const moegg_norm_problem* problem, const moegg_norm_args* args, void* stream) {
  moegg_status st = check_norm(problem, true);
  if (st != MOEGG_OK) return st;
  if (!args) return set_error(MOEGG_ERROR_INVALID_VALUE, "args must be non-NULL");
  const moegg_norm_problem& p = *problem;
  const moegg_norm_args& q = *args;
  const bool any = p.rows > 0, none = !q.dx && !q.dweight;
  if (any && none) return set_error(MOEGG_ERROR_INVALID_VALUE, "one of dx and dweight is required");
  const Pointer ps[] = {{"dy", q.dy, 16, any}, {"h", q.h, 16, any}, {"weight", q.weight, 4, any}, {"dh", q.dh, 16, false},
                        {"dx", q.dx, 16, false}, {"dweight", q.dweight, 4, false}, {"workspace", q.workspace, 16, false}};
  if ((st = check_pointers(ps)) != MOEGG_OK) return st;
  if (q.x || q.residual || q.y || q.codes || q.sf)
    return set_error(MOEGG_ERROR_INVALID_VALUE, "x, residual, y, codes and sf are for moegg_rms_norm");
  const int64_t need = q.dweight ? moegg::rms_norm_backward_workspace(p.rows, p.width) : 0;
  if (need > 0 && (!q.workspace || q.workspace_bytes < need))
    return set_error(MOEGG_ERROR_INVALID_VALUE, "workspace of %lld bytes needed, %lld given", (long long)need,
                     (long long)(q.workspace ? q.workspace_bytes : 0));
  const int64_t n = p.rows * p.width, stream_bytes = n * (p.stream_dtype == MOEGG_DT_F32 ? 4 : 2);
  const Span in[] = {{"dy", q.dy, n * 2}, {"h", q.h, stream_bytes}, {"weight", q.weight, int64_t{p.width} * 4}};
  const Span out[] = {{"dx", q.dx, stream_bytes}, {"dweight", q.dweight, int64_t{p.width} * 4}, {"workspace", q.workspace, need}};
  if ((st = check_apart(in, out)) != MOEGG_OK) return st;
  for (const Span& o : out)
    if (overlap(q.dh, stream_bytes, o.p, o.bytes) && (o.p != q.dx || q.dh != q.dx))
      return set_error(MOEGG_ERROR_INVALID_VALUE, "dh and %s overlap", o.name);
  if (none) return launched(hipSuccess, "rms_norm backward");
  return launched(moegg::launch_rms_norm_backward(norm_args(p, q, true), static_cast<hipStream_t>(stream)),
                  "rms_norm backward kernel");
}

}  // extern "C"
