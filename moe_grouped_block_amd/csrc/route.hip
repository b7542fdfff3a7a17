// Router scores, the top-k choice and its gradient.
//
//   softmax   p_e = exp(l_e - max) / sum exp(l - max)
//   sigmoid   p_e = 1 / (1 + exp(-l_e))
//   key_e     l_e without a bias (both scores grow with the logit), p_e + bias_e with one
//   ids       the top_k experts of the largest keys, ties to the lowest index
//   weights   scale p_j, or scale p_j / (sum of the chosen p) with `renormalise`
//
// An expert with a logit of -inf or NaN is never chosen; a token with fewer
// than top_k experts to choose from ends in ids of -1 with weight 0.  +inf
// counts as the largest finite number.
//
// A token is held by LPT lanes (16 up to 256 experts, 64 above), EPL logits
// each, in registers: one pass over the logits.  Four tokens of 16 lanes
// share a wave, so the exchanges of one of the k rounds (best key over the
// token's lanes) are four DPP steps for four tokens.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "layer_internal.h"

namespace moegg {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kMaxF = 3.4028234663852886e38f;

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// ---- exchanges over a token's lanes: every lane ends with the result --------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xF, 0xF, false));
}

// STEP 0..3 pair lanes inside a 16-lane row (1, 2 apart, mirrored halves,
// mirrored row), 4 and 5 exchange rows and half waves.
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t x) {
  if constexpr (STEP == 0) return dpp_u<0xB1>(x);
  else if constexpr (STEP == 1) return dpp_u<0x4E>(x);
  else if constexpr (STEP == 2) return dpp_u<0x141>(x);
  else if constexpr (STEP == 3) return dpp_u<0x140>(x);
  else if constexpr (STEP == 4) {
    const v2u s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (threadIdx.x & 16) ? s.x : s.y;
  } else {
    const v2u s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return (threadIdx.x & 32) ? s.x : s.y;
  }
}
template <int STEP>
__device__ __forceinline__ float partner(float x) {
  return __uint_as_float(partner<STEP>(__float_as_uint(x)));
}
template <int STEP>
__device__ __forceinline__ double partner(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = partner<STEP>(static_cast<uint32_t>(u)), hi = partner<STEP>(static_cast<uint32_t>(u >> 32));
  return __builtin_bit_cast(double, lo | hi << 32);
}

template <int LPT, int STEP = 0, typename F>
__device__ __forceinline__ void steps(F&& f) {
  if constexpr ((1 << STEP) < LPT) {
    f(std::integral_constant<int, STEP>{});
    steps<LPT, STEP + 1>(f);
  }
}
template <int LPT, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
  steps<LPT>([&](auto c) { v += partner<decltype(c)::value>(v); });
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  steps<LPT>([&](auto c) { v = fmaxf(v, partner<decltype(c)::value>(v)); });
  return v;
}

// ---- a token's logits ------------------------------------------------------

__device__ __forceinline__ float from_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ uint32_t to_bf16(float f) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(f)));
}

// Lane l of the token's LPT lanes holds experts (i LPT + l) V + v; V is the
// width of its accesses (16 bytes where EPL and the expert count allow).
template <bool BF16, int LPT, int EPL, int V>
struct Row {
  static constexpr int NI = EPL / V;
  __device__ static __forceinline__ int expert(int lane, int i, int v) { return (i * LPT + lane) * V + v; }
  __device__ static __forceinline__ void load(const void* base, int64_t row, int experts, int lane, float* x) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = expert(lane, i, 0);
#pragma unroll
      for (int v = 0; v < V; ++v) x[i * V + v] = kNegInf;
      if (e >= experts) continue;
      if constexpr (BF16) {
        typedef uint16_t vec __attribute__((ext_vector_type(V)));
        const vec u = *reinterpret_cast<const vec*>(static_cast<const uint16_t*>(base) + row * experts + e);
#pragma unroll
        for (int v = 0; v < V; ++v) x[i * V + v] = from_bf16(u[v]);
      } else {
        typedef float vec __attribute__((ext_vector_type(V)));
        const vec u = *reinterpret_cast<const vec*>(static_cast<const float*>(base) + row * experts + e);
#pragma unroll
        for (int v = 0; v < V; ++v) x[i * V + v] = u[v];
      }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = x[j] > kMaxF ? kMaxF : x[j];   // NaN stays
  }
  __device__ static __forceinline__ void store(void* base, int64_t row, int experts, int lane, const float* x) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = expert(lane, i, 0);
      if (e >= experts) continue;
      if constexpr (BF16) {
        typedef uint16_t vec __attribute__((ext_vector_type(V)));
        vec u;
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = static_cast<uint16_t>(to_bf16(x[i * V + v]));
        *reinterpret_cast<vec*>(static_cast<uint16_t*>(base) + row * experts + e) = u;
      } else {
        typedef float vec __attribute__((ext_vector_type(V)));
        vec u;
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = x[i * V + v];
        *reinterpret_cast<vec*>(static_cast<float*>(base) + row * experts + e) = u;
      }
    }
  }
};

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The weights of the chosen logits l[0..k) (identical in all of a token's
// lanes, -inf where there is none).  `top` and `total`: the softmax's
// maximum and sum over all experts (not renormalised).
// Renormalised, the softmax is one over the chosen experts alone, and the
// sigmoid's ratio is formed from u_j = p_j exp(-m'), m' = min(0, max l):
// u_j = 1 / (exp(m') + exp(m' - l_j)), which does not underflow when every
// chosen score does.
template <typename Get, typename Put>
__device__ __forceinline__ void chosen_weights(const RouteArgs& a, float top, float total, Get&& logit, Put&& put) {
  const int k = a.top_k;
  float m = kNegInf;
  for (int j = 0; j < k; ++j) m = fmaxf(m, logit(j));
  if (a.renormalise) {
    const float mm = a.softmax ? m : fminf(m, 0.0f);
    auto u = [&](float l) {
      if (l == kNegInf) return 0.0f;
      return a.softmax ? expf(l - mm) : 1.0f / (expf(mm) + expf(mm - l));
    };
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) sum += u(logit(j));
    const float r = sum > 0.0f ? a.scale / sum : 0.0f;
    for (int j = 0; j < k; ++j) put(j, u(logit(j)) * r);
  } else {
    for (int j = 0; j < k; ++j) {
      const float l = logit(j);
      put(j, l == kNegInf ? 0.0f : a.scale * (a.softmax ? expf(l - top) / total : sigmoid(l)));
    }
  }
}

// ---- forward ---------------------------------------------------------------

template <bool BF16, int LPT, int EPL, int V, bool BIAS>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  using R = Row<BF16, LPT, EPL, V>;
  using Key = std::conditional_t<BIAS, double, float>;
  constexpr int TPB = 256 / LPT;
  __shared__ float chosen[TPB][kMaxTopK];
  const int lane = threadIdx.x % LPT, slot = threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool live = t < a.tokens;               // idle lanes repeat the last token and store nothing
  const int64_t row = live ? t : a.tokens - 1;
  float x[EPL];
  R::load(a.logits, row, a.experts, lane, x);

  float top = kNegInf, total = 1.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) top = fmaxf(top, x[j]);
  top = lanes_max<LPT>(top);
  const float shift = top == kNegInf ? 0.0f : top;
  if (a.softmax) {
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) total += expf(x[j] - shift);
    total = lanes_sum<LPT>(total);
  }

  // keys: the logit, or score + bias in 64 bits (the choice hangs on the
  // last bits of a sum of two numbers of different size)
  Key key[EPL];
  if constexpr (BIAS) {
    double dt = 0.0;
    if (a.softmax) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        key[j] = exp(static_cast<double>(x[j]) - shift);
        dt += x[j] == x[j] ? key[j] : 0.0;
      }
      dt = 1.0 / lanes_sum<LPT>(dt);
    }
#pragma unroll
    for (int i = 0; i < R::NI; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int j = i * V + v, e = R::expert(lane, i, v);
        const double p = a.softmax ? key[j] * dt : 1.0 / (1.0 + exp(-static_cast<double>(x[j])));
        const double b = e < a.experts ? static_cast<double>(a.bias[e]) : 0.0;
        const double q = p + b;
        key[j] = x[j] > kNegInf && q > -__builtin_inf() ? q : -__builtin_inf();   // NaN: false
      }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = x[j] > kNegInf ? x[j] : kNegInf;
  }

  for (int j = 0; j < a.top_k; ++j) {
    // best of this lane (the lowest expert first: ties keep it), then of the token's lanes
    Key best = key[0];
    int at = R::expert(lane, 0, 0);
    float logit = x[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q)
      if (key[q] > best) {
        best = key[q];
        at = R::expert(lane, q / V, q % V);
        logit = x[q];
      }
    steps<LPT>([&](auto c) {
      constexpr int S = decltype(c)::value;
      const Key ob = partner<S>(best);
      const int oa = static_cast<int>(partner<S>(static_cast<uint32_t>(at)));
      const float ol = partner<S>(logit);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        logit = ol;
      }
    });
    const bool there = best > -static_cast<Key>(__builtin_inf());
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (R::expert(lane, q / V, q % V) == at) key[q] = -static_cast<Key>(__builtin_inf());
    if (lane == 0) {
      if (live) a.ids[t * a.top_k + j] = there ? at : -1;
      chosen[slot][j] = there ? logit : kNegInf;
    }
  }
  __syncthreads();
  if (lane == 0 && live)
    chosen_weights(a, shift, total, [&](int j) { return chosen[slot][j]; },
                   [&](int j, float w) { a.weights[t * a.top_k + j] = w; });
}

// ---- backward --------------------------------------------------------------
//
// With g the gradient of the weights and w the weights themselves:
//   renormalised softmax   dl_j = w_j (g_j - sum g w / scale)           chosen experts only
//   renormalised sigmoid   the same times 1 - p_j
//   softmax                dl_e = p_e (G_e - sum_j G_j p_j), G = scale g at the chosen experts, 0 elsewhere
//   sigmoid                dl_j = scale g_j p_j (1 - p_j)
template <bool BF16, int LPT, int EPL, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteArgs a) {
  using R = Row<BF16, LPT, EPL, V>;
  constexpr int TPB = 256 / LPT;
  __shared__ float s_l[TPB][kMaxTopK], s_w[TPB][kMaxTopK];
  __shared__ float s_d[TPB][kMaxTopK];
  __shared__ int s_id[TPB][kMaxTopK];
  const int lane = threadIdx.x % LPT, slot = threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool live = t < a.tokens;
  const int64_t row = live ? t : a.tokens - 1;
  const int k = a.top_k;
  for (int j = lane; j < k; j += LPT) {
    int id = a.ids[row * k + j];
    if (id < 0 || id >= a.experts) id = -1;
    float l = kNegInf;
    if (id >= 0) {
      l = BF16 ? from_bf16(static_cast<const uint16_t*>(a.logits)[row * a.experts + id])
               : static_cast<const float*>(a.logits)[row * a.experts + id];
      l = l > kMaxF ? kMaxF : l;
    }
    s_id[slot][j] = id;
    s_l[slot][j] = l;
    s_d[slot][j] = id >= 0 ? a.dweights[row * k + j] : 0.0f;
  }
  float x[EPL];
  float top = 0.0f, total = 1.0f;
  const bool full = a.softmax && !a.renormalise;      // every expert has a gradient
  if (full) {
    R::load(a.logits, row, a.experts, lane, x);
    top = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) top = fmaxf(top, x[j]);
    top = lanes_max<LPT>(top);
    if (top == kNegInf) top = 0.0f;
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) total += expf(x[j] - top);
    total = lanes_sum<LPT>(total);
  }
  __syncthreads();
  // every lane forms the same k numbers; lane 0 keeps them
  float dot = 0.0f;
  chosen_weights(a, top, total, [&](int j) { return s_l[slot][j]; },
                 [&](int j, float w) {
                   dot += s_d[slot][j] * w;
                   if (lane == 0) s_w[slot][j] = w;
                 });
  __syncthreads();
  if (a.renormalise) dot = a.scale != 0.0f ? dot / a.scale : 0.0f;
  for (int j = lane; j < k; j += LPT) {
    const float g = s_d[slot][j], w = s_w[slot][j];
    float d;
    if (a.renormalise) {
      d = w * (g - dot);
      if (!a.softmax) d *= sigmoid(-s_l[slot][j]);
    } else {
      d = a.softmax ? g * a.scale : g * w * sigmoid(-s_l[slot][j]);
    }
    s_d[slot][j] = s_id[slot][j] >= 0 ? d : 0.0f;
  }
  __syncthreads();
  float out[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) out[q] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int id = s_id[slot][j];
    const float d = s_d[slot][j];
#pragma unroll
    for (int q = 0; q < EPL; ++q) out[q] += R::expert(lane, q / V, q % V) == id ? d : 0.0f;
  }
  if (full) {
    const float r = total > 0.0f ? 1.0f / total : (total == 0.0f ? 0.0f : total);   // NaN stays
#pragma unroll
    for (int q = 0; q < EPL; ++q) out[q] = expf(x[q] - top) * r * (out[q] - dot);
  }
  if (live) R::store(a.dlogits, t, a.experts, lane, out);
}

template <bool BF16, int LPT, int EPL, int V>
hipError_t launch_shape(const RouteArgs& a, bool backward, hipStream_t s) {
  constexpr int TPB = 256 / LPT;
  const int64_t blocks = (a.tokens + TPB - 1) / TPB;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(256);
  if (backward) hipLaunchKernelGGL((route_backward_kernel<BF16, LPT, EPL, V>), grid, block, 0, s, a);
  else if (a.bias) hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Accesses of up to 16 bytes where every token's logits start on such a
// boundary (the host checks that the tensors do), else one element each.
template <bool BF16, int LPT, int EPL>
hipError_t launch_width(const RouteArgs& a, bool backward, hipStream_t s) {
  constexpr int V = EPL < (BF16 ? 8 : 4) ? EPL : (BF16 ? 8 : 4);
  return a.experts % V == 0 ? launch_shape<BF16, LPT, EPL, V>(a, backward, s)
                            : launch_shape<BF16, LPT, EPL, 1>(a, backward, s);
}
template <bool BF16>
hipError_t launch_size(const RouteArgs& a, bool backward, hipStream_t s) {
  if (a.experts <= 64) return launch_width<BF16, 16, 4>(a, backward, s);
  if (a.experts <= 128) return launch_width<BF16, 16, 8>(a, backward, s);
  if (a.experts <= 256) return launch_width<BF16, 16, 16>(a, backward, s);
  return launch_width<BF16, 64, 16>(a, backward, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  return a.bf16 ? launch_size<true>(a, false, s) : launch_size<false>(a, false, s);
}
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s) {
  return a.bf16 ? launch_size<true>(a, true, s) : launch_size<false>(a, true, s);
}

}  // namespace moegg
