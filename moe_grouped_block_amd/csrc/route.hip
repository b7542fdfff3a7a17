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

// Lane l of the token's LPT lanes holds experts l EPL + [0, EPL), so that the
// lowest of several experts sits in the lowest lane; V is the width of its
// accesses (16 bytes where EPL and the expert count allow).
template <bool BF16, int LPT, int EPL, int V>
struct Row {
  static constexpr int NI = EPL / V;
  __device__ static __forceinline__ int expert(int lane, int i, int v) { return lane * EPL + i * V + v; }
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
  // one of them, of expert e
  __device__ static __forceinline__ float one(const void* base, int64_t row, int experts, int e) {
    const int64_t i = row * experts + e;
    const float x = BF16 ? from_bf16(static_cast<const uint16_t*>(base)[i]) : static_cast<const float*>(base)[i];
    return x > kMaxF ? kMaxF : x;
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

// A token's lanes all belong to one wave: what one of them put into LDS is
// there for the others once the compiler keeps the order (the LDS runs a
// wave's accesses in order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Choices j = lane, lane + LPT, ... are a lane's own: at most JPL of them.
template <int LPT>
constexpr int kJpl = (kMaxTopK + LPT - 1) / LPT;

// The weights of the chosen logits (l[i]: choice lane + i LPT, -inf where
// there is none).  `top` and `total`: the softmax's maximum and sum over all
// experts (not renormalised).
// Renormalised, the softmax is one over the chosen experts alone, and the
// sigmoid's ratio is formed from u_j = p_j exp(-m'), m' = min(0, max l):
// u_j = 1 / (exp(m') + exp(m' - l_j)), which does not underflow when every
// chosen score does.
template <int LPT>
__device__ __forceinline__ void chosen_weights(const RouteArgs& a, float top, float total, const float* l, float* w) {
  constexpr int JPL = kJpl<LPT>;
  if (a.renormalise) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < JPL; ++i) m = fmaxf(m, l[i]);
    m = lanes_max<LPT>(m);
    const float mm = a.softmax ? m : fminf(m, 0.0f);
    const float em = a.softmax ? 0.0f : expf(mm);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < JPL; ++i) {
      const float e = a.softmax ? expf(l[i] - mm) : 1.0f / (em + expf(mm - l[i]));
      w[i] = l[i] == kNegInf ? 0.0f : e;
      sum += w[i];
    }
    sum = lanes_sum<LPT>(sum);
    const float r = sum > 0.0f ? a.scale / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < JPL; ++i) w[i] *= r;
  } else {
#pragma unroll
    for (int i = 0; i < JPL; ++i) {
      const float p = a.softmax ? expf(l[i] - top) / total : sigmoid(l[i]);
      w[i] = l[i] == kNegInf ? 0.0f : a.scale * p;
    }
  }
}

// ---- forward ---------------------------------------------------------------

// The `rounds` largest keys of a token (-inf: cannot be chosen), largest
// first, ties to the lowest expert: its ids[] and, where wanted, keys[].  A
// round: the largest key of the token's lanes, the first expert that has it,
// which is taken out.  (The first of a lane's equal keys is singled out in the
// masks of the comparisons, by scalar instructions: three vector instructions
// a key.  With the logit carried along and the position compared again it was
// six, and 16381 tokens of 256 experts took 17.6 us instead of 16.8.)
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
template <int LPT, int EPL, typename Key>
__device__ __forceinline__ void choose(Key* key, int rounds, int lane, int* ids, Key* keys) {
  constexpr Key none = -static_cast<Key>(__builtin_inff());
  for (int j = 0; j < rounds; ++j) {
    Key mine = key[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q) mine = larger(mine, key[q]);
    Key best = mine;
    steps<LPT>([&](auto c) { best = larger(best, partner<decltype(c)::value>(best)); });
    // the first of the token's lanes that has it
    const uint64_t have = __ballot(mine == best) >> (threadIdx.x & 63 & ~(LPT - 1));
    if (lane == __builtin_ctzll(have)) {
      int at = 0;
      bool found = false;
#pragma unroll
      for (int q = 0; q < EPL; ++q) {
        const bool hit = key[q] == best && !found;
        found |= hit;
        key[q] = hit ? none : key[q];
        at = hit ? q : at;
      }
      ids[j] = best > none ? lane * EPL + at : -1;
      if (keys) keys[j] = best;
    }
  }
}

// e^x by the exponential unit, for sums and keys with bounds of their own.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// With a bias the keys are sums of two numbers of different size, whose
// order can hang on bits that fp32 does not have.  They are formed in fp32
// first, with kSpare choices more than asked for.  Where two neighbours in
// that order are nearer than the error of both, and not made of the same
// numbers (whose sums are equal in any precision), the choices up to the next
// clear gap are put into the order of their keys in 64 bits, one key a lane;
// where no gap follows, the wave's tokens are chosen again with all keys in 64
// bits.  Measured, 16381 tokens, 256 experts, sigmoid: 64 bits for every token
// 30 us, this form 17 us.
constexpr int kSpare = 2;
constexpr int kSlots = kMaxTopK + kSpare;

template <bool BF16, int LPT, int EPL, int V, bool BIAS>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  using R = Row<BF16, LPT, EPL, V>;
  constexpr int TPB = 256 / LPT, JPL = kJpl<LPT>;
  __shared__ float s_logit[TPB][kSlots];
  __shared__ int s_id[TPB][kSlots];
  __shared__ float s_key[BIAS ? TPB : 1][kSlots];
  __shared__ int s_flag[BIAS ? TPB : 1][kSlots];
  __shared__ double s_exact[BIAS ? TPB : 1][kSlots];
  const int lane = threadIdx.x % LPT, slot = threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool live = t < a.tokens;               // idle lanes repeat the last token and store nothing
  const int64_t row = live ? t : a.tokens - 1;
  const int k = a.top_k;
  float x[EPL];
  R::load(a.logits, row, a.experts, lane, x);

  float top = 0.0f, total = 1.0f;
  if (a.softmax) {
    top = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, x[j]);
    top = lanes_max<LPT>(fmaxf(top, kNegInf));   // (a token of NaN: -inf)
    if (top == kNegInf) top = 0.0f;
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) total += fast_exp(x[j] - top);
    total = lanes_sum<LPT>(total);
  }

  float key[EPL];
  if constexpr (!BIAS) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = x[j] > kNegInf ? x[j] : kNegInf;
    choose<LPT, EPL, float>(key, k, lane, s_id[slot], s_logit[slot]);   // (the keys are the logits)
    wave_sync();
  } else {
    // a NaN in the softmax's sum leaves the choice among the others
    float valid = total;
    if (a.softmax && __any(!(total == total))) {
      valid = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) valid += x[j] == x[j] ? fast_exp(x[j] - top) : 0.0f;
      valid = lanes_sum<LPT>(valid);
    }
    const float rt = 1.0f / valid;
#pragma unroll
    for (int i = 0; i < R::NI; ++i) {
      typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
      const int e = R::expert(lane, i, 0);
      const vec bv = *reinterpret_cast<const vec*>(a.bias + (e < a.experts ? e : 0));   // (whole groups of V exist)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int j = i * V + v;
        const float b = bv[v];
        const float p = a.softmax ? fast_exp(x[j] - top) * rt : __builtin_amdgcn_rcpf(1.0f + fast_exp(-x[j]));
        const float q = p + b;
        key[j] = x[j] > kNegInf && q > kNegInf ? q : kNegInf;    // NaN: false
      }
    }
    const int cand = min(k + kSpare, a.experts);
    choose<LPT, EPL, float>(key, cand, lane, s_id[slot], s_key[slot]);
    float rest = key[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q) rest = fmaxf(rest, key[q]);
    rest = lanes_max<LPT>(rest);                   // the best that is left
    wave_sync();
    auto fetch_logits = [&](int n) __attribute__((always_inline)) {
      for (int j = lane; j < n; j += LPT) {
        const int e = s_id[slot][j];
        s_logit[slot][j] = e >= 0 ? R::one(a.logits, row, a.experts, e) : kNegInf;
      }
      wave_sync();
    };
    fetch_logits(cand);
    // Choice j against the next: 0 clear, 1 the same numbers, 2 in doubt.  A key
    // is off by a rounding of its sum and by p's error: p <= 1, its exponential's
    // argument (p |x| < 0.4), the unit's last places and a sum of up to 16 + 6
    // terms, below 50 2^-24.
    constexpr float kP = 2.0f * 50.0f * 5.9604645e-8f, kSum = 2.4e-7f;
    bool maybe = false;
    for (int j = lane; j < cand; j += LPT) {
      const float k0 = s_key[slot][j], k1 = j + 1 < cand ? s_key[slot][j + 1] : rest;
      int f = 0;
      if (k1 > kNegInf && !(k0 - k1 > kP + kSum * (fabsf(k0) + fabsf(k1)))) {
        f = 2;
        if (j + 1 < cand && s_logit[slot][j] == s_logit[slot][j + 1] &&
            a.bias[s_id[slot][j]] == a.bias[s_id[slot][j + 1]])
          f = 1;
      }
      s_flag[slot][j] = f;
      maybe |= f && j < k;
    }
    wave_sync();
    if (__any(maybe)) {
      int m = k;                                   // choices up to the next clear gap
      while (m < cand && s_flag[slot][m - 1]) ++m;
      const bool open = s_flag[slot][m - 1] != 0;
      bool doubt = false;
      for (int j = 0; j < m; ++j) doubt |= s_flag[slot][j] == 2;
      if (__any(doubt)) {
        const bool all = __any(doubt && open);
        double exact[EPL];
        double dt = 1.0;
        if (a.softmax || all) {
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            exact[j] = a.softmax ? exp(static_cast<double>(x[j]) - top) : 1.0 / (1.0 + exp(-static_cast<double>(x[j])));
            sum += x[j] == x[j] ? exact[j] : 0.0;
          }
          if (a.softmax) dt = 1.0 / lanes_sum<LPT>(sum);
        }
        if (all) {
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            const int e = R::expert(lane, j / V, j % V);
            const double q = exact[j] * dt + a.bias[e < a.experts ? e : 0];
            exact[j] = x[j] > kNegInf && q > -__builtin_inf() ? q : -__builtin_inf();
          }
          choose<LPT, EPL, double>(exact, k, lane, s_id[slot], nullptr);
          wave_sync();
          fetch_logits(k);
        } else {
          constexpr int N = (kSlots + LPT - 1) / LPT;
          double mine[N];
          int id[N], rank[N];
          float lg[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int j = lane + i * LPT;
            id[i] = j < m ? s_id[slot][j] : -1;
            lg[i] = j < m ? s_logit[slot][j] : kNegInf;
            mine[i] = 0.0;
            if (id[i] >= 0) {
              const double l = lg[i];
              mine[i] = (a.softmax ? exp(l - top) * dt : 1.0 / (1.0 + exp(-l))) + a.bias[id[i]];
              s_exact[slot][j] = mine[i];
            }
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < N; ++i) {
            rank[i] = 0;
            for (int j = 0; j < m; ++j) {
              const double o = s_exact[slot][j];
              const int oid = s_id[slot][j];
              if (oid >= 0 && (o > mine[i] || (o == mine[i] && oid < id[i]))) ++rank[i];
            }
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (id[i] >= 0) {
              s_id[slot][rank[i]] = id[i];
              s_logit[slot][rank[i]] = lg[i];
            }
        }
        wave_sync();
      }
    }
  }

  float l[JPL], w[JPL];
#pragma unroll
  for (int i = 0; i < JPL; ++i) {
    const int j = lane + i * LPT;
    l[i] = j < k ? s_logit[slot][j] : kNegInf;
  }
  chosen_weights<LPT>(a, top, total, l, w);
#pragma unroll
  for (int i = 0; i < JPL; ++i) {
    const int j = lane + i * LPT;
    if (live && j < k) {
      a.ids[t * k + j] = s_id[slot][j];
      a.weights[t * k + j] = w[i];
    }
  }
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
  constexpr int TPB = 256 / LPT, JPL = kJpl<LPT>;
  __shared__ float s_d[TPB][kMaxTopK];
  __shared__ int s_id[TPB][kMaxTopK];
  const int lane = threadIdx.x % LPT, slot = threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool live = t < a.tokens;
  const int64_t row = live ? t : a.tokens - 1;
  const int k = a.top_k;
  float l[JPL], g[JPL], w[JPL];
  int id[JPL];
#pragma unroll
  for (int i = 0; i < JPL; ++i) {
    const int j = lane + i * LPT;
    id[i] = j < k ? a.ids[row * k + j] : -1;
    if (id[i] < 0 || id[i] >= a.experts) id[i] = -1;
    l[i] = kNegInf;
    g[i] = 0.0f;
    if (id[i] >= 0) {
      l[i] = BF16 ? from_bf16(static_cast<const uint16_t*>(a.logits)[row * a.experts + id[i]])
                  : static_cast<const float*>(a.logits)[row * a.experts + id[i]];
      l[i] = l[i] > kMaxF ? kMaxF : l[i];
      g[i] = a.dweights[row * k + j];
    }
  }
  float x[EPL];
  float top = 0.0f, total = 1.0f;
  const bool full = a.softmax && !a.renormalise;      // every expert has a gradient
  if (full) {
    R::load(a.logits, row, a.experts, lane, x);
    top = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, x[j]);
    top = lanes_max<LPT>(fmaxf(top, kNegInf));
    if (top == kNegInf) top = 0.0f;
    total = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) total += fast_exp(x[j] - top);
    total = lanes_sum<LPT>(total);
  }
  chosen_weights<LPT>(a, top, total, l, w);
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < JPL; ++i) dot += g[i] * w[i];
  dot = lanes_sum<LPT>(dot);
  if (a.renormalise) dot = a.scale != 0.0f ? dot / a.scale : 0.0f;
#pragma unroll
  for (int i = 0; i < JPL; ++i) {
    const int j = lane + i * LPT;
    float d;
    if (a.renormalise) {
      d = w[i] * (g[i] - dot);
      if (!a.softmax) d *= sigmoid(-l[i]);
    } else {
      d = a.softmax ? g[i] * a.scale : g[i] * w[i] * sigmoid(-l[i]);
    }
    if (j < k) {
      s_id[slot][j] = id[i];
      s_d[slot][j] = id[i] >= 0 ? d : 0.0f;
    }
  }
  wave_sync();
  float out[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) out[q] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int e = s_id[slot][j];
    const float d = s_d[slot][j];
#pragma unroll
    for (int q = 0; q < EPL; ++q) out[q] += R::expert(lane, q / V, q % V) == e ? d : 0.0f;
  }
  if (full) {
    const float r = total > 0.0f ? 1.0f / total : (total == 0.0f ? 0.0f : total);   // NaN stays
#pragma unroll
    for (int q = 0; q < EPL; ++q) out[q] = fast_exp(x[q] - top) * r * (out[q] - dot);
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
