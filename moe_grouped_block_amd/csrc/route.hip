// Router scores, the top-k choice and its gradient.
//
//   softmax   p_e = exp(l_e - max) / sum exp(l - max)
//   sigmoid   p_e = 1 / (1 + exp(-l_e))
//   key_e     l_e without a bias (both scores grow with the logit), p_e + bias_e with one
//   ids       the top_k experts of the largest keys, ties to the lowest index
//   weights   scale p_j, or scale p_j / (sum of the chosen p) with `renormalise`
//   groups    (where asked for) only experts of the top_groups groups with the
//             largest scores can be chosen, ties to the lowest group; a group's
//             score is the largest key of its experts, or the sum of its two
//             largest p_e + bias_e
//
// An expert with a logit of -inf or NaN is never chosen; a token with fewer
// than top_k experts to choose from ends in ids of -1 with weight 0.  +inf
// counts as the largest finite number.
//
// A token is held by LPT lanes (16 up to 256 experts, 64 above and for few tokens), EPL logits
// each, in registers: one pass over the logits.  Four tokens of 16 lanes
// share a wave, so the exchanges of one of the k rounds (best key over the
// token's lanes) are four DPP steps for four tokens.
#include "lanes.h"
#include "layer_internal.h"

namespace moegg {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kMaxF = 3.4028234663852886e38f;

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

// The bits of a token's lanes.
template <int LPT>
__device__ __forceinline__ uint64_t token_ballot(bool b) {
  const uint64_t all = __ballot(b);
  return LPT == 64 ? all : (all >> (threadIdx.x & 63 & ~(LPT - 1))) & ((1ull << (LPT & 63)) - 1);
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
  const int k = a.top_k;
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
      w[i] = 0.0f;
      if (i * LPT >= k) continue;                // (the same for all)
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
      w[i] = 0.0f;
      if (i * LPT >= k) continue;
      const float p = a.softmax ? expf(l[i] - top) / total : sigmoid(l[i]);
      w[i] = l[i] == kNegInf ? 0.0f : a.scale * p;
    }
  }
}

// ---- forward ---------------------------------------------------------------

// The `rounds` largest keys of a token (-inf: cannot be chosen), largest
// first, ties to the lowest expert: its ids[] and, where wanted, keys[].  A
// round: the largest key of the token's lanes, the first expert that has it,
// which is taken out.  A lane keeps its keys in ordered pairs: a round looks at
// the larger ones, and where one is taken the smaller moves up.  (The first of a
// lane's equal keys is singled out in the masks of the comparisons, by scalar
// instructions.  16381 tokens of 256 experts: 8.2 us, without pairs 1.0 more; with a
// bias 10.9 and 1.5 more.)
__device__ __forceinline__ int32_t larger(int32_t a, int32_t b) { return max(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
// fp32 keys are compared as integers of the same order (-0 is 0): a step of a
// maximum is one instruction then, exchange included.
__device__ __forceinline__ int32_t ordered(float x) {
  const int32_t u = __float_as_int(x + 0.0f);
  return u ^ (u >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float number(int32_t u) { return __int_as_float(u ^ (u >> 31 & 0x7FFFFFFF)); }
__device__ __forceinline__ double ordered(double x) { return x; }
__device__ __forceinline__ double number(double x) { return x; }
template <int LPT, int EPL, typename Key>
__device__ __forceinline__ Key choose(const Key* key, int rounds, int lane, int first, int* ids, Key* keys) {
  using Rank = decltype(ordered(Key{}));
  const Rank none = ordered(-static_cast<Key>(__builtin_inff()));
  constexpr int P = EPL / 2;
  Rank hi[P], lo[P];
  uint32_t odd = 0;                              // pairs whose larger key is the second
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const Rank k0 = ordered(key[2 * q]), k1 = ordered(key[2 * q + 1]);
    hi[q] = k1 > k0 ? k1 : k0;
    lo[q] = k1 > k0 ? k0 : k1;
    odd |= k1 > k0 ? 1u << q : 0u;
  }
  auto most = [&]() __attribute__((always_inline)) {
    Rank m = hi[0];
#pragma unroll
    for (int q = 1; q < P; ++q) m = larger(m, hi[q]);
    return m;
  };
  for (int j = 0; j < rounds; ++j) {
    const Rank mine = most();
    Rank best = mine;
    steps<LPT>([&](auto c) { best = larger(best, partner<decltype(c)::value>(best)); });
    // the first of the token's lanes that has it
    const uint64_t have = __ballot(mine == best) >> (threadIdx.x & 63 & ~(LPT - 1));
    if (lane == (LPT < 64 ? __builtin_ctz(static_cast<uint32_t>(have)) : __builtin_ctzll(have))) {
      int at = 0;
      bool found = false;
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const bool hit = hi[q] == best && !found;
        found |= hit;
        hi[q] = hit ? lo[q] : hi[q];
        lo[q] = hit ? none : lo[q];
        at = hit ? q : at;
      }
      ids[j] = best > none ? first + 2 * at + static_cast<int>(odd >> at & 1) : -1;
      if (keys) keys[j] = number(best);
      odd ^= 1u << at;
    }
  }
  return number(most());
}

// e^x by the exponential unit, for sums and keys with bounds of their own.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-x)); }

// With a bias the keys are sums of two numbers of different size, whose
// order can hang on bits that fp32 does not have.  They are formed in fp32
// first, with kSpare choices more than asked for.  Where two neighbours in
// that order are nearer than the error of both, and not made of the same
// numbers (whose sums are equal in any precision), the choices up to the next
// clear gap are put into the order of their keys in 64 bits, one key a lane;
// where no gap follows, the wave's tokens are chosen again with all keys in 64
// bits.  Measured, 16381 tokens, 256 experts, sigmoid: 64 bits for every token
// 30 us, this form 10.9 us.
constexpr int kSpare = 2;
constexpr int kSlots = kMaxTopK + kSpare;

// What a key p + bias is off by, formed in fp32: a rounding of its sum (u = 2^-24
// of it, four are counted) and p's error.  e^x: 1.22 |x| u by its argument and 2 u by
// the unit.  Sigmoid: p (1 - p) of that (|x| p (1 - p) < 0.23), the sum's u and
// the reciprocal's 2 u, below 4 u; softmax: p |x| < 0.4, and a sum of up to 16 + 6
// terms with errors of their own, below 50 u.  The sigmoid's is taken twice: what
// counts is how few tokens are in doubt, whose waves end last (16381 x 256, 4 of 8
// groups with a bias, with 50 u for both 0.6 us more).
constexpr float kUnit = 5.9604645e-8f, kKeySum = 4.0f * kUnit;
__device__ __forceinline__ float key_p(const RouteArgs& a) { return (a.softmax ? 50.0f : 8.0f) * kUnit; }

// LDS of the choice of groups for a token (its lanes' own: nothing of it is
// another wave's): its scores, then in their place its groups' scores in 64
// bits; its groups' scores; the last group in and the first one out.  Four
// workgroups fit a compute unit.
template <int LPT, int EPL>
struct alignas(16) GroupScratch {
  union {
    float score[LPT * (EPL + 1)];
    double exact[kMaxGroups];
  };
  float group[kMaxGroups];
  float edge[4];
};

// The two largest of a set, one more value taken in.
__device__ __forceinline__ void take(float& b0, float& b1, float v) {
  b1 = __builtin_amdgcn_fmed3f(b0, b1, v);
  b0 = fmaxf(b0, v);
}

// Bits of the lane's EPL experts that are in no chosen group.  `score`: the
// experts' keys (-inf: not there), or with LOGITS their logits, which are exact
// and of whose largest p_of() makes a group's sum.  A group that is whole
// lanes, a power of two of them (256 experts in 8 groups: 2), is reduced in
// registers; of others lane g scans group g's experts through LDS (rows of a
// lane's EPL scores and a word more, so that neither side of the exchange meets
// a bank twice).  Then lane g counts the groups before its own.
// Scores are formed in fp32; where the last group in and the first one out are
// nearer than the error of both, the groups that may be on either side form
// theirs again in 64 bits.  (It is rare, but among 16381 tokens there always are
// such, and their waves are the last to end.)
// Measured, 16381 tokens, top 8 of 4 of 8 groups of 32 by their two best,
// sigmoid, without a bias (with one): 10.2 (11.3) us, where groups by their best
// logit take 8.2 and no groups 8.2 (10.9); 64 bits for all experts of a wave in
// doubt 6.6 (4 to 6) more.
template <typename R, bool LOGITS, int LPT, int EPL, typename P>
__device__ __forceinline__ uint32_t closed_groups(const RouteArgs& a, GroupScratch<LPT, EPL>& lds, const float* x, const float* score,
                                                  P&& p_of, float top, int64_t row, int lane) {
  constexpr int N = kMaxGroups / LPT;            // groups of a lane
  constexpr double kNone = -__builtin_inf();
  const int groups = a.groups, size = a.experts / groups;
  const bool sums = a.group_sums, sharp = LOGITS && !sums;
  const float kp = key_p(a);
  float mine[N], off[N];
  float low0[N], low1[N], g0 = kNegInf, g1 = kNegInf;     // the groups' two largest: of lane g's, of the lane's own
  auto set = [&](int i, float b0, float b1) __attribute__((always_inline)) {
    low0[i] = b0;
    low1[i] = b1;
    const bool two = sums && b1 > kNegInf;
    if (LOGITS && sums) {
      b0 = b0 > kNegInf ? p_of(b0) : kNegInf;
      b1 = p_of(b1);
    }
    mine[i] = two ? b0 + b1 : b0;
    off[i] = sharp || !(b0 > kNegInf) ? 0.0f : two ? 2.0f * kp + kKeySum * (fabsf(b0) + fabsf(b1)) : kp + kKeySum * fabsf(b0);
  };
  if (a.group_lanes) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) take(g0, g1, score[j]);
    steps<LPT>([&](auto c) {
      constexpr int S = decltype(c)::value;
      if ((1 << S) >= a.group_lanes) return;     // (the same for all lanes)
      const float o0 = partner<S>(g0), o1 = partner<S>(g1);
      g1 = fmaxf(fmaxf(g1, o1), fminf(g0, o0));
      g0 = fmaxf(g0, o0);
    });
    set(0, g0, g1);
    // by group, for lane g
    if (lane % a.group_lanes == 0) {
      lds.group[lane / a.group_lanes] = mine[0];
      lds.score[lane / a.group_lanes] = off[0];
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * LPT < groups) {
        mine[i] = lane + i * LPT < groups ? lds.group[lane + i * LPT] : kNegInf;
        off[i] = lane + i * LPT < groups ? lds.score[lane + i * LPT] : 0.0f;
      }
    wave_sync();
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) lds.score[lane * (EPL + 1) + j] = score[j];
    wave_sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i * LPT >= groups) break;
      const int g = lane + i * LPT;
      float b0 = kNegInf, b1 = kNegInf;
      if (g < groups) {
#pragma unroll 4
        for (int e = g * size; e < (g + 1) * size; ++e) take(b0, b1, lds.score[e + e / EPL]);
      }
      set(i, b0, b1);
    }
    wave_sync();
  }
  // (places behind the last group, up to a multiple of 4: -inf, never counted)
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * LPT < groups) lds.group[lane + i * LPT] = lane + i * LPT < groups ? mine[i] : kNegInf;
  wave_sync();
  auto rank_of = [&](float v, int g) __attribute__((always_inline)) {
    typedef float v4f __attribute__((ext_vector_type(4)));
    int rank = 0;
    for (int o = 0; o < groups; o += 4) {
      const v4f q = *reinterpret_cast<const v4f*>(&lds.group[o]);
#pragma unroll
      for (int e = 0; e < 4; ++e) rank += (q[e] > v) | ((q[e] == v) & (o + e < g));     // (no branches)
    }
    return rank;
  };
  uint64_t mask = 0;                             // the token's open groups
  auto add = [&](int i, bool open) __attribute__((always_inline)) { mask |= token_ballot<LPT>(open) << (i * LPT); };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * LPT >= groups) break;
    const int g = lane + i * LPT, rank = g < groups ? rank_of(mine[i], g) : kMaxGroups;
    add(i, rank < a.top_groups);
    if (rank == a.top_groups - 1 || rank == a.top_groups) lds.edge[rank == a.top_groups] = mine[i];
  }
  if (!sharp) {
    wave_sync();
    float most = 0.0f;                           // what any of the token's groups may be off by
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * LPT < groups) most = fmaxf(most, lane + i * LPT < groups ? off[i] : 0.0f);
    most = 2.0f * lanes_max<LPT>(most);
    const float in = lds.edge[0], out = lds.edge[1];
    const bool doubt = out > kNegInf && !(in - out > most);
    if (__any(doubt)) {
      double total = 1.0;
      if (a.softmax) {
        total = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) total += x[j] == x[j] ? exp(static_cast<double>(x[j]) - top) : 0.0;
        total = lanes_sum<LPT>(total);
      }
      auto exact = [&](double l, int e) __attribute__((always_inline)) {
        const double q = (a.softmax ? exp(l - top) / total : 1.0 / (1.0 + exp(-l))) + (a.bias ? a.bias[e] : 0.0f);
        return l > kNone && q > kNone ? q : kNone;                     // NaN: false
      };
      auto take2 = [](double& b0, double& b1, double v) __attribute__((always_inline)) {
        b1 = fmax(b1, fmin(b0, v));
        b0 = fmax(b0, v);
      };
      // Groups that are in or out whatever the errors are count as infinities;
      // of the others the experts that may be among the two largest are formed again.
      auto sure = [&](float v) __attribute__((always_inline)) {
        return v - out > most ? __builtin_inf() : in - v > most ? kNone : 0.0;
      };
      auto near = [&](float v, float b0, float b1) __attribute__((always_inline)) {
        const float least = sums && b1 > kNegInf ? b1 : b0;
        return v > kNegInf && !(least - v > (LOGITS ? 0.0f : 2.0f * (kp + kKeySum * fabsf(least))));
      };
      double again[N];
      if (a.group_lanes) {
        const float own = lds.group[lane / a.group_lanes & (kMaxGroups - 1)];
        const bool hot = doubt && lane / a.group_lanes < groups && sure(own) == 0.0;
        double b0 = kNone, b1 = kNone;
        uint32_t want = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) want |= hot && near(score[j], g0, g1) ? 1u << j : 0u;
        while (__any(want != 0)) {                // (the lanes' next experts together: the exponentials are what takes long)
          const int at = want ? __builtin_ctz(want) : 0;
          float l = x[0];
#pragma unroll
          for (int j = 1; j < EPL; ++j) {
            l = at == j ? x[j] : l;
            asm("" : "+v"(l));                    // (or the compiler makes it an access to memory)
          }
          const double v = exact(l, min(lane * EPL + at, a.experts - 1));
          if (want) take2(b0, b1, v);
          want &= want - 1;
        }
        steps<LPT>([&](auto c) {
          constexpr int S = decltype(c)::value;
          if ((1 << S) >= a.group_lanes) return;
          const double o0 = partner<S>(b0), o1 = partner<S>(b1);
          b1 = fmax(fmax(b1, o1), fmin(b0, o0));
          b0 = fmax(b0, o0);
        });
        if (lane % a.group_lanes == 0 && lane / a.group_lanes < groups)
          lds.exact[lane / a.group_lanes] = hot ? (sums && b1 > kNone ? b0 + b1 : b0) : sure(own);
        wave_sync();
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i * LPT < groups) again[i] = lane + i * LPT < groups ? lds.exact[lane + i * LPT] : kNone;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (i * LPT >= groups) break;
          const int g = lane + i * LPT;
          again[i] = g < groups ? sure(mine[i]) : kNone;
          const bool hot = doubt && again[i] == 0.0;
          double b0 = kNone, b1 = kNone;
          for (int e0 = 0; e0 < size; e0 += 32) {
            uint32_t want = 0;
#pragma unroll 4
            for (int e = e0; e < min(size, e0 + 32); ++e) {
              const int at = hot ? g * size + e : 0;
              want |= hot && near(lds.score[at + at / EPL], low0[i], low1[i]) ? 1u << (e - e0) : 0u;
            }
            while (__any(want != 0)) {
              const int e = want ? g * size + e0 + __builtin_ctz(want) : 0;
              const double v = exact(R::one(a.logits, row, a.experts, e), e);
              if (want) take2(b0, b1, v);
              want &= want - 1;
            }
          }
          if (again[i] == 0.0) again[i] = sums && b1 > kNone ? b0 + b1 : b0;
        }
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * LPT < groups && lane + i * LPT < groups) lds.exact[lane + i * LPT] = again[i];
      wave_sync();
      const uint64_t before = mask;
      mask = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (i * LPT >= groups) break;
        const int g = lane + i * LPT;
        int rank = kMaxGroups;
        if (g < groups) {
          rank = 0;
#pragma unroll 4
          for (int o = 0; o < groups; ++o) {
            const double v = lds.exact[o];
            rank += (v > again[i]) | ((v == again[i]) & (o < g));
          }
        }
        add(i, rank < a.top_groups);
      }
      if (!doubt) mask = before;
    }
  }
  if (a.group_lanes) return mask >> (lane / a.group_lanes & 63) & 1 ? 0u : ~0u;
  uint32_t closed = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const uint32_t g = (static_cast<uint32_t>(lane * EPL + j) * a.group_magic) >> 22;
    closed |= (g < kMaxGroups && (mask >> g & 1) ? 0u : 1u) << j;
  }
  return closed;
}

// The best keys of the token's experts as choose() has them, and the best that
// is left.  Where the open groups are whole lanes and at most half of them, the
// closed ones take half of their keys each: a round then looks at half as many
// (16381 tokens, 4 of 8 groups of 32, a bias: 1.9 us less; of 128 experts 0.8).
template <int LPT, int EPL>
__device__ __forceinline__ float choose_open(const RouteArgs& a, GroupScratch<LPT, EPL>& lds, float* key, bool open, int rounds,
                                             int lane, int* ids, float* keys) {
  constexpr int H = EPL / 2, ROW = EPL + 4;       // (a row's 16 bytes more: its lanes meet no bank twice)
  static_assert(LPT / 2 * ROW <= LPT * (EPL + 1) && LPT / 2 <= kMaxGroups, "rows of the open lanes");
  const int count = a.top_groups * a.group_lanes;
  const uint64_t all = token_ballot<LPT>(open);
  wave_sync();
  if (open) {
    const int r = __builtin_popcountll(all & ((1ull << lane) - 1));
#pragma unroll
    for (int j = 0; j < EPL; ++j) lds.score[r * ROW + j] = key[j];
    lds.group[r] = __int_as_float(lane * EPL);
  }
  wave_sync();
  const int r = lane >> 1, half = (lane & 1) * H;
  float mine[H];
#pragma unroll
  for (int j = 0; j < H; ++j) mine[j] = r < count ? lds.score[r * ROW + half + j] : kNegInf;
  const int first = r < count ? __float_as_int(lds.group[r]) + half : 0;
  return lanes_max<LPT>(choose<LPT, H, float>(mine, rounds, lane, first, ids, keys));
}

template <bool BF16, int LPT, int EPL, int V, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  using R = Row<BF16, LPT, EPL, V>;
  constexpr int TPB = 256 / LPT, JPL = kJpl<LPT>;
  uint32_t closed = 0;
  __shared__ float s_logit[TPB][kSlots];
  __shared__ int s_id[TPB][kSlots];
  __shared__ float s_key[BIAS ? TPB : 1][kSlots];
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

  // (a NaN in the softmax's sum leaves the choice among the others)
  float valid = total;
  if ((BIAS || GROUPS) && a.softmax && __any(!(total == total))) {
    valid = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) valid += x[j] == x[j] ? fast_exp(x[j] - top) : 0.0f;
    valid = lanes_sum<LPT>(valid);
  }
  const float rt = 1.0f / valid;
  auto score_of = [&](float l) __attribute__((always_inline)) { return a.softmax ? fast_exp(l - top) * rt : fast_sigmoid(l); };

  float key[EPL];
  // the `rounds` best, and the best that is left
  auto best_of = [&](auto& scratch, int rounds, float* keys) __attribute__((always_inline)) {
    if constexpr (GROUPS && EPL >= 8) {
      if (a.group_lanes && 2 * a.top_groups * a.group_lanes <= LPT)
        return choose_open<LPT, EPL>(a, scratch[slot], key, !closed, rounds, lane, s_id[slot], keys);
    }
    if constexpr (GROUPS) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = closed >> j & 1 ? kNegInf : key[j];
    }
    return lanes_max<LPT>(choose<LPT, EPL, float>(key, rounds, lane, lane * EPL, s_id[slot], keys));
  };
  __shared__ GroupScratch<LPT, GROUPS ? EPL : 1> scratch[GROUPS ? TPB : 1];
  if constexpr (!BIAS) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = x[j] > kNegInf ? x[j] : kNegInf;
    if constexpr (GROUPS) {
      closed = closed_groups<R, true>(a, scratch[slot], x, key, score_of, top, row, lane);
    }
    best_of(scratch, k, s_logit[slot]);            // (the keys are the logits)
    wave_sync();
  } else {
    // (the score's choice outside of the loop: inside it every key waits for the one
    // before; fmaf by name, since equal numbers have to give equal keys and the
    // compiler by itself fuses the sums of some of them)
    auto keys_of = [&](auto plus) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < R::NI; ++i) {
        typedef float vec __attribute__((ext_vector_type(V), aligned(4)));
        const int e = R::expert(lane, i, 0);
        const vec bv = *reinterpret_cast<const vec*>(a.bias + (e < a.experts ? e : 0));   // (whole groups of V exist)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int j = i * V + v;
          key[j] = x[j] == kNegInf ? kNegInf : fmaxf(plus(x[j], bv[v]), kNegInf);    // (NaN: -inf)
        }
      }
    };
    if (a.softmax) keys_of([&](float l, float b) __attribute__((always_inline)) { return fmaf(fast_exp(l - top), rt, b); });
    else keys_of([&](float l, float b) __attribute__((always_inline)) { return fast_sigmoid(l) + b; });
    if constexpr (GROUPS) {
      closed = closed_groups<R, false>(a, scratch[slot], x, key, score_of, top, row, lane);
    }
    const int cand = min(k + kSpare, a.experts);
    const float rest = best_of(scratch, cand, s_key[slot]);
    wave_sync();
    auto fetch_logits = [&](int n) __attribute__((always_inline)) {
      for (int j = lane; j < n; j += LPT) {
        const int e = s_id[slot][j];
        s_logit[slot][j] = e >= 0 ? R::one(a.logits, row, a.experts, e) : kNegInf;
      }
      wave_sync();
    };
    fetch_logits(cand);
    // Choice j against the next: clear, of the same numbers (`same`), in doubt
    // (`near`): a bit each.
    const float kp = 2.0f * key_p(a);
    uint64_t near = 0, same = 0;
    for (int j0 = 0; j0 < cand; j0 += LPT) {
      const int j = j0 + lane;
      bool n = false, e = false;
      if (j < cand) {
        const float k0 = s_key[slot][j], k1 = j + 1 < cand ? s_key[slot][j + 1] : rest;
        n = k1 > kNegInf && !(k0 - k1 > kp + kKeySum * (fabsf(k0) + fabsf(k1)));
        if (n && j + 1 < cand && s_logit[slot][j] == s_logit[slot][j + 1] &&
            a.bias[s_id[slot][j]] == a.bias[s_id[slot][j + 1]]) {
          n = false;
          e = true;
        }
      }
      near |= token_ballot<LPT>(n) << j0;
      same |= token_ballot<LPT>(e) << j0;
    }
    const uint64_t tied = near | same;
    if (__any((tied & ((1ull << k) - 1)) != 0)) {
      const int m = min(cand, k + __builtin_ctzll(~(tied >> (k - 1))));      // choices up to the next clear gap
      const bool open = tied >> (m - 1) & 1;
      const bool doubt = (near & ((1ull << m) - 1)) != 0;
      if (__any(doubt)) {
        const bool all = __any(doubt && open);
        double exact[EPL];
        double dt = 1.0;                           // (and fma by name, as for the keys in fp32)
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
            const double q = fma(exact[j], dt, static_cast<double>(a.bias[e < a.experts ? e : 0]));
            exact[j] = x[j] > kNegInf && !(closed >> j & 1) && q > -__builtin_inf() ? q : -__builtin_inf();
          }
          choose<LPT, EPL, double>(exact, k, lane, lane * EPL, s_id[slot], nullptr);
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
              mine[i] = fma(a.softmax ? exp(l - top) : 1.0 / (1.0 + exp(-l)), dt, static_cast<double>(a.bias[id[i]]));
              s_exact[slot][j] = mine[i];
            }
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < N; ++i) {
            rank[i] = 0;
            if (!__any(id[i] >= 0)) continue;        // (the waves in doubt are the last to end)
#pragma unroll 4
            for (int j = 0; j < m; ++j) {
              const double o = s_exact[slot][j];
              const int oid = s_id[slot][j];
              rank[i] += (oid >= 0) & ((o > mine[i]) | ((o == mine[i]) & (oid < id[i])));
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
  // The choices go to their experts' places by LDS, unless two of them are one
  // expert's, which shows where each has written its number: those are added in
  // their order.  (Every lane looking at every choice took 7.0 instead of 5.3 us,
  // 16381 x 256, and 4.7 instead of 4.3 of 64 experts.)
  constexpr int PITCH = EPL + 4;                  // (16 bytes more: a row's lanes meet no bank twice)
  typedef float v4f __attribute__((ext_vector_type(4)));
  __shared__ __attribute__((aligned(16))) float s_row[TPB][LPT * PITCH];
  float* const own = s_row[slot] + lane * PITCH;
#pragma unroll
  for (int q = 0; q < EPL; q += 4) *reinterpret_cast<v4f*>(own + q) = v4f{};
  wave_sync();
  auto place = [&](int e) __attribute__((always_inline)) { return s_row[slot] + e / EPL * PITCH + e % EPL; };
#pragma unroll
  for (int i = 0; i < JPL; ++i)
    if (id[i] >= 0) *place(id[i]) = __int_as_float(lane + i * LPT);
  wave_sync();
  bool twice = false;
#pragma unroll
  for (int i = 0; i < JPL; ++i)
    if (id[i] >= 0) twice |= __float_as_int(*place(id[i])) != lane + i * LPT;
  wave_sync();
  if (!__any(twice)) {
#pragma unroll
    for (int i = 0; i < JPL; ++i)
      if (id[i] >= 0) *place(id[i]) = s_d[slot][lane + i * LPT] + 0.0f;
    wave_sync();
#pragma unroll
    for (int q = 0; q < EPL; q += 4) {
      const v4f v = *reinterpret_cast<const v4f*>(own + q);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[q + e] = v[e];
    }
  } else {
    for (int j = 0; j < k; ++j) {
      const int e = s_id[slot][j];
      const float d = s_d[slot][j];
#pragma unroll
      for (int q = 0; q < EPL; ++q) out[q] += R::expert(lane, q / V, q % V) == e ? d : 0.0f;
    }
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
  else if (a.bias && a.groups > 1) hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, true, true>), grid, block, 0, s, a);
  else if (a.bias) hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, true, false>), grid, block, 0, s, a);
  else if (a.groups > 1) hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<BF16, LPT, EPL, V, false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Accesses of up to 16 bytes where every token's logits start on such a
// boundary (the host checks that the tensors do), else one element each.
template <bool BF16, int LPT, int EPL>
hipError_t launch_width(const RouteArgs& args, bool backward, hipStream_t s) {
  RouteArgs a = args;
  const int lanes = a.experts / a.groups / EPL;
  a.group_lanes = a.experts / a.groups % EPL == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  constexpr int V = EPL < (BF16 ? 8 : 4) ? EPL : (BF16 ? 8 : 4);
  return a.experts % V == 0 ? launch_shape<BF16, LPT, EPL, V>(a, backward, s)
                            : launch_shape<BF16, LPT, EPL, 1>(a, backward, s);
}
template <bool BF16>
hipError_t launch_size(const RouteArgs& a, bool backward, hipStream_t s) {
  if (a.experts <= 64) return launch_width<BF16, 16, 4>(a, backward, s);
  // Few tokens leave most of the chip empty: a wave a token then, whose keys are
  // half or a quarter as many a lane.  us by a wave a token / by 16 lanes, BF16, top
  // 8, without a bias, and of the gradient:
  //   128 experts,    1 token    3.6 / 3.9    2.6 / 2.7
  //                1024 tokens   4.0 / 4.25   3.0 / 3.0
  //                1536          4.4 / 4.2    3.2 / 3.0
  //                2048          4.4 / 4.2    3.2 / 3.1
  //   256 experts,    1          3.7 / 5.5    2.6 / 2.8
  //                1024          4.0 / 5.8    2.9 / 3.2
  //                2048          4.4 / 5.6    3.3 / 3.25
  //                4096          5.6 / 5.6    3.5 / 3.5
  // (96 experts are as 128, 160 as 256.)
  if (a.experts <= 256 && a.tokens <= (a.experts <= 128 ? 1024 : 2048)) return launch_width<BF16, 64, 4>(a, backward, s);
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
