// Routing with a bias for balance and groups of experts, and its backward.
//
//   s_i = softmax(l)_i or sigmoid(l_i)      v_i = s_i + b_i        (b only decides the choice)
//   v_i = -infinity where l_i is: a masked expert stays behind the others whatever its bias
//   a group's score: the sum of its one or two largest v; the best groups stay
//   the k largest v of those are chosen, in order; ties go to the lower index
//   w_j = c s_j, or c s_j / sum of the chosen s
//
// Choice. v is formed in 64 bits: two scores that differ in float32's last bits decide which expert
// a token goes to, and sigmoid saturates in float32. A candidate is one positive double, its key:
// v's bits in an order-preserving form, the lowest ten replaced by 1023 - index. The largest key is
// then the largest v (to 2^-41 of it) with the lower index first, and a maximum is one v_max_f64.
// Without a bias, and where no two scores are added, the logits stand in for the scores: they order the
// experts as the scores do, and go on doing so where scores saturate or fall out of 64 bits, as the
// choice of moe_route does.
//
// L lanes work on a token, 16 where there are many tokens of no more than 256 experts, so that a
// wave's rounds of the top-k serve four tokens, else a wave; expert i belongs to lane i % L. The
// kernel is bound by instructions (64-bit exponentials and k rounds over the keys), not by its
// 4 E + 8 k bytes a token: 8192 tokens, 8 of 256 experts in 8 groups, 11 to 12 us where the bytes take
// 1.7; one token 4.6 us.
#include <algorithm>

#include "device_common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kRouteBlock = 256;
constexpr int kMaxGroups = 64;

// ---- reductions over the L lanes of a token (16: a DPP row; 64: the wave); every lane gets the result
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  // every lane of the row is active: nothing else is left in the result
  const uint32_t lo = __builtin_amdgcn_mov_dpp(static_cast<int>(static_cast<uint32_t>(b)), CTRL, 0xF,
                                               0xF, false);
  const uint32_t hi = __builtin_amdgcn_mov_dpp(static_cast<int>(static_cast<uint32_t>(b >> 32)), CTRL,
                                               0xF, 0xF, false);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b)), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b >> 32)), lane);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// Largest and smallest of two numbers of which neither is NaN (the builtins would put both operands
// through an instruction of its own that quiets NaNs).
__device__ __forceinline__ double max_f64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min_f64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
template <int L, typename T, typename Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
  if constexpr (sizeof(T) == 8) {
    v = op(v, dpp_f64<kDppSwap1>(v));
    v = op(v, dpp_f64<kDppSwap2>(v));
    v = op(v, dpp_f64<kDppHalfMirror>(v));
    v = op(v, dpp_f64<kDppMirror>(v));
    if constexpr (L == 64)
      v = op(op(readlane_f64(v, 0), readlane_f64(v, 16)), op(readlane_f64(v, 32), readlane_f64(v, 48)));
  } else {
    v = op(v, dpp_f32<kDppSwap1>(v));
    v = op(v, dpp_f32<kDppSwap2>(v));
    v = op(v, dpp_f32<kDppHalfMirror>(v));
    v = op(v, dpp_f32<kDppMirror>(v));
    if constexpr (L == 64)
      v = op(op(readlane_f32(v, 0), readlane_f32(v, 16)), op(readlane_f32(v, 32), readlane_f32(v, 48)));
  }
  return v;
}
template <int L, typename T>
__device__ __forceinline__ T lanes_max(T v) {
  return lanes_reduce<L>(v, [](T a, T b) __attribute__((always_inline)) {
    if constexpr (sizeof(T) == 8) return max_f64(a, b);
    else return fmaxf(a, b);
  });
}
template <int L, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
  return lanes_reduce<L>(v, [](T a, T b) __attribute__((always_inline)) { return a + b; });
}

// The key of candidate idx with value v: positive, finite, larger for a larger v and, where v is the
// same, for a lower idx. NaN ranks below -infinity. |v| < 2^1023 (float32 sums are).
__device__ __forceinline__ double route_key(double v, int idx) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 as 0
  uint64_t o = (b >> 63) ? ~b : (b | (uint64_t{1} << 63));
  // an infinite v gives the largest finite key
  o = min(o, uint64_t{0xFFBFFFFFFFFFFFFFull});
  if (v != v) o = 0;
  o = (o >> 1) + (uint64_t{1} << 52);  // above every taken candidate's key, which has no exponent
  return __builtin_bit_cast(double, (o & ~uint64_t{1023}) | static_cast<uint64_t>(1023 - idx));
}
__device__ __forceinline__ int key_index(double key) {
  return 1023 - static_cast<int>(__builtin_bit_cast(uint64_t, key) & 1023);
}

// e^x to 2^-45 for |x| <= 708, larger |x| taken as 708 (e^-708 is 0 beside any other score): x is cut
// at a multiple of ln 2, taken off in two parts (Cody and Waite's reduction, Software Manual for the
// Elementary Functions, 1980), and the rest (at most ln 2 / 2) goes through the Taylor polynomial of
// degree 12, whose next term is below 2^-52. Equal arguments give equal values, so ties stay ties.
__device__ __forceinline__ double route_exp(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -708.0), 708.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  // the first 15 bits of ln 2, so that n times them is exact, and what is left of it
  constexpr double high = 22713.0 / 32768, low = 1.4286068203094172e-06;
  double r = __builtin_fma(n, -high, x);
  r = __builtin_fma(n, -low, r);
  constexpr double c[] = {1.0 / 479001600, 1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320,
                          1.0 / 5040,      1.0 / 720,      1.0 / 120,     1.0 / 24,     1.0 / 6,
                          0.5,             1.0,            1.0};
  double y = c[0];
#pragma unroll
  for (int i = 1; i < 13; ++i) y = __builtin_fma(y, r, c[i]);
  return __builtin_ldexp(y, static_cast<int>(n));
}
// 1 / x for x in [1, 2^1023): the hardware's estimate and two steps of Newton's method.
__device__ __forceinline__ double route_rcp(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
  return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}

// ---- weights of the chosen. Lane j < k of a token holds slot j's logit l; the others hold
// -infinity. Ratios are formed so that neither a large negative row nor an
// overflowing exponential turns them into 0 / 0: with m the largest chosen logit,
//   sigmoid(l) / sigmoid(m) = e^(l-m) (1 + e^m) / (1 + e^l)   for m <= 0,  sigmoid itself above.
// A row whose chosen logits are all -infinity gets weights 0; logits of +infinity share the whole of a
// softmax.
__device__ __forceinline__ float sigmoid_precise(float l) { return 1.0f / (1.0f + expf(-l)); }
// e^(l - m) for l <= m, 1 where both are the same infinity
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

template <int L>
__device__ __forceinline__ float renorm_weight(float l, bool act, int sigmoid, float c) {
  const float m = lanes_max<L>(l);
  if (m == -INFINITY) return 0.f;
  float e;
  if (!sigmoid) {
    e = act ? exp_below(l, m) : 0.f;
  } else if (m > 0.f) {
    e = act ? sigmoid_precise(l) : 0.f;
  } else {
    e = act ? expf(l - m) * (1.0f + expf(m)) / (1.0f + expf(l)) : 0.f;
  }
  return c * e / lanes_sum<L>(e);
}

template <int L, int NV>
__global__ __launch_bounds__(kRouteBlock) void route_grouped_kernel(
    moe_grouped_router r, const float* __restrict__ logits, const float* __restrict__ bias,
    int32_t* __restrict__ ids, float* __restrict__ w) {
  constexpr int TPB = kRouteBlock / L;  // tokens a block
  // a token's values with a gap after each group, so that the lanes that scan the groups of a token
  // do not meet in a bank
  constexpr int ROW = L * NV + kMaxGroups + 1;  // the last place is written and not read
  __shared__ double vals[TPB * ROW];
  __shared__ double gscore[TPB * (L == 16 ? 16 : kMaxGroups)];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool there = t < r.T;
  const int E = r.E;
  const float* l = logits + (there ? t : 0) * E;  // lanes past the last token repeat the first
  float lg[NV];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + L * i;
    lg[i] = l[min(e, E - 1)];  // loads without branches; what lies past the row is put aside
    if (e >= E) lg[i] = -INFINITY;
    mx = fmaxf(mx, lg[i]);
  }
  mx = lanes_max<L>(mx);
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  const bool by_logit = !bias && (r.groups == 1 || r.group_top == 1);
  double v[NV];
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = static_cast<double>(lg[i]);
  } else {
    // sigmoid(l) = 1 / (1 + e^-l); softmax from l - max, whose exponential is 1 at the largest logit,
    // an infinite one too. A logit of -infinity adds nothing to the sum and gives v = -infinity after
    // the bias, NaN stays NaN.
    const double shift = sigmoid || mx == -INFINITY ? 0.0 : static_cast<double>(mx);
    const double sign = sigmoid ? -1.0 : 1.0, one = sigmoid ? 1.0 : 0.0;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = one + route_exp((static_cast<double>(lg[i]) - shift) * sign);
      if (lg[i] == mx && !sigmoid) v[i] = 1.0;
      if (lg[i] == -INFINITY && !sigmoid) v[i] = 0.0;
      sum += v[i];
    }
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = route_rcp(v[i]);
    } else {
      sum = lanes_sum<L>(sum);
      // below 1 only where no logit is a number above -infinity
      const double inv = sum >= 1.0 ? route_rcp(sum) : 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lg[i] != lg[i]) v[i] = static_cast<double>(lg[i]);
    if (bias) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] += static_cast<double>(bias[min(lane + L * i, E - 1)]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lg[i] == -INFINITY) v[i] = -INFINITY;
  }
  double key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + L * i;
    key[i] = route_key(v[i], e);
    if (e >= E) key[i] = 0.0;
  }
  if (r.groups > 1) {
    const int gs = E / r.groups;
    const float inv_gs = 1.0f / static_cast<float>(gs);
    // e / gs: half an expert keeps the product off the borders by far more than its rounding
    auto group_of = [&](int e) __attribute__((always_inline)) {
      return static_cast<int>((static_cast<float>(e) + 0.5f) * inv_gs);
    };
    double* row = vals + slot * ROW;
    double* sc = gscore + slot * (L == 16 ? 16 : kMaxGroups);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + L * i;
      row[e < E ? e + group_of(e) : ROW - 1] = v[i];
    }
    __syncthreads();
    // a group's experts are looked through by S lanes (1, 2, 4 or 8), which then merge their two best
    const int S = r.groups * 8 <= L ? 8 : r.groups * 4 <= L ? 4 : r.groups * 2 <= L ? 2 : 1;
    const int group = lane / S;
    double a = -INFINITY, b = -INFINITY;  // the largest and the second
    if (group < r.groups) {
      const double* g = row + group * (gs + 1);
#pragma unroll 4
      for (int i = lane & (S - 1); i < gs; i += S) {
        const double x = g[i] != g[i] ? -INFINITY : g[i];
        b = max_f64(b, min_f64(a, x));
        a = max_f64(a, x);
      }
    }
    auto merge = [&](double oa, double ob) __attribute__((always_inline)) {
      b = max_f64(min_f64(a, oa), max_f64(b, ob));
      a = max_f64(a, oa);
    };
    if (S >= 2) merge(dpp_f64<kDppSwap1>(a), dpp_f64<kDppSwap1>(b));
    if (S >= 4) merge(dpp_f64<kDppSwap2>(a), dpp_f64<kDppSwap2>(b));
    if (S >= 8) merge(dpp_f64<kDppHalfMirror>(a), dpp_f64<kDppHalfMirror>(b));
    double mine = r.group_top == 2 && gs > 1 ? a + b : a;
    if (mine != mine) mine = -INFINITY;
    const bool head = group < r.groups && (lane & (S - 1)) == 0;
    if (head) sc[group] = mine;
    __syncthreads();
    int rank = 0;
#pragma unroll 8
    for (int h = 0; h < r.groups; ++h) {
      const double o = sc[h];
      rank += o > mine || (o == mine && h < group);
    }
    // Sums of -infinity (fewer than two free experts): the largest v decides between those. Lanes of a
    // token are in one wave, and rows without masks skip this.
    if (r.group_top == 2 && __any(head && mine == -INFINITY)) {
      const int first = threadIdx.x % kWave / L * L;
      rank = 0;
      for (int h = 0; h < r.groups; ++h) {
        const double o = sc[h], oa = __shfl(a, first + h * S, kWave);
        const bool tie = o == mine, best = tie && o == -INFINITY && oa != a;
        rank += best ? oa > a : o > mine || (tie && h < group);
      }
    }
    // bit g S of this token's lanes: group g stays
    uint64_t kept = __ballot(head && rank < r.topk_groups);
    if (L < 64) kept >>= threadIdx.x % kWave / L * L;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + L * i;
      if (!((kept >> (group_of(min(e, E - 1)) * S)) & 1)) key[i] = 0.0;
    }
  }
  int id = 0;
  for (int j = 0; j < r.k; ++j) {
    double m[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) m[i] = key[i];
#pragma unroll
    for (int n = NV; n > 1; n >>= 1)
#pragma unroll
      for (int i = 0; i < n / 2; ++i) m[i] = max_f64(m[i], m[i + n / 2]);
    const int idx = key_index(lanes_max<L>(m[0]));
    if (lane == j) id = idx;
    // taken: without its upper half a key is below every other
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t b = __builtin_bit_cast(uint64_t, key[i]);
      if (idx == lane + L * i) b &= 0xffffffffu;
      key[i] = __builtin_bit_cast(double, b);
    }
  }
  const bool act = lane < r.k;
  const float chosen = act ? l[id] : -INFINITY;
  float wj;
  if (r.renorm) {
    wj = renorm_weight<L>(chosen, act, sigmoid, r.scale);
  } else if (sigmoid) {
    wj = r.scale * sigmoid_precise(chosen);
  } else {
    float s = 0.f;
    const float m = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += exp_below(lg[i], m);
    s = lanes_sum<L>(s);
    wj = s == 0.f ? 0.f : r.scale * (exp_below(chosen, m) / s);
  }
  if (there && act) {
    ids[t * r.k + lane] = id;
    w[t * r.k + lane] = wj;
  }
}

// d logits from the gradient D at the weights, which reaches the scores of the chosen alone:
//   renormalised, p_j = s_j / sum of the chosen s
//     softmax   dl_j = c p_j (D_j - sum_i D_i p_i)
//     sigmoid   the same times 1 - s_j = sigmoid(-l_j)
//   as they are, p = s
//     softmax   dl_i = c p_i (D_i - sum_j D_j p_j) for every expert i (D_i = 0 where not chosen)
//     sigmoid   dl_j = c D_j s_j (1 - s_j)
// A token's row is put together in LDS: zeros, the chosen over them, and out in whole lines. Only
// softmax as it is reads the row of logits; the others read the chosen k alone. Bound by the row
// written (16384 tokens, 8 of 128 experts, renormalised: 4.3 us, 4 TB/s in and out).
template <int L, int NV>
__global__ __launch_bounds__(kRouteBlock) void route_grouped_bwd_kernel(
    moe_grouped_router r, const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, float* __restrict__ dlogits) {
  constexpr int TPB = kRouteBlock / L, ROW = L * NV;
  __shared__ float rows[TPB * ROW];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + slot;
  const bool there = t < r.T;
  const int E = r.E, k = r.k;
  const int64_t tt = there ? t : 0;
  const float* l = logits + tt * E;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID, act = lane < k;
  int id = 0;
  float chosen = -INFINITY, d = 0.f;
  if (act) {
    id = ids[tt * k + lane];
    // ids come from the forward; one out of range (a caller's error) stays in bounds
    if (id < 0 || id >= E) id = 0;
    chosen = l[id];
    d = dw[tt * k + lane];
  }
  float* row = rows + slot * ROW;
#pragma unroll
  for (int i = 0; i < NV; ++i) row[lane + L * i] = 0.f;
  const bool full = !sigmoid && !r.renorm;
  float lg[NV];
  if (full) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      lg[i] = l[min(lane + L * i, E - 1)];
      if (lane + L * i >= E) lg[i] = -INFINITY;
    }
  }
  __syncthreads();
  float u = r.scale * d;
  if (r.renorm) {
    const float p = renorm_weight<L>(chosen, act, sigmoid, 1.0f);
    const float mean = lanes_sum<L>(act ? u * p : 0.f);
    u = p * (u - mean);
    // a chosen logit of -infinity has the weight 0 and no gradient
    if (sigmoid) u *= sigmoid_precise(-chosen);
    if (p == 0.f) u = 0.f;
  } else if (sigmoid) {
    u *= sigmoid_precise(chosen) * sigmoid_precise(-chosen);
  }
  if (act) row[id] = u;
  __syncthreads();
  float out[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) out[i] = row[lane + L * i];
  if (full) {
    float m = lg[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, lg[i]);
    m = lanes_max<L>(m);
    if (m == -INFINITY) m = 0.f;
    float s = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      lg[i] = exp_below(lg[i], m);
      s += lg[i];
      dot = fmaf(lg[i], out[i], dot);
    }
    s = lanes_sum<L>(s);
    const float inv = s == 0.f ? 0.f : 1.0f / s;
    dot = lanes_sum<L>(dot) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = lg[i] * inv * (out[i] - dot);
  }
  if (there) {
    float* o = dlogits + t * E;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + L * i < E) o[lane + L * i] = out[i];
  }
}

// Calls go with the lanes a token takes and the experts a lane holds.
template <typename F>
hipError_t by_experts(const moe_grouped_router& r, F&& go) {
  using std::integral_constant;
  typedef integral_constant<int, 16> L16;
  typedef integral_constant<int, 64> L64;
  // 16 lanes hold up to 16 slots and 16 groups. Up to 4096 tokens leave lanes idle either way, and a
  // token's chain of steps is shorter with a wave of its own (256 experts in 8 groups, 2048 tokens:
  // 7.0 us against 8.7 with 16 lanes; 4096: 9.0 against 8.9; 8192: 15.2 against 12.1).
  if (r.E <= 256 && r.k <= 16 && r.groups <= 16 && r.T > 4096) {
    if (r.E <= 32) return go(L16(), integral_constant<int, 2>());
    if (r.E <= 64) return go(L16(), integral_constant<int, 4>());
    if (r.E <= 128) return go(L16(), integral_constant<int, 8>());
    return go(L16(), integral_constant<int, 16>());
  }
  if (r.E <= 64) return go(L64(), integral_constant<int, 1>());
  if (r.E <= 256) return go(L64(), integral_constant<int, 4>());
  return go(L64(), integral_constant<int, 16>());
}

// Calls go(first token, router of the launch's tokens, grid) for launches of at most 2^31 threads (a
// grid holds fewer than 2^32).
template <int L, typename F>
hipError_t in_parts(moe_grouped_router r, F&& go) {
  constexpr int TPB = kRouteBlock / L;
  constexpr int64_t part = (int64_t{1} << 31) / L;
  const int64_t T = r.T;
  for (int64_t t = 0; t < T; t += part) {
    r.T = static_cast<int32_t>(std::min(part, T - t));
    go(t, r, dim3(static_cast<unsigned>((static_cast<int64_t>(r.T) + TPB - 1) / TPB)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route_grouped(const moe_grouped_router& r, const float* logits,
                                const float* bias, int32_t* ids, float* w, hipStream_t s) {
  return by_experts(r, [&](auto lanes, auto nv) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
    return in_parts<L>(r, [&](int64_t t, const moe_grouped_router& q, dim3 grid) {
      hipLaunchKernelGGL((route_grouped_kernel<L, NV>), grid, dim3(kRouteBlock), 0, s, q,
                         logits + t * r.E, bias, ids + t * r.k, w + t * r.k);
    });
  });
}

hipError_t launch_route_grouped_bwd(const moe_grouped_router& r, const float* logits,
                                    const int32_t* ids, const float* dw, float* dlogits,
                                    hipStream_t s) {
  return by_experts(r, [&](auto lanes, auto nv) {
    constexpr int L = decltype(lanes)::value, NV = decltype(nv)::value;
    return in_parts<L>(r, [&](int64_t t, const moe_grouped_router& q, dim3 grid) {
      hipLaunchKernelGGL((route_grouped_bwd_kernel<L, NV>), grid, dim3(kRouteBlock), 0, s, q,
                         logits + t * r.E, ids + t * r.k, dw + t * r.k, dlogits + t * r.E);
    });
  });
}

}  // namespace moe
