// The experts of every token from the router's logits x [M, E]:
//   s   = softmax(x) or 1 / (1 + exp(-x))
//   key = s + bias, or s, or, where only the order of x counts, x itself
//   the best topk_group of n_group groups by the sum of a group's best group_top keys
//   the topk largest keys of those, ties to the lowest index
//   w   = scale * s[pick] (/ the sum of s over the picks)
//
// One wavefront a row; lane i holds the experts i, i + 64, ..., each lane's
// sorted, so that a pick is one maximum over the lanes' first keys and one lane's
// step to its next.  Bound by those steps (some 20 instructions a pick) and by the
// loads of x.
//
// Which of two nearly equal scores is larger must not hang on a rounding: keys
// are computed in fp32, and a row where two keys that decide something are closer
// than fp32's error is done again in fp64 by the same wavefront.  Keys that are x
// itself are exact.
#include <algorithm>

#include "base.h"
#include "common.h"
#include "internal.h"

namespace mlr {
namespace {

constexpr int kWaves = 4;  // of a workgroup, a row each

// Partner's value in a butterfly step, 32 or 64 bits.
template <typename T>
__device__ __forceinline__ T partner(T v, int o) {
  if constexpr (sizeof(T) == 4) {
    return butterfly_partner(v, o);
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __float_as_uint(butterfly_partner(__uint_as_float(uint32_t(u)), o));
    const uint32_t hi = __float_as_uint(butterfly_partner(__uint_as_float(uint32_t(u >> 32)), o));
    return __builtin_bit_cast(T, uint64_t(hi) << 32 | lo);
  }
}
template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const T u = partner(v, o);
    v = u > v ? u : v;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += partner(v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T from_lane(T v, int src) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), src));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u)), src));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u >> 32)), src));
    return __builtin_bit_cast(T, uint64_t(hi) << 32 | lo);
  }
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// exp(x - m), also where both are the same infinity
template <typename T>
__device__ __forceinline__ T exp_from(T x, T m) {
  return x == m ? T(1) : exp_of(x - m);
}

template <typename T>
constexpr T kNone = -T(__builtin_huge_val());  // masked, or picked already

// Whether fp32 leaves open which of two keys a >= b is larger.  A score is off by
// less than 2^-19: by the exponential (its argument's rounding |d| 2^-24 exp(d) and
// its own, below 2^-22 of values up to 1), the sum (22 additions at most) and the
// quotient; the bias adds a rounding of the key, a group's sum another.
__device__ __forceinline__ bool open_between(float a, float b) {
  return b > kNone<float> && !(a - b > 0x1p-17f + 0x1p-21f * fmaxf(fabsf(a), fabsf(b)));
}
__device__ __forceinline__ bool open_between(double, double) { return false; }

struct Picks {
  int id;       // lane r: the r-th pick, or -1
  bool open;    // (fp32) some decision is open
};

// Picks by `key` (key[j] is expert 64 j + lane's; kNone: masked).  With CHECKED
// fp32 keys, ends where a decision is open.
template <typename T, int V, bool CHECKED>
__device__ __forceinline__ Picks pick(const RouteParams& p, T (&key)[V], T* lds) {
  const int lane = lane_id();
  constexpr bool kCheck = CHECKED && sizeof(T) == 4;
  Picks out{-1, false};
  if (p.n_group > 1) {
    // 64 / n_group lanes (a power of two) a group: each finds the best two of its
    // part, a butterfly joins them
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (64 * j + lane < p.E) lds[64 * j + lane] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int lanes = 1 << (31 - __builtin_clz(uint32_t(kWave / p.n_group)));
    const int group = lane / lanes, sub = lane % lanes;
    T a = kNone<T>, b = kNone<T>;  // a >= b
    if (group < p.n_group) {
      for (int i = sub; i < p.size; i += lanes) {
        const T v = lds[group * p.size + i];
        b = v > a ? a : (v > b ? v : b);
        a = v > a ? v : a;
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      if (o >= lanes) continue;
      const T c = partner(a, o), d = partner(b, o);
      const T low = c > a ? a : c;
      a = c > a ? c : a;
      const T high = d > b ? d : b;
      b = low > high ? low : high;
    }
    if (p.group_top == 2 && b > kNone<T>) a += b;
    // a group's rank, and the scores on both sides of the cut
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const T v = from_lane(a, g * lanes);
      rank += v > a || (v == a && g < group);
    }
    const uint64_t kept = __ballot(sub == 0 && group < p.n_group && rank < p.topk_group);
    if (kCheck && p.topk_group < p.n_group) {
      const uint64_t in = __ballot(sub == 0 && group < p.n_group && rank == p.topk_group - 1);
      const uint64_t next = __ballot(sub == 0 && group < p.n_group && rank == p.topk_group);
      if (open_between(from_lane(a, __builtin_ctzll(in)), from_lane(a, __builtin_ctzll(next)))) {
        out.open = true;
        return out;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = 64 * j + lane;
      const uint32_t g = e * p.inv_size >> 20;
      if (e < uint32_t(p.E) && !(kept >> (g * lanes) & 1)) key[j] = kNone<T>;
    }
  }
  // each lane's keys in descending order, equal ones as they were
  int at[V];
#pragma unroll
  for (int j = 0; j < V; ++j) at[j] = j;
#pragma unroll
  for (int n = V - 1; n > 0; --n)
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const bool swap = key[j + 1] > key[j];
      const T k = key[j];
      const int t = at[j];
      key[j] = swap ? key[j + 1] : k;
      key[j + 1] = swap ? k : key[j + 1];
      at[j] = swap ? at[j + 1] : t;
      at[j + 1] = swap ? t : at[j + 1];
    }
  T last = kNone<T>;
  for (int r = 0; r < p.topk + (kCheck ? 1 : 0); ++r) {
    const T top = from_lane(wave_max(key[0]), 0);  // (a scalar)
    if (!(top > kNone<T>)) break;
    if (kCheck && r > 0 && open_between(last, top)) {
      out.open = true;
      return out;
    }
    if (r == p.topk) break;
    const uint64_t equal = __ballot(key[0] == top);
    int win = __builtin_ctzll(equal);
    if (equal & (equal - 1)) {  // the lowest index: the lowest of `at`, then of the lanes
#pragma unroll
      for (int j = V - 1; j >= 0; --j) {
        const uint64_t here = __ballot(key[0] == top && at[0] == j);
        if (here) win = __builtin_ctzll(here);
      }
    }
    const int id = 64 * __builtin_amdgcn_readlane(at[0], win) + win;
    if (lane == r) out.id = id;
    if (lane == win) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1], at[j] = at[j + 1];
      key[V - 1] = kNone<T>;
    }
    last = top;
  }
  return out;
}

// Keys that are scores (plus bias), in T.
template <typename T, int V>
__device__ __forceinline__ bool score_keys(const RouteParams& p, const float (&x)[V], float m, T (&key)[V]) {
  const int lane = lane_id();
  T s[V], sum = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    // a masked or missing expert has no share
    s[j] = !(x[j] > kNone<float>) ? T(0) : p.sigmoid ? T(1) / (T(1) + exp_of(-T(x[j]))) : exp_from(T(x[j]), T(m));
    sum += s[j];
  }
  if (!p.sigmoid) {
    sum = wave_sum(sum);
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] /= sum;
  }
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 64 * j + lane;
    key[j] = s[j];
    if (p.bias && e < p.E) key[j] += T(p.bias[e]);
    const bool live = x[j] > kNone<float>;
    nan |= live && key[j] != key[j];
    if (!live || key[j] != key[j]) key[j] = kNone<T>;
  }
  return nan;
}

template <typename X, int V, bool BY_SCORE>
__device__ __forceinline__ void route_row(const RouteParams& p, int64_t row, double* lds) {
  const int lane = lane_id();
  const X* logits = reinterpret_cast<const X*>(p.logits) + row * p.E;
  auto logit = [&](int e) {
    if constexpr (sizeof(X) == 2)
      return bf16_to_f32(logits[e]);
    else
      return logits[e];
  };
  float x[V];
  bool nan = false;
  float m = kNone<float>;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = 64 * j + lane;
    x[j] = e < p.E ? logit(e) : kNone<float>;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    nan |= x[j] != x[j];
    if (x[j] != x[j]) x[j] = kNone<float>;  // never picked
    m = x[j] > m ? x[j] : m;
  }
  m = wave_max(m);
  Picks picks;
  if constexpr (BY_SCORE) {
    float key[V];
    nan |= score_keys(p, x, m, key);
    picks = pick<float, V, true>(p, key, reinterpret_cast<float*>(lds));
    if (picks.open) {
      double wide[V];
      score_keys(p, x, m, wide);
      picks = pick<double, V, true>(p, wide, lds);
    }
  } else {
    float key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j];
    picks = pick<float, V, false>(p, key, reinterpret_cast<float*>(lds));
  }

  // The weights, a pick a lane.  Renormalised, the common factor cancels, and
  // everything is relative to the largest of the picks, so that none underflows.
  const bool have = picks.id >= 0;
  const float xr = have ? logit(picks.id) : kNone<float>;
  float s = 0.0f;
  if (p.renorm) {
    const float top = wave_max(xr);
    if (have) {
      if (!p.sigmoid) {
        s = exp_from(xr, top);
      } else if (xr > 0.0f) {
        s = 1.0f / (1.0f + expf(-xr));
      } else {
        s = exp_from(xr, fminf(top, 0.0f)) / (1.0f + expf(xr));
      }
    }
    const float sum = wave_sum(s);
    if (sum > 0.0f) s /= sum;
  } else if (p.sigmoid) {
    if (have) s = xr > 0.0f ? 1.0f / (1.0f + expf(-xr)) : expf(xr) / (1.0f + expf(xr));
  } else {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += x[j] > kNone<float> ? exp_from(x[j], m) : 0.0f;
    sum = wave_sum(sum);
    if (have) s = exp_from(xr, m) / sum;
  }
  s *= p.scale;
  if (__ballot(nan)) s = __builtin_nanf("");
  if (lane < p.topk) {
    p.ids[row * p.topk + lane] = picks.id;
    p.weights[row * p.topk + lane] = s;
  }
}

template <typename X, int V, bool BY_SCORE>
__global__ void __launch_bounds__(kWaves * kWave) route_kernel(RouteParams p) {
  __shared__ double lds[kWaves][BY_SCORE ? 64 * V : 32 * V];
  const int w = wave_id();
  for (int64_t row = int64_t(blockIdx.x) * kWaves + w; row < p.M; row += int64_t(gridDim.x) * kWaves)
    route_row<X, V, BY_SCORE>(p, row, lds[w]);
}
template <typename X, int V>
hipError_t route_launch(const RouteParams& p, hipStream_t st) {
  // (a launch has fewer than 2^32 threads: beyond that a wavefront takes several rows)
  const dim3 grid(unsigned(std::min<int64_t>((p.M + kWaves - 1) / kWaves, 1 << 22))), block(kWaves * kWave);
  if (p.bias || p.group_top == 2)
    hipLaunchKernelGGL((route_kernel<X, V, true>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((route_kernel<X, V, false>), grid, block, 0, st, p);
  return hipGetLastError();
}

template <typename X>
hipError_t route_of(const RouteParams& p, hipStream_t st) {
  if (p.E <= 64) return route_launch<X, 1>(p, st);
  if (p.E <= 128) return route_launch<X, 2>(p, st);
  if (p.E <= 256) return route_launch<X, 4>(p, st);
  if (p.E <= 512) return route_launch<X, 8>(p, st);
  return route_launch<X, 16>(p, st);
}

}  // namespace

hipError_t launch_route(const RouteParams& p, hipStream_t st) {
  return p.logits_bf16 ? route_of<uint16_t>(p, st) : route_of<float>(p, st);
}

}  // namespace mlr
