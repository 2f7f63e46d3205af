// The experts of every token from the router's logits x [M, E]:
//   s   = softmax(x) or 1 / (1 + exp(-x))
//   key = s + bias, or s, or, where only the order of x counts, x itself
//   the best topk_group of n_group groups by the sum of a group's best group_top keys
//   the topk largest keys of those, ties to the lowest index
//   w   = scale * s[pick] (/ the sum of s over the picks)
//
// One wavefront a row, V consecutive experts a lane, each lane's sorted, so that a
// pick is one maximum over the lanes' first keys and one lane's step to its next,
// and ties fall to the lowest lane.  Bound by those instructions: 65536 rows of 256
// experts in 8 groups 69 us, 480 vector instructions a row (some 22 a pick, 10 a
// score, 60 the groups), the vector units 71 % busy; without groups 56, by logits 36, one
// pick by logits 21 (3.2 TB/s).  8192 x 128 by logits 6.9 us.  A lane
// with every 64th expert instead of V in a row, picks by comparisons of floats and
// weights row by row took 110.
//
// Which of two nearly equal scores is larger must not hang on a rounding: keys
// are computed in fp32, and a row where two keys that decide something are closer
// than fp32's error is done again in fp64 by the same wavefront, when it has been
// through all its rows: at once, both passes' registers together leave four
// wavefronts a SIMD and not six (65536 x 256 in 8 groups 76 us and 69, 32768 x 64 23
// and 24).  Until then such a row's first id is kOpen.  Keys that are x itself are
// exact.
#include <algorithm>

#include "base.h"
#include "common.h"
#include "internal.h"

namespace mlr {
namespace {

constexpr int kWaves = 4;  // of a workgroup, a row each
constexpr int32_t kOpen = INT32_MIN;

// ---------------------------------------------------------------- keys
// fp32 keys are compared as unsigned integers in the same order, so that a step of
// a maximum over lanes is one instruction; fp64 ones as they are.
constexpr float kMasked = -__builtin_huge_valf();
constexpr float kMost = 3.4028234663852886e38f;

template <typename T>
constexpr T none();  // below every key: masked, or picked already
template <>
constexpr uint32_t none<uint32_t>() { return 0; }
template <>
constexpr double none<double>() { return -__builtin_huge_val(); }

// -infinity and NaN become none.
template <typename T, typename F>
__device__ __forceinline__ T key_of(F v) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t u = __float_as_uint(v);
    return v > kMasked ? u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u) : none<T>();
  } else {
    return v > F(kMasked) ? v : none<T>();
  }
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return k == none<uint32_t>() ? kMasked : __uint_as_float(k ^ (~uint32_t(int32_t(k) >> 31) | 0x80000000u));
}
__device__ __forceinline__ double value_of(double k) { return k; }

// ---------------------------------------------------------------- across lanes
// Partner's value in a butterfly step, 32 or 64 bits.
template <typename T>
__device__ __forceinline__ T partner(T v, int o) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, butterfly_partner(__builtin_bit_cast(float, v), o));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __float_as_uint(butterfly_partner(__uint_as_float(uint32_t(u)), o));
    const uint32_t hi = __float_as_uint(butterfly_partner(__uint_as_float(uint32_t(u >> 32)), o));
    return __builtin_bit_cast(T, uint64_t(hi) << 32 | lo);
  }
}
// `v` of lane `src` as a scalar.
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
// The largest of the wavefront, a scalar.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_step<0x111>(v);       // row_shr:1
  v = max_step<0x112>(v);       // row_shr:2
  v = max_step<0x114>(v);       // row_shr:4
  v = max_step<0x118>(v);       // row_shr:8
  v = max_step<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = max_step<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return from_lane(v, kWave - 1);
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const double u = partner(v, o);
    v = u > v ? u : v;
  }
  return from_lane(v, 0);
}
// Sum over the first `n` lanes (a power of two), in each of them.
template <typename T>
__device__ __forceinline__ T sum_over(T v, int n) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    if (o < n) v += partner(v, o);
  return v;
}

__device__ __forceinline__ float exp_of(float v) { return __expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float over_one(float v) { return __builtin_amdgcn_rcpf(v); }

// exp(x - m), also where both are the same infinity
template <typename T>
__device__ __forceinline__ T exp_from(T x, T m) {
  return x == m ? T(1) : exp_of(x - m);
}
__device__ __forceinline__ float exact_exp_from(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// Whether fp32 leaves open which of two keys a >= b is larger.  A sigmoid is off by
// less than 2^-22: s (1 - s) times the exponential's error (1.5 |x| 2^-24 for its
// argument, 2^-23 its own; |x| s (1 - s) < 1/4), the addition's 2^-24 and the
// reciprocal's 2^-23.  A softmax's share is off by less than 2^-18: up to 21 additions
// and the exponentials' errors (|d| < 8 on average) in the sum.  The bias adds a
// rounding of the key.
__device__ __forceinline__ bool open_between(float a, float b, int sigmoid) {
  return b > kMasked && !(a - b > (sigmoid ? 0x1p-20f : 0x1p-16f) + 0x1p-21f * fmaxf(fabsf(a), fabsf(b)));
}

// ---------------------------------------------------------------- picking
// A group's score, and the size of the keys in it: what their roundings go by, where
// two of opposite signs leave a small sum.
template <typename F>
struct GroupScore {
  F sum, size;
};

// Groups' ranks from their scores, the same in all `lanes` lanes of a group.
// Returns whether fp32 leaves the cut open: whether some group's score is nearer to
// the middle of the two next to the cut than it may be off, two keys' scores (see
// open_between) and three roundings of at most its size.  All are looked at, not
// those two alone: one group's keys may be far larger than the others'.
template <typename F>
__device__ __forceinline__ bool rank_groups(const RouteParams& p, const GroupScore<F>& of, int group, int lanes,
                                            int* rank) {
  const F score = of.sum;
  int r = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const F v = from_lane(score, g * lanes);
    r += v > score || (v == score && g < group);
  }
  *rank = r;
  if (p.topk_group == p.n_group) return false;
  const uint64_t in = __ballot(group < p.n_group && r == p.topk_group - 1);
  const uint64_t next = __ballot(group < p.n_group && r == p.topk_group);
  if constexpr (sizeof(F) == 4) {
    const float low = from_lane(score, __builtin_ctzll(next));
    if (!(low > kMasked)) return false;  // behind the cut all are empty
    const float cut = 0.5f * from_lane(score, __builtin_ctzll(in)) + 0.5f * low;
    const bool sure = fabsf(score - cut) > fmaf(0x1p-22f, of.size, p.sigmoid ? 0x1p-21f : 0x1p-17f);
    return __ballot(group < p.n_group && !sure) != 0;
  }
  return false;
}

// The best two of all keys of this lane's group, from those of a lane, a >= b; the
// group's score.
template <typename T>
__device__ __forceinline__ GroupScore<decltype(value_of(T()))> group_score(const RouteParams& p, T a, T b, int lanes) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (o >= lanes) continue;
    const T c = partner(a, o), d = partner(b, o);
    const T low = c > a ? a : c, high = d > b ? d : b;
    a = c > a ? c : a;
    b = low > high ? low : high;
  }
  auto s = value_of(a), size = s;
  if constexpr (sizeof(T) == 4) size = fabsf(s);
  if (p.group_top == 2 && b > none<T>()) {
    s += value_of(b);
    // a sum below fp32's range is no empty group's: two of them are left to fp64
    if constexpr (sizeof(T) == 4) s = fmaxf(s, -kMost), size += fabsf(value_of(b));
  }
  if constexpr (sizeof(T) == 4) size = fminf(size, kMost);  // (an empty group's is far from any cut)
  return {s, size};
}

// What another lane of this wavefront wrote to LDS before is read behind this.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The groups' ranks from keys in LDS, 64 / n_group lanes (a power of two) a group.
// Returns whether the cut is open; *kept has the bit of expert e's group at (its
// number << shift).
template <typename T>
__device__ __forceinline__ bool groups_in_lds(const RouteParams& p, const T* lds, int shift, uint64_t* kept) {
  const int lane = lane_id(), lanes = 1 << shift, group = lane >> shift;
  T a = none<T>(), b = none<T>();
  if (group < p.n_group) {
    for (int i = lane & (lanes - 1); i < p.size; i += lanes) {
      const T v = lds[group * p.size + i];
      b = v > a ? a : (v > b ? v : b);
      a = v > a ? v : a;
    }
  }
  int rank;
  const bool open = rank_groups(p, group_score(p, a, b, lanes), group, lanes, &rank);
  *kept = __ballot(rank < p.topk_group);
  return open;
}
__device__ __forceinline__ int group_lane_shift(const RouteParams& p) {
  return 31 - __builtin_clz(uint32_t(kWave / p.n_group));
}

// Picks by `key`; key[j] is expert V lane + j's.  The r-th goes to *id of lane
// `first` + r.  Returns whether some decision is left open; then *id may hold
// anything in these lanes.
template <int V, bool kCheck>
__device__ __forceinline__ bool pick(const RouteParams& p, uint32_t (&key)[V], uint32_t* lds, int first, int* id) {
  using T = uint32_t;
  const int lane = lane_id();
  // compared where they are needed: kept as masks across rows they would fill the
  // scalar registers
  int E = p.E, group_shift = p.group_shift, topk = p.topk;
  asm volatile("" : "+s"(E), "+s"(group_shift), "+s"(topk));
  // groups of a power of two lanes need no exchange through LDS
  const bool whole = group_shift >= 0;
  if (p.n_group > 1 && !whole) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (V * lane + j < E) lds[V * lane + j] = key[j];
    wave_sync();
    const int shift = group_lane_shift(p);
    uint64_t kept;
    if (groups_in_lds(p, lds, shift, &kept) && kCheck) return true;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = V * lane + j, g = e * p.inv_size >> 20;
      if (e < uint32_t(E) && !(kept >> (g << shift) & 1)) key[j] = none<T>();
    }
    wave_sync();  // the next row's keys go there
  }
  // this lane's keys in descending order, equal ones as they were, and where they
  // were, four bits each
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
  constexpr int kWords = (V + 7) / 8;
  uint32_t where[kWords] = {};
#pragma unroll
  for (int j = 0; j < V; ++j) where[j / 8] |= uint32_t(at[j]) << 4 * (j % 8);
  if (p.n_group > 1 && whole) {
    const int lanes = 1 << group_shift, group = lane >> group_shift;
    int rank;
    const bool open = rank_groups(p, group_score(p, key[0], V > 1 ? key[V > 1] : none<T>(), lanes), group, lanes,
                                  &rank);
    if (open && kCheck) return true;
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = rank < p.topk_group ? key[j] : none<T>();
  }
  T mine = none<T>(), beyond = none<T>();
  asm volatile("" : "+s"(topk));
  int r = 0;
  for (; r < topk; ++r) {
    const T top = wave_max(key[0]);
    if (!(top > none<T>())) break;
    const int win = __builtin_ctzll(__ballot(key[0] == top));
    const int e = V * win + int(uint32_t(__builtin_amdgcn_readlane(int(where[0]), win)) & 15);
    const bool here = lane == first + r;
    *id = here ? e : *id;
    if constexpr (kCheck) mine = here ? top : mine;
    const bool step = lane == win;
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = step ? (j + 1 < V ? key[j + 1 < V ? j + 1 : j] : none<T>()) : key[j];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t n = where[i] >> 4;
      if (i + 1 < kWords) n |= where[i + 1 < kWords ? i + 1 : i] << 28;
      where[i] = step ? n : where[i];
    }
  }
  if constexpr (kCheck) {
    if (r == topk) beyond = wave_max(key[0]);
    // (every lane takes part in the exchange, the last pick's too)
    const T below = __shfl_down(mine, 1), next = lane == first + topk - 1 ? beyond : below;
    return __ballot(uint32_t(lane - first) < uint32_t(topk) && open_between(value_of(mine), value_of(next), p.sigmoid));
  }
  return false;
}

// Keys that are scores (plus bias); whether an unmasked one is NaN.
template <int V>
__device__ __forceinline__ bool score_keys(const RouteParams& p, const float (&x)[V], const float (&bias)[V],
                                           float m, uint32_t (&key)[V]) {
  float s[V], sum = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    // a masked or missing expert has no share
    const float v = p.sigmoid ? over_one(1.0f + exp_of(-x[j])) : exp_from(x[j], m);
    s[j] = x[j] > kMasked ? v : 0.0f;
    sum += s[j];
  }
  if (!p.sigmoid) {
    sum = over_one(sum_over(sum, kWave));
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] *= sum;
  }
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float v = x[j] > kMasked ? s[j] + bias[j] : kMasked;
    nan |= v != v;
    key[j] = key_of<uint32_t>(v);
  }
  return nan;
}

// A row's logits, V consecutive ones a lane; what is not there is -infinity.
template <typename X, int V>
__device__ __forceinline__ void load_row(const RouteParams& p, const X* row, float (&x)[V]) {
  int e = V * lane_id();
  asm volatile("" : "+v"(e));  // addresses are not to be kept across rows: they take registers
  if (p.vectors) {  // (E is a multiple of V)
    constexpr int kBytes = V * int(sizeof(X)), kWords = (kBytes + 3) / 4;
    uint32_t q[kWords];
    const X* from = row + min(e, p.E - V);
    if constexpr (kBytes == 2) q[0] = *from;
    if constexpr (kBytes == 4) q[0] = *reinterpret_cast<const uint32_t*>(from);
    if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      q[0] = v.x, q[1] = v.y;
    }
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(from)[i / 4];
        q[i] = v.x, q[i + 1] = v.y, q[i + 2] = v.z, q[i + 3] = v.w;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float v = sizeof(X) == 4 ? __uint_as_float(q[j * sizeof(X) / 4])
                                     : __uint_as_float(j % 2 ? q[j / 2] & 0xffff0000u : q[j / 2] << 16);
      x[j] = e < p.E ? v : kMasked;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const X v = row[min(e + j, p.E - 1)];
      x[j] = e + j >= p.E ? kMasked : sizeof(X) == 4 ? float(v) : bf16_to_f32(uint16_t(v));
    }
  }
}

// What a lane holds between a row's picking and the weighing: its pick, and of the
// pick's row the largest logit, the sum of the softmax and whether there was NaN.
struct Lane {
  int id;
  float m, sum;
  bool nan;
};

// Picks of a row, into lanes first .. first + topk - 1 (`mine`: whether this is one).
// Returns whether fp32 leaves some open.
template <typename X, int V, bool BY_SCORE>
__device__ __forceinline__ bool pick_row(const RouteParams& p, const float (&x)[V], const float (&bias)[V],
                                         double* lds, int first, bool mine, Lane* out) {
  bool nan = false, open = false;
  uint32_t top = none<uint32_t>();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    nan |= x[j] != x[j];
    if (!p.sigmoid && (BY_SCORE || !p.renorm)) top = max(top, key_of<uint32_t>(x[j] + 0.0f));
  }
  // the largest logit, where scores are relative to it
  const float m = !p.sigmoid && (BY_SCORE || !p.renorm) ? value_of(wave_max(top)) : 0.0f;
  if (!p.sigmoid && !p.renorm) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sum += x[j] > kMasked ? exact_exp_from(x[j], m) : 0.0f;
      __builtin_amdgcn_sched_barrier(0);
    }
    sum = sum_over(sum, kWave);
    out->m = mine ? m : out->m;
    out->sum = mine ? sum : out->sum;
  }
  if constexpr (BY_SCORE) {
    uint32_t key[V];
    nan |= score_keys(p, x, bias, m, key);
    open = pick<V, true>(p, key, reinterpret_cast<uint32_t*>(lds), first, &out->id);
  } else {
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = key_of<uint32_t>(x[j] + 0.0f);  // (both zeros are one)
    pick<V, false>(p, key, reinterpret_cast<uint32_t*>(lds), first, &out->id);
  }
  const bool bad = __ballot(nan) != 0;
  out->nan = mine ? bad : out->nan;
  return open;
}

// The same picks in fp64, into the first lanes.  Few rows come here: an expert at a
// time, the keys in LDS, so that it takes few registers.
template <typename X>
__device__ __forceinline__ Lane pick_again(const RouteParams& p, const X* row, double* lds) {
  const int lane = lane_id();
  bool nan = false;
  auto logit = [&](int e) {
    if constexpr (sizeof(X) == 4)
      return row[e];
    else
      return bf16_to_f32(row[e]);
  };
  uint32_t top = none<uint32_t>();
#pragma unroll 1
  for (int e = lane; e < p.E; e += kWave) top = max(top, key_of<uint32_t>(logit(e) + 0.0f));
  const double m = value_of(wave_max(top));
  double sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < p.E; e += kWave) {
    const float x = logit(e);
    const double s = p.sigmoid ? 1.0 / (1.0 + exp(-double(x))) : exp_from(double(x), m);
    nan |= x != x;
    lds[e] = x > kMasked ? s : none<double>();
    sum += x > kMasked ? s : 0.0;
  }
  sum = p.sigmoid ? 1.0 : sum_over(sum, kWave);
#pragma unroll 1
  for (int e = lane; e < p.E; e += kWave) {
    const double s = lds[e];
    const double key = s / sum + (p.bias ? double(p.bias[e]) : 0.0);
    nan |= s > none<double>() && key != key;
    lds[e] = s > none<double>() ? key_of<double>(key) : s;
  }
  wave_sync();
  if (p.n_group > 1) {
    const int shift = group_lane_shift(p);
    uint64_t kept;
    groups_in_lds(p, lds, shift, &kept);
    wave_sync();
#pragma unroll 1
    for (int e = lane; e < p.E; e += kWave)
      if (!(kept >> (uint32_t(e) * p.inv_size >> 20 << shift) & 1)) lds[e] = none<double>();
    wave_sync();
  }
  Lane out{-1, float(m), float(sum), __ballot(nan) != 0};
  for (int r = 0; r < p.topk; ++r) {
    double best = none<double>();
    uint32_t at = 0;
#pragma unroll 1
    for (int e = lane; e < p.E; e += kWave) {
      const double v = lds[e];
      at = v > best ? uint32_t(e) : at;
      best = v > best ? v : best;
    }
    const double most = wave_max(best);
    if (!(most > none<double>())) break;
    const int e = int(~wave_max(best == most ? ~at : 0u));  // the lowest of equal ones
    out.id = lane == r ? e : out.id;
    if (lane == 0) lds[e] = none<double>();
    wave_sync();
  }
  return out;
}

// The weights of `rows` rows, a pick a lane, 2^each lanes a row; `open` has the rows
// to be done again.
// Renormalised, the common factor cancels, and everything is relative to the
// largest of the row's picks, so that none underflows.
template <typename X>
__device__ __forceinline__ void weigh_rows(const RouteParams& p, int64_t row0, int rows, int each, const Lane& in,
                                           uint64_t open) {
  const int lane = lane_id(), q = lane >> each, r = lane & ((1 << each) - 1);
  const int64_t row = row0 + q;
  const bool have = in.id >= 0;
  float x = kMasked;
  if (have) {
    const X v = (reinterpret_cast<const X*>(p.logits) + row * p.E)[in.id];
    x = sizeof(X) == 4 ? float(v) : bf16_to_f32(uint16_t(v));
  }
  float s = 0.0f;
  if (p.renorm) {
    float ref = x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
      if (o < 1 << each) ref = fmaxf(ref, partner(ref, o));
    if (have) {
      if (!p.sigmoid) {
        s = exact_exp_from(x, ref);
      } else if (x > 0.0f) {
        s = 1.0f / (1.0f + expf(-x));
      } else {
        s = exact_exp_from(x, fminf(ref, 0.0f)) / (1.0f + expf(x));
      }
    }
    const float sum = sum_over(s, 1 << each);
    if (sum > 0.0f) s /= sum;
  } else if (have) {
    if (!p.sigmoid)
      s = exact_exp_from(x, in.m) / in.sum;
    else
      s = x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x) / (1.0f + expf(x));
  }
  s *= p.scale;
  if (in.nan) s = __builtin_nanf("");
  if (r < p.topk && q < rows) {
    p.ids[row * p.topk + r] = r == 0 && (open >> q & 1) ? kOpen : in.id;
    p.weights[row * p.topk + r] = s;
  }
}

// Each wavefront takes p.batch rows in a row, as many as have their picks in its
// lanes at once, then weighs them together, and goes on to others.
template <typename X, int V, bool BY_SCORE>
__global__ void __launch_bounds__(kWaves * kWave) route_kernel(RouteParams p) {
  __shared__ double lds[kWaves][BY_SCORE ? 64 * V : 32 * V];
  const int lane = lane_id(), w = wave_id(), each = p.slot_shift;
  const X* logits = reinterpret_cast<const X*>(p.logits);
  const int64_t step = int64_t(gridDim.x) * kWaves * p.batch;
  const int64_t first = (int64_t(blockIdx.x) * kWaves + w) * p.batch;
  int64_t row0 = first;
  if (row0 >= p.M) return;
  bool any = false;
  float bias[V];
#pragma unroll
  for (int j = 0; j < V; ++j) bias[j] = BY_SCORE && p.bias ? p.bias[min(V * lane + j, p.E - 1)] : 0.0f;
  float x[V], next[V];
  load_row<X, V>(p, logits + row0 * p.E, x);
  for (; row0 < p.M; row0 += step) {
    const int rows = int(std::min<int64_t>(p.batch, p.M - row0));
    Lane out{-1, 0.0f, 1.0f, false};
    uint64_t open = 0;  // rows to be done again
    for (int q = 0; q < rows; ++q) {
      // (behind the last row of all: one that is there)
      const int64_t ahead = q + 1 < rows ? row0 + q + 1 : row0 + step < p.M ? row0 + step : row0;
      load_row<X, V>(p, logits + ahead * p.E, next);
      const bool again = pick_row<X, V, BY_SCORE>(p, x, bias, lds[w], q << each, lane >> each == q, &out);
      if (BY_SCORE && again) open |= uint64_t(1) << q;
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = next[j];
    }
    weigh_rows<X>(p, row0, rows, each, out, open);
    any |= open != 0;
  }
  if (!BY_SCORE || !any) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // another lane wrote the id
  for (row0 = first; row0 < p.M; row0 += step) {
    const int rows = int(std::min<int64_t>(p.batch, p.M - row0));
    uint64_t open = __ballot(lane < rows && p.ids[(row0 + std::min(lane, rows - 1)) * p.topk] == kOpen);
    for (; open; open &= open - 1) {
      const int64_t row = row0 + __builtin_ctzll(open);
      weigh_rows<X>(p, row, 1, each, pick_again(p, logits + row * p.E, lds[w]), 0);
    }
  }
}

template <typename X, int V>
hipError_t route_launch(RouteParams p, hipStream_t st) {
  p.vectors = p.E % V == 0 && reinterpret_cast<uintptr_t>(p.logits) % std::min<size_t>(16, V * sizeof(X)) == 0;
  const int lanes = p.size / V;
  p.group_shift = p.size % V == 0 && (lanes & (lanes - 1)) == 0 ? __builtin_ctz(lanes) : -1;
  // Rows whose picks a wavefront has room for, and how many of them it takes: with
  // few rows one, for the sake of the others.
  p.slot_shift = 0;
  while (1 << p.slot_shift < p.topk) ++p.slot_shift;
  const int64_t waves = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * 16;
  p.batch = int32_t(std::min<int64_t>(kWave >> p.slot_shift, std::max<int64_t>(1, p.M / waves)));
  const int64_t want = (p.M + int64_t(p.batch) * kWaves - 1) / (int64_t(p.batch) * kWaves);
  const dim3 grid(unsigned(std::min(want, 8 * waves))), block(kWaves * kWave);
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
