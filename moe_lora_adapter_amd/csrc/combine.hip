// out[m] = bf16( sum_k w[m, k] y[m, k] + residual[m] ): a token's expert outputs
// joined, in ascending k, in fp32, rounded once.  A pair whose expert is not here
// is not read (its row of y was never written).
//
// Memory-bound: each value is read once, 16 bytes a lane, the loads of kAtOnce
// pairs in flight before the first is used.  8192 tokens x 8 x 2048 columns 60 us,
// 5.4 TB/s (a copy reaches 5.2); 16 x 4 x 2880 2.5 us in a graph, launch and one
// round trip.
#include <algorithm>

#include "base.h"
#include "common.h"
#include "internal.h"

namespace mlr {
namespace {

constexpr int kTC = 256;
constexpr int kAtOnce = 4;

template <bool WEIGHTS, bool IDS>
__global__ void __launch_bounds__(kTC) combine_kernel(CombineParams p, int64_t chunks) {
  const int64_t c = int64_t(blockIdx.x) * kTC + threadIdx.x;
  if (c >= chunks) return;
  const int per = p.N / 8;
  const int64_t m = c / per;
  const int col = int(c - m * per) * 8;
  const uint16_t* y = p.y + m * p.topk * p.N + col;
  float s[8];
  if (p.residual) {
    const uint4 r = *reinterpret_cast<const uint4*>(p.residual + m * p.N + col);
    const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) s[2 * j] = bf16_lo(q[j]), s[2 * j + 1] = bf16_hi(q[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.0f;
  }
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int k0 = 0; k0 < p.topk; k0 += kAtOnce) {
    uint4 v[kAtOnce];
    float w[kAtOnce];
    bool in[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int k = k0 + i;
      in[i] = k < p.topk;
      w[i] = 1.0f;
      v[i] = make_uint4(0, 0, 0, 0);
      if (IDS && in[i]) in[i] = uint32_t(p.ids[m * p.topk + k]) < uint32_t(p.E);
      if (WEIGHTS && in[i]) w[i] = p.wt[m * p.topk + k];
      if (in[i]) v[i] = *reinterpret_cast<const uint4*>(y + int64_t(k) * p.N);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (!in[i]) continue;
      const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[2 * j] = fmaf(w[i], bf16_lo(q[j]), acc[2 * j]);
        acc[2 * j + 1] = fmaf(w[i], bf16_hi(q[j]), acc[2 * j + 1]);
      }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(acc[2 * j] + s[2 * j], acc[2 * j + 1] + s[2 * j + 1]);
  *reinterpret_cast<uint4*>(p.out + m * p.N + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool WEIGHTS, bool IDS>
hipError_t combine_launch(const CombineParams& p, hipStream_t st) {
  const int64_t chunks = p.M * (p.N / 8);
  hipLaunchKernelGGL((combine_kernel<WEIGHTS, IDS>), dim3(unsigned((chunks + kTC - 1) / kTC)), dim3(kTC), 0, st,
                     p, chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine(const CombineParams& p, hipStream_t st) {
  if (p.wt) return p.ids ? combine_launch<true, true>(p, st) : combine_launch<true, false>(p, st);
  return p.ids ? combine_launch<false, true>(p, st) : combine_launch<false, false>(p, st);
}

}  // namespace mlr
