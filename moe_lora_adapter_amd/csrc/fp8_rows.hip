// Producers of 8-bit rows: RMS norm with the residual's addition, and
// silu(gate) * up.  Both are bound by memory: every value is read once, held
// in registers, and written once in each of the forms a layer reads (the
// stored residual, bf16 rows for the LoRA side, e4m3 rows for the base
// product).
#include <algorithm>

#include "common.h"
#include "fp8.h"
#include "internal.h"

namespace mlr {
namespace {

// Largest of v over the 16 consecutive lanes of a DPP row (one 128-column
// block at 8 columns a lane), in every one of them.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, butterfly_partner(v, 8));
  v = fmaxf(v, butterfly_partner(v, 4));
  v = fmaxf(v, butterfly_partner(v, 2));
  v = fmaxf(v, butterfly_partner(v, 1));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Stores of outputs are non-temporal: the next kernel reads them from memory
// side caches whatever L2 kept, and the inputs keep their place in L2 (norm of
// 4096 x 2880: 23.0 us with the default policy, 17.3 so; of 16384 x 4096: 105.0
// and 101.6.  Non-temporal loads as well: 20.3 and 99.4, not taken).
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store16(uint16_t* p, const uint4& v) {
  const u32x4_t x = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(x, reinterpret_cast<u32x4_t*>(p));
}
__device__ __forceinline__ void store8(uint8_t* p, const uint2& v) {
  const u32x2_t x = {v.x, v.y};
  __builtin_nontemporal_store(x, reinterpret_cast<u32x2_t*>(p));
}

// Largest magnitude of 8 values; NaN entries are passed over (fmaxf), so one
// NaN leaves its block's other values as they are.
__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
  return a;
}

// Scale of a block from its largest magnitude: the division is the IEEE one.
__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax, kMinAmax) / kE4m3Max; }

// 8 values over the scale, each quotient rounded to fp32 as a division does and
// then to e4m3, nearest even.  Values and scale come from few bits, so quotients
// often lie halfway between two e4m3 values; times the rounded reciprocal alone
// some of them would go the other way.  One step on the remainder gives the
// division's quotient (P. Markstein, IBM J. Res. Dev. 34, 1990; no difference in
// 2e7 sampled quotients above 2^-11, smaller ones round to 0 either way).  8192 x
// 1024 without residual: 9.1 us, with the compiler's divisions 10.6, with the
// reciprocal alone 9.0; 16384 x 4096 101.4 with each of them.
// |v| / scale is at most 448 (1 + 2^-23), which rounds to 448: the conversion never
// overflows on finite values.  In an infinite block the reciprocal is 0: finite
// values become 0 and infinities NaN.
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float s) {
  const float inv = 1.0f / s, finite = fminf(s, 0x1.fffffep127f);  // (0 times infinity is NaN)
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = f[i] * inv;
    q[i] = fmaf(fmaf(-q[i], finite, f[i]), inv, q[i]);
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2(uint32_t(lo), uint32_t(hi));
}

// One workgroup of T threads a row; thread t holds the 8-column chunks t,
// t + T, ... (CH of them).  16384 x 4096 with the residual (9 bytes a value): 101
// us, 6.0 TB/s, where a copy runs at 5.1; 16 x 2880 in a graph 2.5 us, of which
// an empty kernel is 1.8.
template <int T, int CH, bool RES>
__global__ void __launch_bounds__(T) rms_norm_fp8_kernel(NormParams p) {
  __shared__ float part[T / kWave];
  const int64_t row = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  if (row >= p.M) return;
  const int nc = p.H / 8;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.H);
  float v[CH][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * T;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (c < nc) {
      unpack8(x[c], v[i]);
      if constexpr (RES) {
        float r[8];
        unpack8(reinterpret_cast<const uint4*>(p.residual + row * p.H)[c], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        // the norm is of the sum as it is stored
        const uint4 h = pack8(v[i]);
        store16(p.residual_out + row * p.H + 8 * c, h);
        unpack8(h, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += butterfly_partner(sum, o);
  if constexpr (T > kWave) {
    if (lane_id() == 0) part[wave_id()] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < T / kWave; ++i) sum += part[i];
  }
  const float rstd = 1.0f / sqrtf(sum / float(p.H) + p.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * T;
    float amax = 0.0f;
    if (c < nc) {
      float w[8];
      unpack8(reinterpret_cast<const uint4*>(p.weight)[c], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
      amax = amax8(v[i]);
    }
    const float s = block_scale(row16_max(amax));
    if (c < nc) {
      if (p.y) store16(p.y + row * p.H + 8 * c, pack8(v[i]));
      store8(p.q + row * p.H + 8 * c, quantise8(v[i], s));
      if ((c & 15) == 0) p.scales[int64_t(c >> 4) * p.M + row] = s;
    }
  }
}

// 16 lanes a (row, block of 128 columns); a workgroup takes the same block of 16
// consecutive rows, whose scales are neighbours.  65536 x 768 (7 bytes a value): 62
// us, 5.7 TB/s; 64 workgroups a CU, 16 of them took 66 us.  The exponential is the
// hardware's power of two of a rounded argument: off by some |g| 2^-24 of its
// value, 2^-17 at most where it counts, against bf16's 2^-8 and e4m3's 2^-4 at the
// output (the library's exact one: 4096 x 2880 18.7 us, so 17.6).
constexpr int kTS = 256, kRows = kTS / 16;
__global__ void __launch_bounds__(kTS) silu_mul_fp8_kernel(SiluParams p, int32_t nb, int64_t items) {
  const int sub = threadIdx.x & 15;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / nb * kRows + threadIdx.x / 16;
    const int j = int(it % nb);
    const int col = j * kScaleBlock + sub * 8;
    const bool in = row < p.P && col < p.I;
    float v[8];
    float amax = 0.0f;
    if (in) {
      const uint16_t* g = p.y + row * 2 * p.I + col;
      float u[8];
      unpack8(*reinterpret_cast<const uint4*>(g), v);
      unpack8(*reinterpret_cast<const uint4*>(g + p.I), u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + __expf(-v[i])) * u[i];
      amax = amax8(v);
    }
    const float s = block_scale(row16_max(amax));
    if (in) {
      if (p.h) store16(p.h + row * p.I + col, pack8(v));
      store8(p.q + row * p.I + col, quantise8(v, s));
      if (sub == 0) p.scales[int64_t(j) * p.P + row] = s;
    }
  }
}

template <int T, int CH>
hipError_t norm_of(const NormParams& p, hipStream_t st) {
  // a launch has fewer than 2^32 threads along one axis
  const int64_t most = (int64_t(1) << 32) / T - 1, y = (p.M + most - 1) / most;
  const dim3 grid(unsigned((p.M + y - 1) / y), unsigned(y));
  if (p.residual)
    hipLaunchKernelGGL((rms_norm_fp8_kernel<T, CH, true>), grid, dim3(T), 0, st, p);
  else
    hipLaunchKernelGGL((rms_norm_fp8_kernel<T, CH, false>), grid, dim3(T), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm_fp8(const NormParams& p, hipStream_t st) {
  // One 8-column chunk a thread where a workgroup can hold the row so (16 x 2880:
  // 384 and 512 threads 2.5 us, 256 with two chunks 2.9; 16384 x 4096: 512 threads
  // 101.6 us, 256 with two 104.4); narrow rows in one wavefront, without a
  // barrier (8192 x 1024: 12.4 us, 256 threads 13.2).
  const int nc = p.H / 8;
  if (nc <= 128) return norm_of<64, 2>(p, st);
  if (nc <= 256) return norm_of<256, 1>(p, st);
  if (nc <= 512) return norm_of<512, 1>(p, st);
  if (nc <= 2048) return norm_of<512, 4>(p, st);
  return norm_of<1024, 8>(p, st);
}

hipError_t launch_silu_mul_fp8(const SiluParams& p, hipStream_t st) {
  const int32_t nb = int32_t(scale_blocks(p.I));
  const int64_t items = (p.P + kRows - 1) / kRows * nb;
  const int64_t cap = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * 64;
  hipLaunchKernelGGL(silu_mul_fp8_kernel, dim3(unsigned(std::min(items, cap))), dim3(kTS), 0, st, p, nb,
                     items);
  return hipGetLastError();
}

}  // namespace mlr
