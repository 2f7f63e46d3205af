// The 8-bit rows shared by the kernels of the base side: OCP e4m3 values with
// one fp32 scale per (row, block of 128 columns), the scales block-major.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlr {

constexpr int kScaleBlock = 128;        // columns that share a scale
constexpr float kE4m3Max = 448.0f;      // largest finite e4m3 value
constexpr float kMinAmax = 0x1p-40f;    // blocks below this are scaled as if at it

inline int64_t scale_blocks(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// ---------------------------------------------------------------- row producers
struct NormParams {
  const uint16_t* x;         // [M, H]
  const uint16_t* residual;  // [M, H] or null
  const uint16_t* weight;    // [H]
  uint16_t* residual_out;    // [M, H]; null exactly when residual is
  uint16_t* y;               // [M, H] or null
  uint8_t* q;                // [M, H]
  float* scales;             // [ceil(H / 128), M]
  int64_t M;
  int32_t H;
  float eps;
};

struct SiluParams {
  const uint16_t* y;  // [P, 2 I]
  uint16_t* h;        // [P, I] or null
  uint8_t* q;         // [P, I]
  float* scales;      // [ceil(I / 128), P]
  int64_t P;
  int32_t I;
};

constexpr int32_t kMaxNormWidth = 65536;

hipError_t launch_rms_norm_fp8(const NormParams& p, hipStream_t st);
hipError_t launch_silu_mul_fp8(const SiluParams& p, hipStream_t st);

// ---------------------------------------------------------------- products
struct GemmParams {
  const uint8_t* x;       // [rows, K]
  const float* xs;        // [KB, rows]
  const uint8_t* w;       // [E, S, Ns, K]
  const float* ws;        // [E, S, NB, KB]
  uint16_t* y;            // [M, S Ns], or [M topk, S Ns] when grouped
  int64_t rows;           // rows of x
  int64_t M;              // dense: rows; grouped: tokens
  int32_t K, Ns, S, KB, NB;
  // grouped (null / unused when dense)
  const int32_t* sorted;  // [cap]
  const int32_t* eids;    // [cap / block_m]
  const int32_t* ntpp;    // [1]
  const float* wt;        // [M topk]; null: not applied
  int32_t numel, topk, E, block_m, x_per_pair;
  int32_t blocks;         // align blocks: at most this many, of this launch
  int32_t block0;         // and its first
};

hipError_t launch_fp8_gemm(GemmParams p, hipStream_t st);      // dense
hipError_t launch_fp8_moe_gemm(GemmParams p, hipStream_t st);  // grouped

}  // namespace mlr
