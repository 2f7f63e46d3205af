// Parameters of the bf16 base side: routing, products with an epilogue, combine.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mlr {

// ---------------------------------------------------------------- routing
constexpr int32_t kMaxRouteTopk = 64;     // a pick each lane
constexpr int32_t kMaxRouteExperts = 1024;

struct RouteParams {
  const void* logits;  // [M, E], fp32 or bf16
  const float* bias;   // [E] or null
  int32_t* ids;        // [M, topk]
  float* weights;      // [M, topk]
  int64_t M;
  int32_t E, topk;
  int32_t n_group, topk_group, group_top;
  int32_t size;        // experts of a group
  uint32_t inv_size;   // e / size = e * inv_size >> 20, e < 1024
  int32_t group_shift; // a group is the experts of 2^group_shift lanes; -1: not whole lanes
  int32_t vectors;     // a lane's logits may be loaded together
  int32_t slot_shift, batch; // a row's picks take 2^slot_shift lanes; rows a wavefront takes at once
  int32_t logits_bf16, sigmoid, renorm;
  float scale;
};

hipError_t launch_route(const RouteParams& p, hipStream_t st);

// ---------------------------------------------------------------- products
enum Activation { kActNone = 0, kActSilu = 1, kActGeluTanh = 2, kActSiluMul = 3, kActSwigluClamp = 4 };
inline bool act_gated(int32_t act) { return act == kActSiluMul || act == kActSwigluClamp; }

struct ProductParams {
  const uint16_t* x;         // [rows, K]
  const uint16_t* w;         // [E, N, K]
  const uint16_t* bias;      // [E, N] or null
  const uint16_t* delta;     // [M, N], or [M topk, N] when grouped; or null
  const uint16_t* residual;  // [M, No] or null (dense)
  void* y;                   // [M, No] or [M topk, No], bf16 or fp32
  int64_t rows;              // rows of x
  int64_t M;                 // dense: rows; grouped: tokens
  int32_t K, N, No;          // No = N, or N / 2 with a gated activation
  int32_t KB;                // blocks of 64 of K
  int32_t act, gated, out32;
  // grouped (null / unused when dense)
  const int32_t* sorted;     // [cap]
  const int32_t* eids;       // [cap / block_m]
  const int32_t* ntpp;       // [1]
  const float* wt;           // [M topk]; null: not applied
  int32_t numel, topk, E, block_m, x_per_pair;
  int32_t blocks;            // align blocks: at most this many, of this launch
  int32_t block0;            // and its first
};

hipError_t launch_gemm(ProductParams p, hipStream_t st);      // dense
hipError_t launch_moe_gemm(ProductParams p, hipStream_t st);  // grouped
// The kernels they launch: name and tile.
const char* gemm_name(const ProductParams& p);
const char* moe_gemm_name(const ProductParams& p);

// ---------------------------------------------------------------- combine
struct CombineParams {
  const uint16_t* y;         // [M, topk, N]
  const float* wt;           // [M, topk] or null
  const int32_t* ids;        // [M, topk] or null
  const uint16_t* residual;  // [M, N] or null
  uint16_t* out;             // [M, N]
  int64_t M;
  int32_t topk, N, E;
};

hipError_t launch_combine(const CombineParams& p, hipStream_t st);

}  // namespace mlr
