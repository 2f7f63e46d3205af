// C ABI of the 8-bit base side: argument checks and dispatch.  As in api.hip,
// every check runs on the host before any HIP call.
#include <stdint.h>

#include "../../include/moe_lora.h"
#include "fp8.h"
#include "internal.h"

using namespace mlr;

namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxK = int64_t(1) << 22;  // a tile of 256 rows stays below 2 GiB

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes of a product that do not depend on its rows.  On success fills the
// scale blocks.
int check_weights(int64_t K, int64_t Ns, int64_t S, GemmParams* p) {
  if (K < 16 || (K & 15) || Ns < 8 || (Ns & 7) || S < 1) return MOE_LORA_ERR_INVALID;
  if (K > kMaxK || Ns * K > kInt32Max || S * Ns > kInt32Max) return MOE_LORA_ERR_UNSUPPORTED;
  p->K = int32_t(K);
  p->Ns = int32_t(Ns);
  p->S = int32_t(S);
  p->KB = int32_t(scale_blocks(K));
  p->NB = int32_t(scale_blocks(Ns));
  return MOE_LORA_OK;
}

// Workgroups of a launch: 16 rows x 16 columns is the smallest tile.
bool grid_fits(int64_t blocks, int64_t S, int64_t Ns) {
  const int64_t tiles = S * ((Ns + 15) / 16);
  return blocks <= kInt32Max / tiles;
}

}  // namespace

extern "C" {

int moe_lora_rms_norm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                          int64_t M, int32_t H, float eps, uint16_t* residual_out, uint16_t* y,
                          uint8_t* q, float* scales, void* stream) {
  if (M < 0 || H < 8 || (H & 7) || !(eps >= 0.0f)) return MOE_LORA_ERR_INVALID;
  if (H > kMaxNormWidth || M > kInt32Max) return MOE_LORA_ERR_UNSUPPORTED;
  if ((residual == nullptr) != (residual_out == nullptr)) return MOE_LORA_ERR_INVALID;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !weight || !q || !scales) return MOE_LORA_ERR_INVALID;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
      !aligned16(y) || !aligned16(q) || !aligned4(scales))
    return MOE_LORA_ERR_INVALID;
  const NormParams p{x, residual, weight, residual_out, y, q, scales, M, H, eps};
  return launch_rms_norm_fp8(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                                : MOE_LORA_ERR_HIP;
}

int moe_lora_silu_mul_fp8(const uint16_t* y, int64_t P, int32_t I, uint16_t* h, uint8_t* q,
                          float* scales, void* stream) {
  if (P < 0 || I < 8 || (I & 7)) return MOE_LORA_ERR_INVALID;
  if (P > kInt32Max || I > kInt32Max / 2) return MOE_LORA_ERR_UNSUPPORTED;
  if (P == 0) return MOE_LORA_OK;
  if (!y || !q || !scales) return MOE_LORA_ERR_INVALID;
  if (!aligned16(y) || !aligned16(h) || !aligned16(q) || !aligned4(scales))
    return MOE_LORA_ERR_INVALID;
  const SiluParams p{y, h, q, scales, P, I};
  return launch_silu_mul_fp8(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                                : MOE_LORA_ERR_HIP;
}

int moe_lora_fp8_gemm(const uint8_t* x, const float* x_scales, const uint8_t* w,
                      const float* w_scales, int64_t M, int32_t K, int32_t Ns, int32_t S,
                      uint16_t* y, void* stream) {
  GemmParams p{};
  if (M < 0) return MOE_LORA_ERR_INVALID;
  const int rc = check_weights(K, Ns, S, &p);
  if (rc != MOE_LORA_OK) return rc;
  if (M > kInt32Max || M * p.KB > kInt32Max / 4 || !grid_fits((M + 15) / 16, S, Ns))
    return MOE_LORA_ERR_UNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !x_scales || !w || !w_scales || !y) return MOE_LORA_ERR_INVALID;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned4(x_scales) || !aligned4(w_scales))
    return MOE_LORA_ERR_INVALID;
  p.x = x;
  p.xs = x_scales;
  p.w = w;
  p.ws = w_scales;
  p.y = y;
  p.rows = p.M = M;
  return launch_fp8_gemm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                            : MOE_LORA_ERR_HIP;
}

int moe_lora_fp8_moe_gemm(const uint8_t* x, const float* x_scales, int32_t x_per_pair,
                          const uint8_t* w, const float* w_scales,
                          const int32_t* sorted_token_ids, const int32_t* expert_ids,
                          const int32_t* num_tokens_post_padded, const float* topk_weights,
                          int32_t mul_routed_weight, int64_t M, int32_t topk, int32_t K,
                          int32_t Ns, int32_t S, int32_t E, int32_t block_m, uint16_t* y,
                          void* stream) {
  GemmParams p{};
  // the align step's own limits on M, topk, E and block_m, for one slot
  const int64_t cap = moe_lora_align_capacity(M, topk, E, block_m);
  if (cap < 0) return int(cap);
  const int rc = check_weights(K, Ns, S, &p);
  if (rc != MOE_LORA_OK) return rc;
  if ((x_per_pair != 0 && x_per_pair != 1) || (mul_routed_weight != 0 && mul_routed_weight != 1))
    return MOE_LORA_ERR_INVALID;
  const int64_t numel = M * topk, rows = x_per_pair ? numel : M;
  const int64_t blocks = max_total_blocks(numel, E, block_m);
  if (rows * K > kInt32Max || rows * p.KB > kInt32Max / 4 || !grid_fits(blocks * (block_m / 16), S, Ns))
    return MOE_LORA_ERR_UNSUPPORTED;
  if (numel == 0) return MOE_LORA_OK;
  if (!x || !x_scales || !w || !w_scales || !sorted_token_ids || !expert_ids ||
      !num_tokens_post_padded || !y || (mul_routed_weight && !topk_weights))
    return MOE_LORA_ERR_INVALID;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned4(x_scales) || !aligned4(w_scales))
    return MOE_LORA_ERR_INVALID;
  p.x = x;
  p.xs = x_scales;
  p.w = w;
  p.ws = w_scales;
  p.y = y;
  p.rows = rows;
  p.M = M;
  p.sorted = sorted_token_ids;
  p.eids = expert_ids;
  p.ntpp = num_tokens_post_padded;
  p.wt = mul_routed_weight ? topk_weights : nullptr;
  p.numel = int32_t(numel);
  p.topk = topk;
  p.E = E;
  p.block_m = block_m;
  p.x_per_pair = x_per_pair;
  p.blocks = int32_t(blocks);
  return launch_fp8_moe_gemm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                                : MOE_LORA_ERR_HIP;
}

}  // extern "C"
