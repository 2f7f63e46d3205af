// C ABI of the bf16 base side: argument checks and dispatch.  As in api.hip, every
// check runs on the host before any HIP call.
#include <cmath>
#include <stdint.h>

#include "../../include/moe_lora.h"
#include "base.h"
#include "internal.h"

using namespace mlr;

namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxK = int64_t(1) << 21;      // a tile of 256 rows stays below 2 GiB
constexpr int64_t kMaxElements = (int64_t(1) << 30) - 1;  // 2 GiB of bf16
constexpr int64_t kStageK = 64;

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool flag(int32_t v) { return v == 0 || v == 1; }

// Sizes and activation of a product.  On success fills them in.
int check_product(int64_t K, int64_t Ns, int64_t S, int32_t act, ProductParams* p) {
  if (K < 8 || (K & 7) || Ns < 8 || (Ns & 7) || S < 1) return MOE_LORA_ERR_INVALID;
  if (act < kActNone || act > kActSwigluClamp || (act_gated(act) && S != 2)) return MOE_LORA_ERR_INVALID;
  if (K > kMaxK || Ns > kMaxElements || S * Ns > kMaxElements / K) return MOE_LORA_ERR_UNSUPPORTED;
  p->K = int32_t(K);
  p->N = int32_t(S * Ns);
  p->No = int32_t(act_gated(act) ? Ns : S * Ns);
  p->KB = int32_t((K + kStageK - 1) / kStageK);
  p->act = act;
  p->gated = act_gated(act);
  return MOE_LORA_OK;
}

// Workgroups of a launch: 16 rows x 16 columns is the smallest tile.
bool grid_fits(int64_t blocks, int64_t N) { return blocks <= kInt32Max / ((N + 15) / 16); }

// All sizes of a dense product.
int check_dense(int64_t M, int64_t K, int64_t Ns, int64_t S, int32_t act, ProductParams* p) {
  if (M < 0) return MOE_LORA_ERR_INVALID;
  const int rc = check_product(K, Ns, S, act, p);
  if (rc != MOE_LORA_OK) return rc;
  if (M > kInt32Max || !grid_fits((M + 15) / 16, p->N)) return MOE_LORA_ERR_UNSUPPORTED;
  p->rows = p->M = M;
  return MOE_LORA_OK;
}

// And of a grouped one.
int check_grouped(int64_t M, int32_t topk, int64_t K, int64_t Ns, int64_t S, int32_t E, int32_t block_m,
                  int32_t x_per_pair, int32_t act, ProductParams* p) {
  // the align step's own limits on M, topk, E and block_m, for one slot
  const int64_t cap = moe_lora_align_capacity(M, topk, E, block_m);
  if (cap < 0) return int(cap);
  const int rc = check_product(K, Ns, S, act, p);
  if (rc != MOE_LORA_OK) return rc;
  if (!flag(x_per_pair)) return MOE_LORA_ERR_INVALID;
  const int64_t numel = M * topk, rows = x_per_pair ? numel : M;
  const int64_t blocks = max_total_blocks(numel, E, block_m);
  if (rows > kMaxElements / K || !grid_fits(blocks * (block_m / 16), p->N)) return MOE_LORA_ERR_UNSUPPORTED;
  p->rows = rows;
  p->M = M;
  p->numel = int32_t(numel);
  p->topk = topk;
  p->E = E;
  p->block_m = block_m;
  p->x_per_pair = x_per_pair;
  p->blocks = int32_t(blocks);
  return MOE_LORA_OK;
}

}  // namespace

extern "C" {

int moe_lora_route(const void* logits, int32_t logits_bf16, const float* bias, int64_t M, int32_t E,
                   int32_t topk, int32_t scoring, int32_t n_group, int32_t topk_group,
                   int32_t group_top, int32_t renormalize, float scale, int32_t* topk_ids,
                   float* topk_weights, void* stream) {
  if (M < 0 || E < 1 || topk < 1 || n_group < 1 || topk_group < 1 || group_top < 1 || group_top > 2)
    return MOE_LORA_ERR_INVALID;
  if (!flag(logits_bf16) || !flag(renormalize) || !flag(scoring) || !std::isfinite(scale))
    return MOE_LORA_ERR_INVALID;
  if (E % n_group || topk_group > n_group || group_top > E / n_group || (n_group == 1 && group_top == 2))
    return MOE_LORA_ERR_INVALID;
  if (int64_t(topk) > int64_t(topk_group) * (E / n_group)) return MOE_LORA_ERR_INVALID;
  if (E > kMaxRouteExperts || topk > kMaxRouteTopk || n_group > 64 || M > kInt32Max / topk)
    return MOE_LORA_ERR_UNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!logits || !topk_ids || !topk_weights) return MOE_LORA_ERR_INVALID;
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_weights, 4))
    return MOE_LORA_ERR_INVALID;
  RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.ids = topk_ids;
  p.weights = topk_weights;
  p.M = M;
  p.E = E;
  p.topk = topk;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.group_top = group_top;
  p.size = E / n_group;
  p.inv_size = uint32_t(((1 << 20) + p.size - 1) / p.size);
  p.logits_bf16 = logits_bf16;
  p.sigmoid = scoring;
  p.renorm = renormalize;
  p.scale = scale;
  return launch_route(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                         : MOE_LORA_ERR_HIP;
}

int moe_lora_gemm(const uint16_t* x, const uint16_t* w, const uint16_t* bias, const uint16_t* delta,
                  const uint16_t* residual, int64_t M, int32_t K, int32_t Ns, int32_t S,
                  int32_t activation, int32_t y_fp32, void* y, void* stream) {
  ProductParams p{};
  if (!flag(y_fp32)) return MOE_LORA_ERR_INVALID;
  const int rc = check_dense(M, K, Ns, S, activation, &p);
  if (rc != MOE_LORA_OK) return rc;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !w || !y) return MOE_LORA_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(delta, 16) ||
      !aligned(residual, 16) || !aligned(y, 16))
    return MOE_LORA_ERR_INVALID;
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.delta = delta;
  p.residual = residual;
  p.y = y;
  p.out32 = y_fp32;
  return launch_gemm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                        : MOE_LORA_ERR_HIP;
}

int moe_lora_moe_gemm(const uint16_t* x, int32_t x_per_pair, const uint16_t* w, const uint16_t* bias,
                      const uint16_t* delta, const int32_t* sorted_token_ids,
                      const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                      const float* topk_weights, int32_t mul_routed_weight, int64_t M, int32_t topk,
                      int32_t K, int32_t Ns, int32_t S, int32_t E, int32_t block_m,
                      int32_t activation, uint16_t* y, void* stream) {
  ProductParams p{};
  if (!flag(mul_routed_weight)) return MOE_LORA_ERR_INVALID;
  const int rc = check_grouped(M, topk, K, Ns, S, E, block_m, x_per_pair, activation, &p);
  if (rc != MOE_LORA_OK) return rc;
  if (p.numel == 0) return MOE_LORA_OK;
  if (!x || !w || !sorted_token_ids || !expert_ids || !num_tokens_post_padded || !y ||
      (mul_routed_weight && !topk_weights))
    return MOE_LORA_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(delta, 16) || !aligned(y, 16))
    return MOE_LORA_ERR_INVALID;
  p.x = x;
  p.w = w;
  p.bias = bias;
  p.delta = delta;
  p.y = y;
  p.sorted = sorted_token_ids;
  p.eids = expert_ids;
  p.ntpp = num_tokens_post_padded;
  p.wt = mul_routed_weight ? topk_weights : nullptr;
  return launch_moe_gemm(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                            : MOE_LORA_ERR_HIP;
}

const char* moe_lora_gemm_kernel_name(int64_t M, int32_t K, int32_t Ns, int32_t S, int32_t activation) {
  ProductParams p{};
  return check_dense(M, K, Ns, S, activation, &p) == MOE_LORA_OK && M > 0 ? gemm_name(p) : nullptr;
}

const char* moe_lora_moe_gemm_kernel_name(int64_t M, int32_t topk, int32_t K, int32_t Ns, int32_t S, int32_t E,
                                          int32_t block_m, int32_t x_per_pair, int32_t activation) {
  ProductParams p{};
  return check_grouped(M, topk, K, Ns, S, E, block_m, x_per_pair, activation, &p) == MOE_LORA_OK && M > 0
             ? moe_gemm_name(p)
             : nullptr;
}

int moe_lora_combine(const uint16_t* y, const float* topk_weights, const int32_t* topk_ids, int32_t E,
                     const uint16_t* residual, int64_t M, int32_t topk, int32_t N, uint16_t* out,
                     void* stream) {
  if (M < 0 || topk < 1 || N < 8 || (N & 7) || (topk_ids && E < 1)) return MOE_LORA_ERR_INVALID;
  // (a launch has fewer than 2^32 threads, each eight columns)
  if (M > kInt32Max / topk || M * N >= int64_t(1) << 34) return MOE_LORA_ERR_UNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!y || !out) return MOE_LORA_ERR_INVALID;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(topk_weights, 4) ||
      !aligned(topk_ids, 4))
    return MOE_LORA_ERR_INVALID;
  const CombineParams p{y, topk_weights, topk_ids, residual, out, M, topk, N, E};
  return launch_combine(p, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_LORA_OK
                                                                           : MOE_LORA_ERR_HIP;
}

}  // extern "C"
