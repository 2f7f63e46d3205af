// e4m3 x e4m3 products with a scale per (row of X, 128 of K) and per
// (128 columns, 128 of K) of W, dense or over the routed pairs of an expert's
// blocks:
//   Y[m, n] = bf16( sum_j xs[j, m] ws[n / 128, j] sum_{k in block j} xq[m, k] wq[n, k] )
//
// One v_mfma_f32_16x16x128_f8f6f4 covers exactly one scale block of K, so the
// sums inside a block stay in the matrix core and each of its fp32 results
// costs one multiply-add by the block's combined scale.  W is the instruction's
// first operand and X the second: a lane then holds one row of X (lane % 16)
// and four consecutive columns of Y, the row's scale is one value per lane and
// the column block's is wave-uniform.  Both operands give lane group g = lane /
// 16 the 16-byte chunks g and g + 4 of a row's 128 bytes; any assignment of k
// to lanes serves as long as both operands use the same one.
#include <algorithm>

#include "common.h"
#include "dma.h"
#include "fp8.h"
#include "internal.h"

namespace mlr {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma_e4m3(const i32x8_t& w, const i32x8_t& x) {
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8_t join(const uint4& a, const uint4& b) {
  return i32x8_t{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
}

// The sum of two byte offsets, past every range when either is: both are below
// 2 GiB or kOob, and 2 kOob wraps to 0, so the sum saturates instead.
__device__ __forceinline__ uint32_t at(uint32_t row, uint32_t k) {
  return row == kOob || k == kOob ? kOob : row + k;
}

// Where a block's rows come from and go to.
struct RowMap {
  int64_t x_row;  // row of X, or -1
  int64_t y_row;  // row of Y, or -1
};
template <bool GROUPED>
__device__ __forceinline__ RowMap row_of(const GemmParams& p, int64_t first, int i) {
  if constexpr (GROUPED) {
    const uint32_t pair = i < p.block_m ? uint32_t(p.sorted[first + i]) : uint32_t(p.numel);
    if (pair >= uint32_t(p.numel)) return {-1, -1};
    return {int64_t(p.x_per_pair ? pair : pair / uint32_t(p.topk)), int64_t(pair)};
  } else {
    const int64_t r = first + i;
    return r < p.M ? RowMap{r, r} : RowMap{-1, -1};
  }
}

// ---------------------------------------------------------------- few rows
// One workgroup computes 16 MT rows x 16 NT columns: its KW wavefronts take
// the K blocks w, w + KW, ... straight from memory (together they read KW x 128
// consecutive bytes of each row of W) and add their sums in LDS, in order.
template <int MT, int NT, int KW, bool GROUPED>
__global__ void __launch_bounds__(KW * kWave) fp8_gemm_rows_kernel(GemmParams p, int ntiles) {
  __shared__ f32x4_t red[KW][MT * NT][kWave];
  const int tile = blockIdx.x % (p.S * ntiles);
  const int blk = blockIdx.x / (p.S * ntiles);
  int64_t e = 0;
  if constexpr (GROUPED) {
    if (int64_t(blk) * p.block_m >= p.ntpp[0]) return;
    e = p.eids[blk];
    if (e < 0 || e >= p.E) return;
  }
  const int slice = tile / ntiles, n0 = (tile % ntiles) * 16 * NT;
  const int64_t first = GROUPED ? int64_t(blk) * p.block_m : int64_t(blk) * 16 * MT;
  const int lane = lane_id(), w = wave_id(), a = lane & 15, g = lane >> 4;

  const uint8_t* wbase = p.w + (e * p.S + slice) * p.Ns * int64_t(p.K);
  const auto wr = make_rsrc(wbase, uint32_t(p.Ns) * uint32_t(p.K));
  const float* wscale = p.ws + ((e * p.S + slice) * p.NB + n0 / kScaleBlock) * p.KB;
  uint32_t woff[NT];
#pragma unroll
  for (int f = 0; f < NT; ++f) {
    const int n = n0 + 16 * f + a;
    woff[f] = n < p.Ns ? uint32_t(n) * uint32_t(p.K) + 16 * g : kOob;
  }
  // rows of X: dense tiles are addressed from their first row, grouped ones
  // from row 0 (X is below 2 GiB there)
  const int64_t x0 = GROUPED ? 0 : first;
  const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, 16 * MT);
  const auto xr = make_rsrc(p.x + x0 * p.K, uint32_t(xrows * p.K));
  uint32_t xoff[MT];
  int64_t srow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const RowMap r = row_of<GROUPED>(p, first, 16 * i + a);
    xoff[i] = r.x_row >= 0 ? uint32_t((r.x_row - x0) * p.K) + 16 * g : kOob;
    srow[i] = r.x_row;
  }

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int f = 0; f < NT; ++f) acc[i][f] = f32x4_t{0, 0, 0, 0};

  for (int kb = w; kb < p.KB; kb += KW) {
    const uint32_t k = uint32_t(kb) * kScaleBlock;
    const uint32_t lo = k + 16 * g < uint32_t(p.K) ? k : kOob;
    const uint32_t hi = k + 64 + 16 * g < uint32_t(p.K) ? k + 64 : kOob;
    const float sw = wscale[kb];
    i32x8_t wf[NT], xf[MT];
    float sx[MT];
#pragma unroll
    for (int f = 0; f < NT; ++f)
      wf[f] = join(buf_ld16(wr, at(woff[f], lo), 0), buf_ld16(wr, at(woff[f], hi), 0));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      xf[i] = join(buf_ld16(xr, at(xoff[i], lo), 0), buf_ld16(xr, at(xoff[i], hi), 0));
      sx[i] = srow[i] >= 0 ? p.xs[int64_t(kb) * p.rows + srow[i]] * sw : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NT; ++f) {
        const f32x4_t d = mfma_e4m3(wf[f], xf[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[j], sx[i], acc[i][f][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int f = 0; f < NT; ++f) red[w][i * NT + f][lane] = acc[i][f];
  __syncthreads();
  for (int t = w; t < MT * NT; t += KW) {
    const int i = t / NT, f = t % NT;
    f32x4_t s = red[0][t][lane];
#pragma unroll
    for (int v = 1; v < KW; ++v) s += red[v][t][lane];
    const RowMap r = row_of<GROUPED>(p, first, 16 * i + a);
    const int n = n0 + 16 * f + 4 * g;
    if (r.y_row < 0 || n >= p.Ns) continue;
    if constexpr (GROUPED) {
      if (p.wt) s *= p.wt[r.y_row];
    }
    uint2 o = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    *reinterpret_cast<uint2*>(p.y + r.y_row * (int64_t(p.S) * p.Ns) + slice * p.Ns + n) = o;
  }
}

template <int MT, int NT, int KW, bool GROUPED>
hipError_t rows_of(const GemmParams& p, hipStream_t st) {
  const int ntiles = (p.Ns + 16 * NT - 1) / (16 * NT);
  const int64_t grid = int64_t(p.blocks) * p.S * ntiles;
  hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, NT, KW, GROUPED>), dim3(unsigned(grid)),
                     dim3(KW * kWave), 0, st, p, ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(GemmParams p, hipStream_t st) {
  const int rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  p.blocks = int32_t((p.M + rows - 1) / rows);
  if (rows == 16) return rows_of<1, 1, 8, false>(p, st);
  if (rows == 32) return rows_of<2, 1, 8, false>(p, st);
  return rows_of<4, 1, 8, false>(p, st);
}

hipError_t launch_fp8_moe_gemm(GemmParams p, hipStream_t st) {
  if (p.block_m == 16) return rows_of<1, 1, 8, true>(p, st);
  if (p.block_m == 32) return rows_of<2, 1, 8, true>(p, st);
  if (p.block_m == 64) return rows_of<4, 1, 8, true>(p, st);
  return rows_of<8, 1, 4, true>(p, st);
}

}  // namespace mlr
