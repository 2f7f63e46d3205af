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

// ---------------------------------------------------------------- many rows
// One LDS-direct load of 16 (or 4) bytes a lane: lane i's bytes land at lds +
// 16 i (4 i).  Inline assembly for the reason given at dma16; soff is added to
// every lane's offset.
__device__ __forceinline__ void tile_dma16(i32x4_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
  int saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}
__device__ __forceinline__ void tile_dma4(i32x4_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
  int saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %2, %3, %4 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}

// Work item -> (block of rows, column tile).  Consecutive workgroups go to the
// XCDs in turn, so each XCD takes one contiguous run of items and its L2 holds
// that run's operands; within the run, kGroup blocks of rows share each column
// tile before the next one.
constexpr int kGroup = 4;
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t blocks, uint32_t tiles, uint32_t* blk,
                                        uint32_t* tile) {
  const uint32_t total = blocks * tiles, per = total / kXcds, rem = total % kXcds;
  const uint32_t xcd = id % kXcds, i = id / kXcds;
  const uint32_t t = xcd * per + min(xcd, rem) + i;
  const uint32_t grp = t / (kGroup * tiles), first = grp * kGroup;
  const uint32_t size = min(uint32_t(kGroup), blocks - first), in = t - first * tiles;
  *blk = first + in % size;
  *tile = in / size;
}

// WM x WN wavefronts, each 16 FM rows x 16 FN columns.  A ring of NS stages of
// 128 of K in LDS, filled by LDS-direct loads; a stage holds the rows' bytes,
// the columns' bytes and the rows' scales.  A row's eight 16-byte chunks are
// permuted by an exclusive or with bits of the row number, so that the lanes
// that read one chunk of 16 rows spread over the banks; the load applies it to
// the source address.
template <int WM, int WN, int FM, int FN, int NS, bool GROUPED>
__global__ void __launch_bounds__(WM * WN * kWave, (WM * WN + 3) / 4)
    fp8_gemm_tile_kernel(GemmParams p, int ntiles) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN;
  constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // 1 KiB loads a wavefront and stage
  constexpr int kLoads = XI + WI + 1;
  constexpr int kX = 0, kW = BM * 128, kS = kW + BN * 128, kStage = kS + BM * 4;
  static_assert(XI * 8 * NW == BM && WI * 8 * NW == BN && BM % kWave == 0 && BM / kWave <= NW, "tile");
  constexpr int kFnBits = FN == 1 ? 2 : FN == 2 ? 3 : FN == 4 ? 4 : 5;
  __shared__ __align__(1024) uint8_t lds[NS * kStage];

  const uint32_t tiles = uint32_t(p.S) * ntiles;
  uint32_t blk, tile, blocks = uint32_t(p.blocks);
  if constexpr (GROUPED) blocks = min(blocks, uint32_t(p.ntpp[0]) / BM);
  if (blockIdx.x >= blocks * tiles) return;
  tile_of(blockIdx.x, blocks, tiles, &blk, &tile);
  int64_t e = 0;
  if constexpr (GROUPED) {
    e = p.eids[blk];
    if (e < 0 || e >= p.E) return;
  }
  const int slice = tile / ntiles, n0 = (tile % ntiles) * BN;
  const int64_t first = int64_t(blk) * BM;
  const int lane = lane_id(), w = wave_id(), wm = w / WN, wn = w % WN;
  const int a = lane & 15, g = lane >> 4;

  const int64_t mat = e * p.S + slice;
  const i32x4_t wr = dma_rsrc(p.w + mat * p.Ns * int64_t(p.K), uint32_t(p.Ns) * uint32_t(p.K));
  const int64_t x0 = GROUPED ? 0 : first;
  const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, BM);
  const i32x4_t xr = dma_rsrc(p.x + x0 * p.K, uint32_t(xrows * p.K));
  const i32x4_t sr = dma_rsrc(p.xs + x0, uint32_t(((p.KB - 1) * p.rows + xrows) * 4));
  uint32_t xoff[XI], woff[WI], soff;
  const int rl = lane >> 3, cl = lane & 7;  // row within a load, chunk as stored
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int r = 8 * (w * XI + i) + rl;
    const RowMap m = row_of<GROUPED>(p, first, r);
    xoff[i] = m.x_row < 0 ? kOob : uint32_t((m.x_row - x0) * p.K) + 16 * (cl ^ (r & 7));
  }
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    const int r = 8 * (w * WI + i) + rl, n = n0 + r;
    const int sw = (r & 3) | (((r >> kFnBits) & 1) << 2);
    woff[i] = n >= p.Ns ? kOob : uint32_t(n) * uint32_t(p.K) + 16 * (cl ^ sw);
  }
  const int seg = w % (BM / kWave);
  {
    const RowMap m = row_of<GROUPED>(p, first, seg * kWave + lane);
    soff = m.x_row < 0 ? kOob : uint32_t((m.x_row - x0) * 4);
  }
  const uint32_t base = lds_address(lds);
  const int tail = p.K & (kScaleBlock - 1);  // bytes of K in a short last block
  const uint32_t kstride = uint32_t(p.rows) * 4;

  auto load = [&](int kb) {
    const uint32_t st = base + uint32_t(kb % NS) * kStage;
    const uint32_t k = uint32_t(kb) * kScaleBlock;
    if (kb < p.KB - 1 || (kb == p.KB - 1 && tail == 0)) {
#pragma unroll
      for (int i = 0; i < XI; ++i) tile_dma16(xr, st + kX + 1024 * (w * XI + i), xoff[i], k);
#pragma unroll
      for (int i = 0; i < WI; ++i) tile_dma16(wr, st + kW + 1024 * (w * WI + i), woff[i], k);
      tile_dma4(sr, st + kS + 256 * seg, soff, uint32_t(kb) * kstride);
    } else {
      // the short last block (chunks past K are zeros), or a stage past the
      // end, loaded from nowhere so that every stage counts the same loads
      const int have = kb == p.KB - 1 ? tail : 0;
      const uint32_t kk = have ? k : 0;
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int r = 8 * (w * XI + i) + rl;
        tile_dma16(xr, st + kX + 1024 * (w * XI + i), 16 * (cl ^ (r & 7)) < have ? xoff[i] : kOob, kk);
      }
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const int r = 8 * (w * WI + i) + rl;
        const int sw = (r & 3) | (((r >> kFnBits) & 1) << 2);
        tile_dma16(wr, st + kW + 1024 * (w * WI + i), 16 * (cl ^ sw) < have ? woff[i] : kOob, kk);
      }
      tile_dma4(sr, st + kS + 256 * seg, have ? soff : kOob, have ? uint32_t(kb) * kstride : 0);
    }
  };

  // this wavefront's columns lie in one scale block: lane i keeps that of
  // K block i of the current 64
  const int nblk = std::min((n0 + wn * FN * 16) / kScaleBlock, p.NB - 1);
  const float* wscale = p.ws + (mat * p.NB + nblk) * p.KB;
  float wsv = lane < p.KB ? wscale[lane] : 0.0f;

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = f32x4_t{0, 0, 0, 0};

  const int xrow = wm * FM * 16 + a, wrow = wn * FN * 16 + 4 * FN * (a >> 2) + (a & 3);
  const int xo = kX + xrow * 128 + 16 * (g ^ (a & 7));
  const int wo = kW + wrow * 128 + 16 * (g ^ (a & 7));

#pragma unroll
  for (int s = 0; s < NS - 1; ++s) load(s);
  for (int kb = 0; kb < p.KB; ++kb) {
    if ((kb & 63) == 0 && kb > 0) wsv = kb + lane < p.KB ? wscale[kb + lane] : 0.0f;
    stage_barrier<(NS - 2) * kLoads>();
    load(kb + NS - 1);
    const uint8_t* st = lds + (kb % NS) * kStage;
    const float sw = __uint_as_float(
        __builtin_amdgcn_readlane(__float_as_uint(wsv), kb & 63));
    i32x8_t wf[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f)
      wf[f] = join(*reinterpret_cast<const uint4*>(st + wo + 512 * f),
                   *reinterpret_cast<const uint4*>(st + (wo ^ 64) + 512 * f));
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const i32x8_t xf = join(*reinterpret_cast<const uint4*>(st + xo + 2048 * i),
                              *reinterpret_cast<const uint4*>(st + (xo ^ 64) + 2048 * i));
      const float sx = *reinterpret_cast<const float*>(st + kS + 4 * (xrow + 16 * i)) * sw;
      f32x4_t d[FN];
#pragma unroll
      for (int f = 0; f < FN; ++f) d[f] = mfma_e4m3(wf[f], xf);
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[f][j], sx, acc[i][f][j]);
    }
  }

  // no load into LDS outlives its workgroup
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  const int nl = n0 + wn * FN * 16 + 4 * FN * g;  // this lane's 4 FN columns
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const RowMap m = row_of<GROUPED>(p, first, xrow + 16 * i);
    if (m.y_row < 0) continue;
    float wt = 1.0f;
    if constexpr (GROUPED) {
      if (p.wt) wt = p.wt[m.y_row];
    }
    uint16_t* out = p.y + m.y_row * (int64_t(p.S) * p.Ns) + int64_t(slice) * p.Ns + nl;
    if constexpr (FN == 1) {
      const f32x4_t v = acc[i][0] * wt;
      if (nl < p.Ns)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int f = 0; f < FN; f += 2) {
        const f32x4_t u = acc[i][f] * wt, v = acc[i][f + 1] * wt;
        if (nl + 4 * f < p.Ns)
          *reinterpret_cast<uint4*>(out + 4 * f) =
              make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]),
                         pack_bf16x2(v[2], v[3]));
      }
    }
  }
}

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED>
hipError_t tile_launch(GemmParams p, hipStream_t st) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16;
  if (!GROUPED) p.blocks = int32_t((p.M + BM - 1) / BM);
  const int ntiles = (p.Ns + BN - 1) / BN;
  const int64_t grid = int64_t(p.blocks) * p.S * ntiles;
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<WM, WN, FM, FN, NS, GROUPED>), dim3(unsigned(grid)),
                     dim3(WM * WN * kWave), 0, st, p, ntiles);
  return hipGetLastError();
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
  if (p.M > 64) return tile_launch<2, 4, 8, 4, 2, false>(p, st);
  const int rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  p.blocks = int32_t((p.M + rows - 1) / rows);
  if (rows == 16) return rows_of<1, 1, 8, false>(p, st);
  if (rows == 32) return rows_of<2, 1, 8, false>(p, st);
  return rows_of<4, 1, 8, false>(p, st);
}

hipError_t launch_fp8_moe_gemm(GemmParams p, hipStream_t st) {
  if (p.block_m == 16) return rows_of<1, 1, 8, true>(p, st);
  if (p.block_m == 32) return rows_of<2, 1, 8, true>(p, st);
  if (p.block_m == 64) return tile_launch<1, 4, 4, 4, 2, true>(p, st);
  return tile_launch<1, 4, 8, 4, 2, true>(p, st);
}

}  // namespace mlr
