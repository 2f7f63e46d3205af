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
template <int MT, int NT, int KW, int U, bool GROUPED>
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

  for (int kb0 = w; kb0 < p.KB; kb0 += KW * U) {
    i32x8_t wf[U][NT], xf[U][MT];
    float sx[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + u * KW;
      const uint32_t k = uint32_t(kb) * kScaleBlock;
      const bool in = kb < p.KB;  // past the end everything reads as zero
      const uint32_t lo = in && k + 16 * g < uint32_t(p.K) ? k : kOob;
      const uint32_t hi = in && k + 64 + 16 * g < uint32_t(p.K) ? k + 64 : kOob;
      const float sw = in ? wscale[kb] : 0.0f;
#pragma unroll
      for (int f = 0; f < NT; ++f)
        wf[u][f] = join(buf_ld16(wr, at(woff[f], lo), 0), buf_ld16(wr, at(woff[f], hi), 0));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xf[u][i] = join(buf_ld16(xr, at(xoff[i], lo), 0), buf_ld16(xr, at(xoff[i], hi), 0));
        sx[u][i] = in && srow[i] >= 0 ? p.xs[int64_t(kb) * p.rows + srow[i]] * sw : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NT; ++f) {
          const f32x4_t d = mfma_e4m3(wf[u][f], xf[u][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[j], sx[u][i], acc[i][f][j]);
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

// Work item -> (block of rows, column tile).  Workgroups go to the XCDs in
// turn, so each XCD takes one contiguous run of items, its workgroups in turn;
// its L2 then holds that run's operands.  Within the run kGroup blocks of rows
// share each column tile before the next one.
constexpr int kGroup = 4;
struct Items {
  uint32_t blocks, tiles;  // blocks of rows, column tiles (of all slices)
  uint32_t first, end;     // this XCD's run
  uint32_t step;           // its workgroups

  __device__ __forceinline__ Items(uint32_t b, uint32_t t) : blocks(b), tiles(t) {
    const uint32_t total = b * t, per = total / kXcds, rem = total % kXcds;
    const uint32_t xcd = blockIdx.x % kXcds;
    first = xcd * per + min(xcd, rem);
    end = first + per + (xcd < rem ? 1 : 0);
    step = (gridDim.x - xcd + kXcds - 1) / kXcds;
  }
  __device__ __forceinline__ void at(uint32_t t, uint32_t* blk, uint32_t* tile) const {
    const uint32_t grp = t / (kGroup * tiles), base = grp * kGroup;
    const uint32_t size = min(uint32_t(kGroup), blocks - base), in = t - base * tiles;
    *blk = base + in % size;
    *tile = in / size;
  }
};

// WM x WN wavefronts, each 16 FM rows x 16 FN columns of a tile.  A ring of NS
// stages of 128 of K in LDS, filled by LDS-direct loads; a stage holds the
// rows' bytes, the columns' bytes and their scales.  A row's eight 16-byte
// chunks are permuted by an exclusive or with bits of the row number, so that
// the lanes that read one chunk of 16 rows spread over the banks; the load
// applies it to the source address.
//
// A workgroup takes several tiles, and its ring runs on across them: the last
// stages of one are multiplied while the first of the next are on their way,
// and its results are stored in that time too.
template <int WM, int WN, int FM, int FN, int NS>
struct Tile {
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN;
  static constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // 1 KiB loads a wavefront and stage
  static constexpr int kLoads = XI + WI + 1;
  static constexpr int kX = 0, kW = BM * 128, kS = kW + BN * 128, kStage = kS + BM * 4 + 256;
  // tiles the loads run ahead by, and this one: the pairs of their rows
  static constexpr int kPairs = NS * kStage, kRing = NS + 1;
  static constexpr int lds_bytes(bool grouped) { return kPairs + (grouped ? kRing * BM * 4 : 0); }
  // workgroups of a CU, by LDS and by two wavefronts a SIMD
  static constexpr int groups(bool grouped) {
    const int a = 160 * 1024 / lds_bytes(grouped), b = 8 / NW;
    return a < b ? a : b;
  }
  static_assert(XI * 8 * NW == BM && WI * 8 * NW == BN && BM % kWave == 0, "tile");
  static_assert(BM / kWave < NW && FM % 2 == 0 && NS >= 2, "tile");
};

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED>
__global__ void __launch_bounds__(WM * WN * kWave, 2)
    fp8_gemm_tile_kernel(GemmParams p, int ntiles) {
  using T = Tile<WM, WN, FM, FN, NS>;
  constexpr int BM = T::BM, BN = T::BN, XI = T::XI, WI = T::WI, kLoads = T::kLoads;
  constexpr int kX = T::kX, kW = T::kW, kS = T::kS, kStage = T::kStage;
  constexpr int kFnBits = FN == 1 ? 2 : FN == 2 ? 3 : FN == 4 ? 4 : 5;
  __shared__ __align__(1024) uint8_t lds[T::lds_bytes(GROUPED)];

  uint32_t blocks = uint32_t(p.blocks);
  if constexpr (GROUPED) blocks = min(blocks, uint32_t(p.ntpp[0]) / BM);
  const Items items(blocks, uint32_t(p.S) * ntiles);
  const int lane = lane_id(), w = wave_id(), wm = w / WN, wn = w % WN;
  const int a = lane & 15, g = lane >> 4;
  const int rl = lane >> 3, cl = lane & 7;  // row within a load, chunk as stored
  auto swizzle = [](int r) { return (r & 3) | (((r >> kFnBits) & 1) << 2); };
  auto expert = [&](uint32_t blk) { return GROUPED ? p.eids[blk] : 0; };
  // the item from t on whose expert is one (the run's end if there is none)
  auto valid = [&](uint32_t t) {
    if constexpr (GROUPED) {
      for (; t < items.end; t += items.step) {
        uint32_t blk, tile;
        items.at(t, &blk, &tile);
        if (uint32_t(p.eids[blk]) < uint32_t(p.E)) break;
      }
    }
    return t;
  };

  // ---- the loading side: its tile, and how far it is
  uint32_t lt = valid(items.first + blockIdx.x / kXcds);
  uint32_t ct = lt;  // the tile being multiplied
  if (lt >= items.end) return;
  int lkb = 0, lstage = 0, lring = 0;
  i32x4_t wr, xr, sr;
  // Offsets of this lane's chunks: grouped rows lie anywhere; dense rows and
  // the columns follow each other, 8 rows a load (the columns' chunk order has
  // two forms), and what is behind the last row is behind the resource's range.
  constexpr int kXoff = GROUPED ? XI : 1;
  uint32_t xoff[kXoff], woff[2], soff;
  constexpr int kSegs = BM / kWave, kCols = (BN + kScaleBlock - 1) / kScaleBlock;
  const int sdst = kS + 256 * std::min(w, kSegs);
  const uint32_t sstride = w < kSegs ? uint32_t(p.rows) * 4 : 4;
  const uint32_t step8 = 8 * uint32_t(p.K);
  const uint32_t base = lds_address(lds);
  int32_t* pairs = reinterpret_cast<int32_t*>(lds + T::kPairs);

  auto set_tile = [&]() {
    if (lt >= items.end) {  // nothing left: loads from nowhere
#pragma unroll
      for (int i = 0; i < kXoff; ++i) xoff[i] = kOob;
      woff[0] = woff[1] = soff = kOob;
      return;
    }
    uint32_t blk, tile;
    items.at(lt, &blk, &tile);
    const int slice = tile / ntiles, n0 = (tile % ntiles) * BN;
    const int64_t first = int64_t(blk) * BM;
    const int64_t mat = int64_t(expert(blk)) * p.S + slice;
    wr = dma_rsrc(p.w + mat * p.Ns * int64_t(p.K), uint32_t(p.Ns) * uint32_t(p.K));
    const int64_t x0 = GROUPED ? 0 : first;
    const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, BM);
    xr = dma_rsrc(p.x + x0 * p.K, uint32_t(xrows * p.K));
#pragma unroll
    for (int i = 0; i < kXoff; ++i) {
      const int r = 8 * (w * XI + i) + rl;
      if constexpr (GROUPED) {
        const RowMap m = row_of<GROUPED>(p, first, r);
        xoff[i] = m.x_row < 0 ? kOob : uint32_t(m.x_row * p.K) + 16 * (cl ^ rl);
      } else {
        xoff[i] = uint32_t(r) * uint32_t(p.K) + 16 * (cl ^ rl);
      }
    }
    const int r = 8 * w * WI + rl;
    const uint32_t n = uint32_t(n0 + r) * uint32_t(p.K);
    woff[0] = n + 16 * (cl ^ swizzle(rl));
    woff[1] = n + 16 * (cl ^ swizzle(rl) ^ 4);
    // The stage's scales: the first wavefronts load those of 64 rows each, the
    // others (all alike) those of the tile's column blocks.
    const float* from = w < kSegs ? p.xs + x0 : p.ws + mat * p.NB * p.KB;
    const int64_t count = w < kSegs ? (p.KB - 1) * p.rows + xrows : int64_t(p.NB) * p.KB;
    sr = dma_rsrc(from, uint32_t(count * 4));
    if (w < kSegs) {
      const RowMap m = row_of<GROUPED>(p, first, w * kWave + lane);
      soff = m.x_row < 0 ? kOob : uint32_t((m.x_row - x0) * 4);
      if constexpr (GROUPED) pairs[lring * BM + w * kWave + lane] = int32_t(m.y_row);
    } else {
      const int nb = n0 / kScaleBlock + lane;
      soff = lane < kCols && nb < p.NB ? uint32_t(nb) * uint32_t(p.KB) * 4 : kOob;
    }
  };
  // One of a stage's loads.  Chunks past K in a short last block read as
  // zeros; behind the last tile everything does, so that every stage counts the
  // same loads.  (An offset stays below 2 GiB until kOob's bit is set in it.)
  auto load = [&](int l) {
    const uint32_t st = base + uint32_t(lstage) * kStage;
    const int have = p.K - lkb * kScaleBlock;
    const uint32_t k = uint32_t(lkb) * kScaleBlock;
    if (l < XI) {
      const uint32_t m = 16 * (cl ^ rl) < have ? 0 : kOob;
      const uint32_t o = GROUPED ? xoff[l % kXoff] : xoff[0] + uint32_t(l) * step8;
      tile_dma16(xr, st + kX + 1024 * (w * XI + l), o | m, k);
    } else if (l < XI + WI) {
      const int i = l - XI;
      const int flip = swizzle(8 * (w * WI + i)) >> 2;  // uniform: bit kFnBits of the row
      const uint32_t m = 16 * (cl ^ swizzle(rl) ^ (4 * flip)) < have ? 0 : kOob;
      tile_dma16(wr, st + kW + 1024 * (w * WI + i), ((flip ? woff[1] : woff[0]) + uint32_t(i) * step8) | m, k);
    } else {
      tile_dma4(sr, st + sdst, soff, uint32_t(lkb) * sstride);
    }
  };
  auto loaded = [&]() {  // a stage's loads are all issued
    ++lkb;
    lstage = lstage + 1 == NS ? 0 : lstage + 1;
  };
  auto next_loads = [&]() {
    lkb = 0;
    if (lt < items.end) lt = valid(lt + items.step);
    lring = lring + 1 == T::kRing ? 0 : lring + 1;
    set_tile();
  };

  // ---- the multiplying side
  f32x4_t acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int f = 0; f < FN; ++f) acc[i][f] = f32x4_t{0, 0, 0, 0};
  };
  const int xrow = wm * FM * 16 + a, wrow = wn * FN * 16 + 4 * FN * (a >> 2) + (a & 3);
  const int xo = kX + xrow * 128 + 16 * (g ^ (a & 7));
  const int wo = kW + wrow * 128 + 16 * (g ^ (a & 7));
  const int so = kS + BM * 4 + wn * FN * 16 / kScaleBlock * 4;  // this wavefront's column block

  // A stage is FM steps of FN MFMAs: a step reads the next one's rows, and a
  // result's multiply-adds run FN MFMAs after it.  The loop's one barrier
  // stands before the last step, once every wavefront has its last rows of the
  // stage in registers; behind it the stage's buffer is refilled, and each
  // column operand is replaced by the next stage's after its last use.  The
  // scheduling barriers keep the compiler from undoing this order.
  i32x8_t wf[FN], xf[2];
  float sx[2], sd = 0.0f, sw;
  f32x4_t d[FN];
  auto add = [&](int i, int f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[f][j], sd, acc[i][f][j]);
  };
  auto columns = [&](const uint8_t* st, int f) {
    wf[f] = join(*reinterpret_cast<const uint4*>(st + wo + 512 * f),
                 *reinterpret_cast<const uint4*>(st + (wo ^ 64) + 512 * f));
  };
  auto rows = [&](const uint8_t* st, int i) {
    xf[i & 1] = join(*reinterpret_cast<const uint4*>(st + xo + 2048 * i),
                     *reinterpret_cast<const uint4*>(st + (xo ^ 64) + 2048 * i));
    sx[i & 1] = *reinterpret_cast<const float*>(st + kS + 4 * (xrow + 16 * i));
  };
  set_tile();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) load(l);
    loaded();
    if (lkb == p.KB) next_loads();
  }
  stage_barrier<(NS - 1) * kLoads>();
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    columns(lds, f);
    d[f] = f32x4_t{0, 0, 0, 0};
  }
  rows(lds, 0);
  sw = *reinterpret_cast<const float*>(lds + so);
  clear();
  int kb = 0, stage = 0, ring = 0;
  while (true) {
    // stages until one side changes its tile
    const int n = std::min(p.KB - kb, p.KB - lkb);
    for (int r = 0; r < n; ++r) {
      const uint8_t* st = lds + stage * kStage;
      stage = stage + 1 == NS ? 0 : stage + 1;
      const uint8_t* nx = lds + stage * kStage;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float s = sx[i & 1] * sw;
        if (i < FM - 1) {
          rows(st, i + 1);
        } else {
          stage_barrier<(NS - 2) * kLoads>();
          rows(nx, 0);
          sw = *reinterpret_cast<const float*>(nx + so);
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          add((i + FM - 1) % FM, f);
          d[f] = mfma_e4m3(wf[f], xf[i & 1]);
          if (i == FM - 1) {
            columns(nx, f);
#pragma unroll
            for (int l = kLoads * f / FN; l < kLoads * (f + 1) / FN; ++l) load(l);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        sd = s;
      }
      loaded();
    }
    kb += n;
    if (lkb == p.KB) next_loads();
    if (kb < p.KB) continue;
    // the tile is done
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      add(FM - 1, f);
      d[f] = f32x4_t{0, 0, 0, 0};
    }
    uint32_t blk, tile;
    items.at(ct, &blk, &tile);
    const int slice = tile / ntiles;
    const int nl = (tile % ntiles) * BN + wn * FN * 16 + 4 * FN * g;  // this lane's 4 FN columns
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      int64_t y;
      float wt = 1.0f;
      if constexpr (GROUPED) {
        y = pairs[ring * BM + xrow + 16 * i];
        if (y < 0) continue;
        if (p.wt) wt = p.wt[y];
      } else {
        y = int64_t(blk) * BM + xrow + 16 * i;
        if (y >= p.M) continue;
      }
      uint16_t* out = p.y + y * (int64_t(p.S) * p.Ns) + int64_t(slice) * p.Ns + nl;
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
    ct = valid(ct + items.step);
    if (ct >= items.end) break;
    clear();
    kb = 0;
    ring = ring + 1 == T::kRing ? 0 : ring + 1;
  }
  // no load into LDS outlives its workgroup
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED>
hipError_t tile_launch(GemmParams p, hipStream_t st) {
  using T = Tile<WM, WN, FM, FN, NS>;
  if (!GROUPED) p.blocks = int32_t((p.M + T::BM - 1) / T::BM);
  const int ntiles = (p.Ns + T::BN - 1) / T::BN;
  const int64_t resident = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * T::groups(GROUPED);
  const int64_t grid = std::min(int64_t(p.blocks) * p.S * ntiles, resident);
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<WM, WN, FM, FN, NS, GROUPED>), dim3(unsigned(grid)),
                     dim3(T::NW * kWave), 0, st, p, ntiles);
  return hipGetLastError();
}

template <int MT, int NT, int KW, int U, bool GROUPED>
hipError_t rows_of(const GemmParams& p, hipStream_t st) {
  const int ntiles = (p.Ns + 16 * NT - 1) / (16 * NT);
  const int64_t grid = int64_t(p.blocks) * p.S * ntiles;
  hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, NT, KW, U, GROUPED>), dim3(unsigned(grid)),
                     dim3(KW * kWave), 0, st, p, ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(GemmParams p, hipStream_t st) {
  if (p.M > 64) return tile_launch<2, 4, 8, 4, 2, false>(p, st);
  const int rows = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
  p.blocks = int32_t((p.M + rows - 1) / rows);
  if (rows == 16) return rows_of<1, 1, 8, 2, false>(p, st);
  if (rows == 32) return rows_of<2, 1, 8, 1, false>(p, st);
  return rows_of<4, 1, 8, 1, false>(p, st);
}

hipError_t launch_fp8_moe_gemm(GemmParams p, hipStream_t st) {
  if (p.block_m == 16) return rows_of<1, 2, 8, 1, true>(p, st);
  if (p.block_m == 32) return rows_of<2, 2, 8, 1, true>(p, st);
  if (p.block_m == 64) return tile_launch<1, 4, 4, 2, 3, true>(p, st);
  return tile_launch<2, 4, 4, 4, 3, true>(p, st);
}

}  // namespace mlr
