// bf16 products with an epilogue, dense or over the routed pairs of an expert's
// blocks:
//   z[m, n] = wt[m] (sum_k x[m, k] w[n, k] + bias[n]) + delta[m, n]
//   y[m, n] = act(z)[m, n] + residual[m, n]
// where a gated activation takes gate z[m, n] and up z[m, n + N / 2].
//
// v_mfma_f32_16x16x32_bf16 with W as its first operand and X as its second: a
// lane then holds one row of X (lane % 16) and four consecutive columns of Y.
// Both operands give lane group g = lane / 16 the 16-byte chunks g and g + 4 of
// 128 bytes (64 of K), one for each of two products.  All sums are fp32, and so
// is the epilogue; Y is rounded once.
#include <algorithm>
#include <cmath>

#include "base.h"
#include "common.h"
#include "dma.h"
#include "internal.h"
#include "tiles.h"

namespace mlr {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kStageK = 64;  // of K a stage: 128 bytes

__device__ __forceinline__ f32x4_t mfma_bf16(const uint4& w, const uint4& x, const f32x4_t& acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x),
                                                 acc, 0, 0, 0);
}

// ---------------------------------------------------------------- epilogue
__device__ __forceinline__ f32x4_t widen(const uint2& v) {
  return f32x4_t{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
// 1 / (1 + exp(-v)): the hardware's exponential of a rounded argument, off by some
// |v| 2^-23 of its value, and its reciprocal; 0 from v = -88.7 down
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

__device__ __forceinline__ f32x4_t activate(f32x4_t v, int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= sigmoid(v[j]);
  } else if (act == kActGeluTanh) {
    // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= sigmoid(1.5957691216057308f * (v[j] + 0.044715f * v[j] * v[j] * v[j]));
  }
  return v;
}
__device__ __forceinline__ f32x4_t gate_up(f32x4_t g, f32x4_t u, int act) {
  if (act == kActSiluMul) {
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
  } else {
    // the clamps keep NaN
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = g[j] > 7.0f ? 7.0f : g[j];
      const float b = u[j] > 7.0f ? 7.0f : (u[j] < -7.0f ? -7.0f : u[j]);
      g[j] = a * sigmoid(1.702f * a) * (b + 1.0f);
    }
  }
  return g;
}

// Four columns of a row of Y from the sums of them (and of the up columns).
// `bias` is the expert's; y the row, `col` the first column.
__device__ __forceinline__ f32x4_t finish(const ProductParams& p, f32x4_t v, f32x4_t u, const uint16_t* bias,
                                          int64_t y, int col, float wt) {
  auto four = [](const uint16_t* from) { return widen(*reinterpret_cast<const uint2*>(from)); };
  const int up = p.No;  // the up column of gate column 0
  if (bias) {
    v += four(bias + col);
    if (p.gated) u += four(bias + up + col);
  }
  v *= wt;
  u *= wt;
  if (p.delta) {
    const uint16_t* d = p.delta + y * p.N + col;
    v += four(d);
    if (p.gated) u += four(d + up);
  }
  v = p.gated ? gate_up(v, u, p.act) : activate(v, p.act);
  if (p.residual) v += four(p.residual + y * p.No + col);
  return v;
}
__device__ __forceinline__ void store(const ProductParams& p, f32x4_t v, int64_t y, int col) {
  const int64_t at = y * p.No + col;
  if (p.out32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.y) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// ---------------------------------------------------------------- few rows
// One workgroup computes 16 MT rows x 16 NT columns of W: its kSplit wavefronts
// take the stages w, w + kSplit, ... of K straight from memory and add their sums
// in LDS, in order.  Gated, the even groups of 16 columns are gate's and the odd
// ones the same of up.  Grouped, the workgroups of a block take its pieces of 16
// rows in steps of `step` rows.
constexpr int kSplit = 8;
template <int MT, int NT, bool GROUPED>
__global__ void __launch_bounds__(kSplit * kWave) gemm_rows_kernel(ProductParams p, int ntiles, uint32_t step) {
  __shared__ f32x4_t red[kSplit][MT * NT][kWave];
  const int tile = blockIdx.x % ntiles;
  const int lane = lane_id(), w = wave_id(), a = lane & 15, g = lane >> 4;
  const uint32_t piece = blockIdx.x / ntiles;
  const int64_t first = int64_t(piece) * 16 * MT;  // dense: the first row
  int64_t e = 0;
  // grouped: the block's ids, one or two a lane, which of them are a pair's, and
  // where in the block the piece begins
  int32_t id0 = -1, id1 = -1;
  uint64_t held0 = 0, held1 = 0;
  uint32_t at = 0;
  const uint32_t block_m = p.block_m;
  // goes to the first piece from `at` on, in this workgroup's steps, that has a pair
  auto seek = [&]() {
    for (; at < block_m; at += step)
      if ((at < kWave ? held0 : held1) >> (at % kWave) & ((uint64_t(1) << 16 * MT) - 1)) return true;
    return false;
  };
  // row i of the piece
  auto row_at = [&](int i) {
    if constexpr (GROUPED)
      return row_of_pair(p, uint32_t(__shfl(at < kWave ? id0 : id1, at % kWave + i)));
    else
      return row_of<false>(p, first, i);
  };
  if constexpr (GROUPED) {
    // a block's workgroups are neighbours; what lies behind the last block comes last
    const uint32_t parts = step / (16 * MT), block = piece / parts;
    at = piece % parts * (16 * MT);
    const int64_t start = int64_t(block) * block_m;
    const int32_t* ids = p.sorted + start;
    // (read behind the last block, too, in one wait, and not used)
    const int32_t used = p.ntpp[0];
    if (uint32_t(lane) < block_m) id0 = ids[lane];
    if (uint32_t(kWave + lane) < block_m) id1 = ids[kWave + lane];
    e = p.eids[block];
    if (start >= used || e < 0 || e >= p.E) return;
    held0 = __ballot(uint32_t(id0) < uint32_t(p.numel));
    held1 = __ballot(uint32_t(id1) < uint32_t(p.numel));
    if (!seek()) return;  // padding
  }

  const uint32_t K2 = uint32_t(p.K) * 2;
  const auto wr = make_rsrc(p.w + e * p.N * int64_t(p.K), uint32_t(p.N) * K2);
  // An offset is below 2 GiB or, for rows and columns that are not there, kOob;
  // so is an offset along K.  One of the two takes the sum out of range, which
  // reads as zero; both wrap to 0, and what is read there reaches no output.
  uint32_t woff[NT];
  int col[NT];  // this lane's first column of Y
#pragma unroll
  for (int f = 0; f < NT; ++f) {
    int n;
    if (p.gated) {
      col[f] = tile * 8 * NT + 16 * (f >> 1);
      n = col[f] + a < p.No ? col[f] + a + (f & 1) * p.No : p.N;
    } else {
      col[f] = tile * 16 * NT + 16 * f;
      n = col[f] + a;
    }
    col[f] += 4 * g;
    woff[f] = n < p.N ? uint32_t(n) * K2 + 16 * g : kOob;
  }
  for (;;) {
    // rows of X: dense tiles are addressed from their first row, grouped ones
    // from row 0 (X is below 2 GiB there)
    const int64_t x0 = GROUPED ? 0 : first;
    const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, 16 * MT);
    const auto xr = make_rsrc(p.x + x0 * p.K, uint32_t(xrows * K2));
    uint32_t xoff[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const RowMap r = row_at(16 * i + a);
      xoff[i] = r.x_row >= 0 ? uint32_t((r.x_row - x0) * K2) + 16 * g : kOob;
    }

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NT; ++f) acc[i][f] = f32x4_t{0, 0, 0, 0};

    for (int kb = w; kb < p.KB; kb += kSplit) {
      const uint32_t k = uint32_t(kb) * (2 * kStageK);
      const uint32_t lo = k + 16 * g < K2 ? k : kOob;
      const uint32_t hi = k + 64 + 16 * g < K2 ? k + 64 : kOob;
      uint4 wl[NT], wh[NT], xl[MT], xh[MT];
#pragma unroll
      for (int f = 0; f < NT; ++f) {
        wl[f] = buf_ld16(wr, woff[f] + lo, 0);
        wh[f] = buf_ld16(wr, woff[f] + hi, 0);
      }
      __builtin_amdgcn_sched_barrier(0);  // the columns' loads first, a line's two halves together
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        xl[i] = buf_ld16(xr, xoff[i] + lo, 0);
        xh[i] = buf_ld16(xr, xoff[i] + hi, 0);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NT; ++f) {
          acc[i][f] = mfma_bf16(wl[f], xl[i], acc[i][f]);
          acc[i][f] = mfma_bf16(wh[f], xh[i], acc[i][f]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NT; ++f) red[w][i * NT + f][lane] = acc[i][f];
    __syncthreads();
    const uint16_t* bias = p.bias ? p.bias + e * p.N : nullptr;
#pragma unroll
    for (int t = 0; t < MT * NT; ++t) {
      const int i = t / NT, f = t % NT;
      // gated, the wavefront of the even group takes both
      if (t % kSplit != w || (p.gated && (f & 1))) continue;
      auto sum = [&](int t) {
        f32x4_t s = red[0][t][lane];
#pragma unroll
        for (int v = 1; v < kSplit; ++v) s += red[v][t][lane];
        return s;
      };
      const RowMap r = row_at(16 * i + a);
      const f32x4_t s = sum(t);
      f32x4_t u = {0, 0, 0, 0};
      if (NT > 1 && p.gated) u = sum(NT > 1 ? t + 1 : t);
      if (r.y_row < 0 || col[f] >= p.No) continue;
      const float wt = GROUPED && p.wt ? p.wt[r.y_row] : 1.0f;
      store(p, finish(p, s, u, bias, r.y_row, col[f], wt), r.y_row, col[f]);
    }
    if constexpr (!GROUPED) return;
    at += step;
    if (!seek()) return;
    __syncthreads();  // the sums have been read
  }
}

// ---------------------------------------------------------------- many rows
// WM x WN wavefronts, each 16 FM rows x 16 FN columns of a tile.  A ring of NS
// stages of 64 of K in LDS, filled by LDS-direct loads; a stage holds the rows'
// and the columns' bytes, 128 of each.  A row's eight 16-byte chunks are permuted
// by an exclusive or with bits of the row number, so that the lanes that read one
// chunk of 16 rows spread over the banks; the load applies it to the source
// address.  Gated, four gate columns and the same four of up take turns among a
// tile's columns, so that a lane's two sums of each 32 are the gate's and the up's
// of four columns; only the loads' source addresses and the epilogue know.
//
// A workgroup takes several tiles, and its ring runs on across them: the last
// stages of one are multiplied while the first of the next are on their way,
// and its results are stored in that time too.
//
// KG > 1, for small tiles: a stage has KG blocks of 64, each of which WM x WN
// wavefronts multiply, and their sums meet in LDS.
template <int WM, int WN, int FM, int FN, int NS, int KG = 1>
struct Tile {
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN * KG;
  static constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // 1 KiB loads a wavefront and K block
  static constexpr int kEach = XI + WI, kLoads = KG * kEach;
  static constexpr int kX = 0, kW = BM * 128, kBlock = kW + BN * 128;
  static constexpr int kStage = KG * kBlock;
  static constexpr int kJoin = NS * kStage;  // (KG > 1) sums of the other wavefronts
  // the rows' pairs and weights of the tile being stored, of those whose stages
  // are in the ring (one each where K is one block), and of the next to load
  static constexpr int kPairs = NS * kStage, kRing = NS + 2, kList = kPairs + kRing * BM * 8;
  static constexpr int lds_bytes(bool grouped) {
    return grouped ? kList + int(sizeof(TileList)) : kPairs + (KG - 1) * BM * BN * 4;
  }
  // workgroups of a CU, by LDS and by two wavefronts a SIMD
  static constexpr int groups(bool grouped) {
    const int a = 160 * 1024 / lds_bytes(grouped), b = 8 / NW;
    return a < b ? a : b;
  }
  static_assert(XI * 8 * NW == BM && WI * 8 * NW == BN, "tile");
  static_assert(BM <= NW * kWave && FM % 2 == 0 && FN % 2 == 0 && NS >= 2, "tile");
};

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KG>
__global__ void __launch_bounds__(WM * WN * KG * kWave, 2) gemm_tile_kernel(ProductParams p, int ntiles) {
  using T = Tile<WM, WN, FM, FN, NS, KG>;
  constexpr int BM = T::BM, BN = T::BN, XI = T::XI, WI = T::WI, kLoads = T::kLoads;
  // whether the columns' loads run ahead of the rows' (below)
  constexpr bool kEarly = FM > 2;
  static_assert(KG == 1 || (!GROUPED && !kEarly), "a stage of several K blocks");
  constexpr int kX = T::kX, kW = T::kW, kStage = T::kStage;
  const int stages = (p.KB + KG - 1) / KG;  // of a tile
  __shared__ __align__(1024) uint8_t lds[T::lds_bytes(GROUPED)];

  TileList* list = reinterpret_cast<TileList*>(lds + T::kList);
  int blocks = 0;  // grouped: blocks of this launch
  uint32_t row_tiles;
  if constexpr (GROUPED) {
    blocks = std::min(p.blocks, p.ntpp[0] / p.block_m - p.block0);
    if (blocks <= 0) return;
    row_tiles = list->build(p.eids + p.block0, blocks, p.E, BM / p.block_m,
                            reinterpret_cast<uint64_t*>(lds), T::NW);
  } else {
    row_tiles = uint32_t((p.M + BM - 1) / BM);
  }
  const Items<GROUPED ? 1 : 4> items(row_tiles, uint32_t(ntiles));
  const int lane = lane_id(), w = wave_id(), kg = w / (WM * WN), wm = w / WN % WM, wn = w % WN;
  const int a = lane & 15, g = lane >> 4;
  const int rl = lane >> 3, cl = lane & 7;  // row within a load, chunk as stored
  auto swizzle = [](int r) { return (r & 3) | ((r >> 1) & 4); };  // bits 0, 1, 3
  const uint32_t K2 = uint32_t(p.K) * 2;
  const bool gated = p.gated;

  // ---- the loading side: its tile, and how far it is
  uint32_t lt = items.first + blockIdx.x / kXcds;
  uint32_t ct = lt;  // the tile being multiplied
  if (lt >= items.end) return;
  int lkb = 0, lstage = 0, lring = 0;
  i32x4_t wr, xr;
  // A load takes 8 rows, 8 chunks of each.  Dense rows and the columns follow
  // each other, and what is behind the last one is behind the resource's range
  // (or, of a gate, an up column, which no output takes); grouped rows lie
  // anywhere: lane i keeps the offset of this wavefront's row i.  The columns'
  // chunk order has two forms, by bit 3 of the column.
  const int xc = 16 * (cl ^ rl), wc = 16 * (cl ^ swizzle(rl));
  uint32_t xoff, woff, woff1;
  const uint32_t xstep = 8 * K2, wstep = gated ? 4 * K2 : 8 * K2;
  const uint32_t base = lds_address(lds);
  int2* pairs = reinterpret_cast<int2*>(lds + T::kPairs);

  auto set_tile = [&]() {
    uint32_t nx = kOob, nw = kOob, nw1 = kOob;  // nothing left: loads from nowhere
    if (lt < items.end) {
      // not to be computed once and kept: the registers are needed
      int ln = lane;
      asm volatile("" : "+v"(ln));
      uint32_t row, tile;
      items.at(lt, &row, &tile);
      int64_t first = int64_t(row) * BM, mat = 0;
      const int32_t* eids = p.eids + p.block0;
      int blk = 0, e = 0;
      if constexpr (GROUPED) {
        blk = list->block(row);
        e = eids[blk];
        first = int64_t(p.block0 + blk) * p.block_m;
        mat = e;
      }
      // row i of the tile; a grouped tile ends where its expert does
      auto row_at = [&](int i) {
        if constexpr (GROUPED) {
          const int b = blk + i / p.block_m;
          if (b >= blocks || eids[b] != e) return RowMap{-1, -1};
        }
        return row_of<GROUPED>(p, first, i);
      };
      wr = dma_rsrc(p.w + mat * p.N * int64_t(p.K), uint32_t(p.N) * K2);
      const int64_t x0 = GROUPED ? 0 : first;
      const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, BM);
      xr = dma_rsrc(p.x + x0 * p.K, uint32_t(xrows * K2));
      if constexpr (GROUPED) {
        const RowMap m = row_at(8 * w * XI + ln % (8 * XI));
        if (m.x_row >= 0) nx = uint32_t(m.x_row * K2);
        const int i = w * kWave + ln;
        if (i < BM) {
          const RowMap r = row_at(i);
          const float wt = p.wt && r.y_row >= 0 ? p.wt[r.y_row] : 1.0f;
          pairs[lring * BM + i] = make_int2(int32_t(r.y_row), __float_as_int(wt));
        }
      } else {
        nx = uint32_t(8 * w * XI + (ln >> 3)) * K2 + xc;
      }
      const uint32_t r = ln >> 3;
      const uint32_t n = gated ? tile * (BN / 2) + 4 * w * WI + (r & 3) + (r >> 2) * p.No
                               : tile * BN + 8 * w * WI + r;
      nw = n * K2;
      nw1 = nw + (wc ^ 64);
      nw += wc;
    }
    xoff = nx;
    woff = nw;
    woff1 = nw1;
  };
  // One of a stage's loads.  Chunks past K in a short last block read as
  // zeros; behind the last tile everything does, so that every stage counts the
  // same loads.
  auto load = [&](int l) {
    const int kb = KG == 1 ? lkb : lkb * KG + l / T::kEach;
    const uint32_t st = base + uint32_t(lstage) * kStage + uint32_t(l / T::kEach * T::kBlock);
    l %= T::kEach;
    // (a stage's second block may be past K)
    const uint32_t k = kb < p.KB ? uint32_t(kb) * (2 * kStageK) : 0;
    const int have = kb < p.KB ? int(K2 - k) : 0;
    if (l < XI) {
      const uint32_t o = GROUPED ? __builtin_amdgcn_ds_bpermute(4 * (8 * l + rl), xoff) + xc
                                 : xoff + uint32_t(l) * xstep;
      tile_dma16(xr, st + kX + 1024 * (w * XI + l), xc < have ? o : kOob, k);
    } else {
      const int i = l - XI;
      const int flip = 16 * swizzle(8 * (w * WI + i));
      tile_dma16(wr, st + kW + 1024 * (w * WI + i),
                 (wc ^ flip) < have ? (flip ? woff1 : woff) + uint32_t(i) * wstep : kOob, k);
    }
  };
  auto loaded = [&]() {  // a stage's loads are all issued
    ++lkb;
    lstage = lstage + 1 == NS ? 0 : lstage + 1;
  };
  auto next_loads = [&]() {
    lkb = 0;
    if (lt < items.end) lt += items.step;
    lring = lring + 1 == T::kRing ? 0 : lring + 1;
    set_tile();
  };

  // ---- the multiplying side
  const int xrow = wm * FM * 16 + a, wrow = wn * FN * 16 + 8 * (a >> 2) + (a & 3);
  const int ko = kg * T::kBlock;  // this wavefront's K block of a stage
  const int xo = ko + kX + xrow * 128 + 16 * (g ^ (a & 7));
  const int wo = ko + kW + wrow * 128 + 16 * (g ^ (a & 7));
  constexpr int kWait = (NS - 2) * kLoads + (kEarly ? WI : 0);  // younger loads at a stage's barrier

  set_tile();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) load(l);
    loaded();
    if (lkb == stages) next_loads();
  }
  stage_barrier<(NS - 1) * kLoads>();
  int stage = 0, ring = 0;
  for (; ct < items.end; ct += items.step, ring = ring + 1 == T::kRing ? 0 : ring + 1) {
    uint32_t row, tile;
    items.at(ct, &row, &tile);
    const int n0 = tile * (gated ? BN / 2 : BN) + wn * FN * (gated ? 8 : 16);  // this wavefront's columns of Y
    // A wavefront without a row or a column of the tile only loads and keeps the
    // barriers.
    bool none = n0 >= p.No;
    if constexpr (GROUPED) {
      constexpr int kRows = FM * 16;
      const int2* own = pairs + ring * BM + wm * kRows;
      bool row = own[lane % kRows].x >= 0;
      if constexpr (kRows > kWave) row |= own[kWave + lane].x >= 0;
      none |= __ballot(row) == 0;
    } else {
      none |= int64_t(row) * BM + wm * FM * 16 >= p.M;
    }
    if (none) {
      for (int kb = 0; kb < stages; ++kb) {
        if constexpr (kEarly) {
          asm volatile("s_barrier" ::: "memory");
#pragma unroll
          for (int l = XI; l < XI + WI; ++l) load(l);
        }
        stage_barrier<kWait>();
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          if (!kEarly || l < XI) load(l);
        loaded();
        stage = stage + 1 == NS ? 0 : stage + 1;
        if (lkb == stages) next_loads();
      }
      if constexpr (KG > 1) asm volatile("s_barrier" ::: "memory");  // of the sums
      continue;
    }

    // A stage is FM steps of 2 FN MFMAs: a step reads the next one's rows.  The
    // stage's barrier stands before the last step, once every wavefront has its
    // last rows of the stage in registers; behind it the stage's buffer is
    // refilled, and each column operand is replaced by the next stage's after its
    // last use.  With more than two steps a second barrier, behind the first step,
    // says that every wavefront has the stage's columns in registers, and their
    // buffer is refilled from there on.  The scheduling barriers keep the compiler
    // from undoing this order.
    f32x4_t acc[FM][FN];
    uint4 wf[2][FN], xf[2][2];
    auto columns = [&](const uint8_t* st, int h, int f) {
      const int o = 4096 * (f >> 1) + 512 * (f & 1);
      wf[h][f] = *reinterpret_cast<const uint4*>(st + (h ? wo ^ 64 : wo) + o);
    };
    auto rows = [&](const uint8_t* st, int i) {
      xf[i & 1][0] = *reinterpret_cast<const uint4*>(st + xo + 2048 * i);
      xf[i & 1][1] = *reinterpret_cast<const uint4*>(st + (xo ^ 64) + 2048 * i);
    };
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      columns(lds + stage * kStage, 0, f);
      columns(lds + stage * kStage, 1, f);
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i][f] = f32x4_t{0, 0, 0, 0};
    }
    rows(lds + stage * kStage, 0);
    for (int kb = 0; kb < stages;) {
      // the stages until the loads change their tile
      const int n = std::min(stages - kb, stages - lkb);
      for (int r = 0; r < n; ++r) {
        const uint8_t* st = lds + stage * kStage;
        stage = stage + 1 == NS ? 0 : stage + 1;
        const uint8_t* nx = lds + stage * kStage;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          if (kEarly && i == 1) asm volatile("s_barrier" ::: "memory");
          if (i < FM - 1) {
            rows(st, i + 1);
          } else {
            stage_barrier<kWait>();
            rows(nx, 0);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < FN; ++f) {
              const int at = h * FN + f;
              acc[i][f] = mfma_bf16(wf[h][f], xf[i & 1][h], acc[i][f]);
              if (i == FM - 1) {
                columns(nx, h, f);
#pragma unroll
                for (int l = kLoads * at / (2 * FN); l < kLoads * (at + 1) / (2 * FN); ++l)
                  if (!kEarly || l < XI) load(l);
              }
              if (kEarly && i >= 1 && i < FM - 1) {
                constexpr int kSlots = kEarly ? (FM - 2) * 2 * FN : 1;
                const int slot = (i - 1) * 2 * FN + at;
#pragma unroll
                for (int l = WI * slot / kSlots; l < WI * (slot + 1) / kSlots; ++l) load(XI + l);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
        }
        loaded();
      }
      kb += n;
      if (lkb == stages) next_loads();
    }

    if constexpr (KG > 1) {
      // The first wavefronts add the others' sums, in order, and store.  The next
      // sums are written behind a stage's barrier, when these have been read.
      f32x4_t* other = reinterpret_cast<f32x4_t*>(lds + T::kJoin) + (w % (WM * WN)) * FM * FN * kWave + lane;
      constexpr int kAll = WM * WN * FM * FN * kWave;
      if (kg > 0) {
#pragma unroll
        for (int j = 0; j < FM * FN; ++j) other[(kg - 1) * kAll + j * kWave] = acc[j / FN][j % FN];
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (kg > 0) continue;
#pragma unroll
      for (int j = 0; j < FM * FN; ++j)
#pragma unroll
        for (int v = 0; v < KG - 1; ++v) acc[j / FN][j % FN] += other[v * kAll + j * kWave];
    }
    const uint16_t* bias = p.bias;
    if constexpr (GROUPED) {
      if (bias) bias += int64_t(p.eids[p.block0 + list->block(row)]) * p.N;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      int64_t y;
      float wt = 1.0f;
      if constexpr (GROUPED) {
        const int2 pr = pairs[ring * BM + xrow + 16 * i];
        y = pr.x;
        wt = __int_as_float(pr.y);
      } else {
        y = int64_t(row) * BM + xrow + 16 * i;
        if (y >= p.M) y = -1;
      }
      if (y < 0) continue;
#pragma unroll
      for (int f = 0; f < FN; f += 2) {
        const int col = gated ? n0 + 8 * f + 4 * g : n0 + 16 * f + 8 * g;
        if (col >= p.No) continue;
        if (gated) {
          store(p, finish(p, acc[i][f], acc[i][f + 1], bias, y, col, wt), y, col);
        } else {
          store(p, finish(p, acc[i][f], acc[i][f], bias, y, col, wt), y, col);
          store(p, finish(p, acc[i][f + 1], acc[i][f + 1], bias, y, col + 4, wt), y, col + 4);
        }
      }
    }
  }
  // no load into LDS outlives its workgroup
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

// Columns of Y of a tile of `cols` columns of W.
int own_columns(const ProductParams& p, int cols) { return p.gated ? cols / 2 : cols; }
int column_tiles(const ProductParams& p, int cols) { return (p.No + own_columns(p, cols) - 1) / own_columns(p, cols); }

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KG = 1>
hipError_t tile_launch(ProductParams p, hipStream_t st) {
  using T = Tile<WM, WN, FM, FN, NS, KG>;
  const int ntiles = column_tiles(p, T::BN);
  const int64_t resident = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * T::groups(GROUPED);
  const int32_t all = GROUPED ? p.blocks : int32_t((p.M + T::BM - 1) / T::BM);
  const int32_t most = GROUPED ? kTileBlocks : all;
  for (p.block0 = 0; p.block0 < all; p.block0 += most) {
    p.blocks = std::min(most, all - p.block0);
    const int64_t grid = std::min(int64_t(p.blocks) * ntiles, resident);
    hipLaunchKernelGGL((gemm_tile_kernel<WM, WN, FM, FN, NS, GROUPED, KG>), dim3(unsigned(grid)),
                       dim3(T::NW * kWave), 0, st, p, ntiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Pieces of an align block that start at once: as many as an expert has on
// average, a block's workgroups take the others in turn (starting every piece
// would leave most workgroups to find padding).
template <int MT>
int64_t parts_of(const ProductParams& p) {
  const int64_t each = p.numel / (int64_t(p.E) * 12) + 1;
  return std::min<int64_t>(each, p.block_m / (16 * MT));
}

template <int MT, int NT, bool GROUPED>
int64_t rows_grid(const ProductParams& p) {
  const int64_t pieces = GROUPED ? p.blocks * parts_of<MT>(p) : (p.M + 16 * MT - 1) / (16 * MT);
  return pieces * column_tiles(p, 16 * NT);
}

// Whether one launch takes so many workgroups of the rows kernel: it has fewer
// than 2^32 threads.  (The tiles' workgroups go from tile to tile, any number.)
bool rows_fit(int64_t grid) { return grid < (int64_t(1) << 32) / (kSplit * kWave); }

template <int MT, int NT, bool GROUPED>
hipError_t rows_of(const ProductParams& p, hipStream_t st) {
  hipLaunchKernelGGL((gemm_rows_kernel<MT, NT, GROUPED>), dim3(unsigned(rows_grid<MT, NT, GROUPED>(p))),
                     dim3(kSplit * kWave), 0, st, p, column_tiles(p, 16 * NT),
                     GROUPED ? int(parts_of<MT>(p)) * 16 * MT : 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(ProductParams p, hipStream_t st) {
  const int64_t cus = int64_t(std::max(xcd_compute_units(), 1)) * kXcds;
  auto rounds = [&](int bm, int bn, int64_t at_once) {
    const int64_t tiles = (p.M + bm - 1) / bm * column_tiles(p, bn);
    return (tiles + at_once - 1) / at_once;
  };
  const bool once32 = rounds(32, 32, cus) == 1, once64 = rounds(64, 64, cus) == 1;
  const int64_t cost[5] = {once64 ? 30 : 50 * rounds(64, 64, 2 * cus), 43 * rounds(64, 128, cus),
                           63 * rounds(128, 128, cus), 98 * rounds(128, 256, cus),
                           175 * rounds(256, 256, cus)};
  const int best = int(std::min_element(cost, cost + 5) - cost);
  const int64_t groups = (p.N + 15) / 16, passes = (p.M + 31) / 32;
  const double mb = 2e-6 * p.N * p.K;
  const double by_rows = 1.8 + 1e-3 * p.K + std::max(mb * (p.M <= 16 ? 0.18 : 0.3 * double(passes)),
                                                     (p.M <= 16 ? 8e-4 : 1.6e-3) * double(groups * passes));
  const double by_32 = once32 ? 3.5 + 2.8e-3 * p.K : INFINITY;
  const double by_tile = 3 + 0.01 * p.KB * double(cost[best]);
  const bool wide = p.gated || groups > cus;
  const int64_t grid = p.M > 16 ? (p.gated ? rows_grid<2, 2, false>(p) : rows_grid<2, 1, false>(p))
                       : wide   ? rows_grid<1, 2, false>(p)
                                : rows_grid<1, 1, false>(p);
  if (by_rows < std::min(by_32, by_tile) && rows_fit(grid)) {
    if (p.M > 16) return p.gated ? rows_of<2, 2, false>(p, st) : rows_of<2, 1, false>(p, st);
    return wide ? rows_of<1, 2, false>(p, st) : rows_of<1, 1, false>(p, st);
  }
  if (by_32 < by_tile) return tile_launch<1, 1, 2, 2, 3, false, 4>(p, st);
  switch (best) {
    case 0: return tile_launch<2, 2, 2, 2, 4, false>(p, st);
    case 1: return tile_launch<2, 4, 2, 2, 4, false>(p, st);
    case 2: return tile_launch<2, 4, 4, 2, 2, false>(p, st);
    case 3: return tile_launch<2, 4, 4, 4, 2, false>(p, st);
    default: return tile_launch<2, 4, 8, 4, 2, false>(p, st);
  }
}

hipError_t launch_moe_gemm(ProductParams p, hipStream_t st) {
  const int64_t cus = int64_t(std::max(xcd_compute_units(), 1)) * kXcds;
  const int64_t E = p.E, used = std::min<int64_t>(p.numel, E);
  // tiles of `rows` rows
  auto tiles = [&](int rows) { return std::min<int64_t>(p.numel, std::max(used, p.numel / rows + E / 2)); };
  const double stream = 2.0 * p.N * p.K / 5.5e6;
  const double groups = double((p.N + 31) / 32);
  const double by_rows = 3 + double(tiles(16)) * std::max(stream, 0.004 * groups);
  const double by_tiles = 10 + std::max(0.45 * p.KB, 0.2 * p.KB + double(used) * stream);
  if (by_rows <= by_tiles && rows_fit(rows_grid<1, 2, true>(p))) {
    if (p.numel >= 3 * E && used * column_tiles(p, 64) >= cus) return rows_of<1, 4, true>(p, st);
    return rows_of<1, 2, true>(p, st);
  }
  const int64_t cols = column_tiles(p, 256);
  auto rounds = [&](int rows) { return (tiles(rows) * cols + cus - 1) / cus; };
  const int64_t cost64 = 80 * rounds(64), cost128 = 98 * rounds(128), cost256 = 140 * rounds(256);
  if (p.block_m <= 64 && cost64 <= cost128) return tile_launch<2, 4, 2, 4, 3, true>(p, st);
  if (p.numel <= 96 * E || cost128 <= cost256) return tile_launch<2, 4, 4, 4, 2, true>(p, st);
  return tile_launch<2, 4, 8, 4, 2, true>(p, st);
}

}  // namespace mlr
