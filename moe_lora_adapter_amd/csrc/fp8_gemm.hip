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
//
// The matrix core adds 8 products at a time, aligned to the largest with 13 bits
// below its exponent, and the eights in fp32; every sum outside it is fp32, and
// Y is rounded to bf16 once.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "dma.h"
#include "fp8.h"
#include "internal.h"
#include "tiles.h"

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

// One float; past the range it reads as zero.
__device__ __forceinline__ float buf_ld4(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_raw_buffer_load_b32(r, int(voff), 0, 0)));
}

// ---------------------------------------------------------------- few rows
// One workgroup computes 16 MT rows x 16 NT columns: its kSplit wavefronts take
// the K blocks w, w + kSplit, ... straight from memory (together they read kSplit x 128
// consecutive bytes of each row of W) and add their sums in LDS, in order.
// Bound by the stream of W: 20b-like decode w13 (64 pairs, 464 MB) 79 us, 5.9
// TB/s, with a wavefront's loads of one block ahead of its products; two blocks
// ahead 2 us more.  Grouped, the workgroups of a block take its pieces of 16 rows
// in steps of `step` rows.
constexpr int kSplit = 8;
template <int MT, int NT, bool GROUPED>
__global__ void __launch_bounds__(kSplit * kWave) fp8_gemm_rows_kernel(GemmParams p, int ntiles, uint32_t step) {
  __shared__ f32x4_t red[kSplit][MT * NT][kWave];
  const int tile = blockIdx.x % (p.S * ntiles);
  const int slice = tile / ntiles, n0 = (tile % ntiles) * 16 * NT;
  const int lane = lane_id(), w = wave_id(), a = lane & 15, g = lane >> 4;
  const uint32_t piece = blockIdx.x / (p.S * ntiles);
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
    // A block's workgroups are neighbours, and what lies behind the last block
    // comes last, when nothing waits for its place (8 experts of 512 x 1024, 96
    // rows each: 9.5 us; a block's first pieces, then all second ones, 11.1).
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

  const uint8_t* wbase = p.w + (e * p.S + slice) * p.Ns * int64_t(p.K);
  const auto wr = make_rsrc(wbase, uint32_t(p.Ns) * uint32_t(p.K));
  const float* wscale = p.ws + ((e * p.S + slice) * p.NB + n0 / kScaleBlock) * p.KB;
  // An offset is below 2 GiB or, for rows and columns that are not there, kOob;
  // so is an offset along K.  One of the two takes the sum out of range, which
  // reads as zero; both wrap to 0, and what is read there reaches no output.
  uint32_t woff[NT];
#pragma unroll
  for (int f = 0; f < NT; ++f) {
    const int n = n0 + 16 * f + a;
    woff[f] = n < p.Ns ? uint32_t(n) * uint32_t(p.K) + 16 * g : kOob;
  }
  for (;;) {
    // rows of X: dense tiles are addressed from their first row, grouped ones
    // from row 0 (X is below 2 GiB there)
    const int64_t x0 = GROUPED ? 0 : first;
    const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, 16 * MT);
    const auto xr = make_rsrc(p.x + x0 * p.K, uint32_t(xrows * p.K));
    const auto sr = make_rsrc(p.xs, uint32_t(p.rows * p.KB) * 4);
    uint32_t xoff[MT], soff[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const RowMap r = row_at(16 * i + a);
      xoff[i] = r.x_row >= 0 ? uint32_t((r.x_row - x0) * p.K) + 16 * g : kOob;
      soff[i] = r.x_row >= 0 ? uint32_t(r.x_row) * 4 : kOob;
    }

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NT; ++f) acc[i][f] = f32x4_t{0, 0, 0, 0};

    for (int kb = w; kb < p.KB; kb += kSplit) {
      const uint32_t k = uint32_t(kb) * kScaleBlock;
      const uint32_t lo = k + 16 * g < uint32_t(p.K) ? k : kOob;
      const uint32_t hi = k + 64 + 16 * g < uint32_t(p.K) ? k + 64 : kOob;
      const float sw = wscale[kb];
      i32x8_t wf[NT], xf[MT];
      float sx[MT];
#pragma unroll
      for (int f = 0; f < NT; ++f)
        wf[f] = join(buf_ld16(wr, woff[f] + lo, 0), buf_ld16(wr, woff[f] + hi, 0));
      // the columns' loads first, a line's two halves together (in any order: 128
      // experts of 2880 x 2880, 8 rows each, 213 us; so 196)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sx[i] = buf_ld4(sr, soff[i] + uint32_t(kb) * uint32_t(p.rows) * 4);
        xf[i] = join(buf_ld16(xr, xoff[i] + lo, 0), buf_ld16(xr, xoff[i] + hi, 0));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int f = 0; f < NT; ++f) {
          const f32x4_t d = mfma_e4m3(wf[f], xf[i]);
          const float sc = sx[i] * sw;
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[j], sc, acc[i][f][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int f = 0; f < NT; ++f) red[w][i * NT + f][lane] = acc[i][f];
    __syncthreads();
    for (int t = w; t < MT * NT; t += kSplit) {
      const int i = t / NT, f = t % NT;
      f32x4_t s = red[0][t][lane];
#pragma unroll
      for (int v = 1; v < kSplit; ++v) s += red[v][t][lane];
      const RowMap r = row_at(16 * i + a);
      const int n = n0 + 16 * f + 4 * g;
      if (r.y_row < 0 || n >= p.Ns) continue;
      if constexpr (GROUPED) {
        if (p.wt) s *= p.wt[r.y_row];
      }
      uint2 o = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
      *reinterpret_cast<uint2*>(p.y + r.y_row * (int64_t(p.S) * p.Ns) + slice * p.Ns + n) = o;
    }
    if constexpr (!GROUPED) return;
    at += step;
    if (!seek()) return;
    __syncthreads();  // the sums have been read
  }
}

// ---------------------------------------------------------------- many rows
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
//
// A stage's two operands are read from LDS by WN and WM wavefronts: at 128 x 64 a
// wavefront (256 x 256) that is 24 KiB for 32 MFMAs of 32 cycles, which LDS
// serves in half that time; 128 accumulators are what leaves registers for it.
// 4096 x 4096 x 12288: 180 us once the card's clock has settled (some 200 calls;
// 212 before), 2.29 PFLOP/s, the matrix cores 53 % busy at the 2.0 GHz of the run
// that counted.  Without the loads the same loop takes 141 us, the
// loads alone 89: what is between is stages whose loads take longer than their
// MFMAs, with two of them filling the LDS.
//
// KG > 1, for small tiles: a stage has KG blocks of 128, each of which WM x WN
// wavefronts multiply, and their sums meet in LDS.  A CU takes in some 64 KB a
// microsecond whatever its tile, so where there are few tiles they are small (64
// x 4096 x 4096: 32 x 32 with KG = 4 9.5 us, 64 x 64 with one block a stage 13.2,
// with two 13.8).
template <int WM, int WN, int FM, int FN, int NS, int KG = 1>
struct Tile {
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN * KG;
  static constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // 1 KiB loads a wavefront and K block
  static constexpr int kEach = XI + WI + 1, kLoads = KG * kEach;
  static constexpr int kSegs = (BM + kWave - 1) / kWave;  // loads of the rows' scales
  static constexpr int kX = 0, kW = BM * 128, kS = kW + BN * 128, kBlock = kS + kSegs * 256 + 256;
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
  static_assert(kSegs < NW && FM % 2 == 0 && FN % 2 == 0 && NS >= 2, "tile");
};

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KG>
__global__ void __launch_bounds__(WM * WN * KG * kWave, 2)
    fp8_gemm_tile_kernel(GemmParams p, int ntiles) {
  using T = Tile<WM, WN, FM, FN, NS, KG>;
  constexpr int BM = T::BM, BN = T::BN, XI = T::XI, WI = T::WI, kLoads = T::kLoads;
  // whether the columns' loads run ahead of the rows' (below)
  constexpr bool kEarly = FM > 2;
  static_assert(KG == 1 || (!GROUPED && !kEarly), "a stage of several K blocks");
  constexpr int kX = T::kX, kW = T::kW, kS = T::kS, kStage = T::kStage;
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
  const Items<GROUPED ? 1 : 4> items(row_tiles, uint32_t(p.S) * ntiles);
  const int lane = lane_id(), w = wave_id(), kg = w / (WM * WN), wm = w / WN % WM, wn = w % WN;
  const int a = lane & 15, g = lane >> 4;
  const int rl = lane >> 3, cl = lane & 7;  // row within a load, chunk as stored
  auto swizzle = [](int r) { return (r & 3) | ((r >> 1) & 4); };  // bits 0, 1, 3

  // ---- the loading side: its tile, and how far it is
  uint32_t lt = items.first + blockIdx.x / kXcds;
  uint32_t ct = lt;  // the tile being multiplied
  if (lt >= items.end) return;
  int lkb = 0, lstage = 0, lring = 0;
  i32x4_t wr, xr, sr;
  // A load takes 8 rows, 8 chunks of each.  Dense rows and the columns follow
  // each other, and what is behind the last one is behind the resource's range;
  // grouped rows lie anywhere: lane i keeps the offset of this wavefront's row
  // i.  The columns' chunk order has two forms, by bit 3 of the column.
  const int xc = 16 * (cl ^ rl), wc = 16 * (cl ^ swizzle(rl));
  uint32_t xoff, woff, woff1, soff;
  constexpr int kSegs = T::kSegs, kCols = (BN + kScaleBlock - 1) / kScaleBlock;
  const int sdst = kS + 256 * std::min(w, kSegs);
  const uint32_t sstride = w < kSegs ? uint32_t(p.rows) * 4 : 4;
  const uint32_t step8 = 8 * uint32_t(p.K);
  const uint32_t base = lds_address(lds);
  int2* pairs = reinterpret_cast<int2*>(lds + T::kPairs);

  auto set_tile = [&]() {
    uint32_t nx = kOob, nw = kOob, nw1 = kOob, ns = kOob;  // nothing left: loads from nowhere
    if (lt < items.end) {
      // not to be computed once and kept: the registers are needed
      int ln = lane;
      asm volatile("" : "+v"(ln));
      uint32_t row, tile;
      items.at(lt, &row, &tile);
      const int slice = tile / ntiles, n0 = (tile % ntiles) * BN;
      int64_t first = int64_t(row) * BM, mat = slice;
      const int32_t* eids = p.eids + p.block0;
      int blk = 0, e = 0;
      if constexpr (GROUPED) {
        blk = list->block(row);
        e = eids[blk];
        first = int64_t(p.block0 + blk) * p.block_m;
        mat += int64_t(e) * p.S;
      }
      // row i of the tile; a grouped tile ends where its expert does
      auto row_at = [&](int i) {
        if constexpr (GROUPED) {
          const int b = blk + i / p.block_m;
          if (b >= blocks || eids[b] != e) return RowMap{-1, -1};
        }
        return row_of<GROUPED>(p, first, i);
      };
      wr = dma_rsrc(p.w + mat * p.Ns * int64_t(p.K), uint32_t(p.Ns) * uint32_t(p.K));
      const int64_t x0 = GROUPED ? 0 : first;
      const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, BM);
      xr = dma_rsrc(p.x + x0 * p.K, uint32_t(xrows * p.K));
      if constexpr (GROUPED) {
        const RowMap m = row_at(8 * w * XI + ln % (8 * XI));
        if (m.x_row >= 0) nx = uint32_t(m.x_row * p.K);
      } else {
        nx = uint32_t(8 * w * XI + (ln >> 3)) * uint32_t(p.K) + xc;
      }
      nw = uint32_t(n0 + 8 * w * WI + (ln >> 3)) * uint32_t(p.K);
      nw1 = nw + (wc ^ 64);
      nw += wc;
      // The stage's scales: the first wavefronts load those of 64 rows each,
      // the others (all alike) those of the tile's column blocks.
      const float* from = w < kSegs ? p.xs + x0 : p.ws + mat * p.NB * p.KB;
      const int64_t count = w < kSegs ? (p.KB - 1) * p.rows + xrows : int64_t(p.NB) * p.KB;
      sr = dma_rsrc(from, uint32_t(count * 4));
      if (w < kSegs) {
        const RowMap m = row_at(w * kWave + ln);
        if (m.x_row >= 0) ns = uint32_t((m.x_row - x0) * 4);
        if constexpr (GROUPED) {
          const float wt = p.wt && m.y_row >= 0 ? p.wt[m.y_row] : 1.0f;
          pairs[lring * BM + w * kWave + ln] = make_int2(int32_t(m.y_row), __float_as_int(wt));
        }
      } else {
        const int nb = n0 / kScaleBlock + ln;
        if (ln < kCols && nb < p.NB) ns = uint32_t(nb) * uint32_t(p.KB) * 4;
      }
    }
    xoff = nx;
    woff = nw;
    woff1 = nw1;
    soff = ns;
  };
  // One of a stage's loads.  Chunks past K in a short last block read as
  // zeros; behind the last tile everything does, so that every stage counts the
  // same loads.
  auto load = [&](int l) {
    const int kb = KG == 1 ? lkb : lkb * KG + l / T::kEach;
    const uint32_t st = base + uint32_t(lstage) * kStage + uint32_t(l / T::kEach * T::kBlock);
    l %= T::kEach;
    const int have = p.K - kb * kScaleBlock;
    const uint32_t k = uint32_t(kb) * kScaleBlock;
    if (l < XI) {
      const uint32_t o = GROUPED ? __builtin_amdgcn_ds_bpermute(4 * (8 * l + rl), xoff) + xc
                                 : xoff + uint32_t(l) * step8;
      tile_dma16(xr, st + kX + 1024 * (w * XI + l), xc < have ? o : kOob, k);
    } else if (l < XI + WI) {
      const int i = l - XI;
      const int flip = 16 * swizzle(8 * (w * WI + i));
      tile_dma16(wr, st + kW + 1024 * (w * WI + i),
                 (wc ^ flip) < have ? (flip ? woff1 : woff) + uint32_t(i) * step8 : kOob, k);
    } else {
      // (a stage's second block may be past K: its scales are zeros, too)
      const bool in = KG == 1 || kb < p.KB;
      tile_dma4(sr, st + sdst, in ? soff : kOob, uint32_t(in ? kb : 0) * sstride);
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
  const int so = ko + kS + kSegs * 256 + wn * FN * 16 / kScaleBlock * 4;  // this wavefront's column block
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
  int young = 0;  // stages still waited for whose loads are older than the last tile's stores
  for (; ct < items.end; ct += items.step, ring = ring + 1 == T::kRing ? 0 : ring + 1) {
    uint32_t row, tile;
    items.at(ct, &row, &tile);
    const int slice = tile / ntiles, n0 = (tile % ntiles) * BN;
    // A wavefront without a row or a column of the tile only loads and keeps the
    // barriers.
    bool none = n0 + wn * FN * 16 >= p.Ns;
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
          if (!kEarly || l < XI || l == kLoads - 1) load(l);
        loaded();
        stage = stage + 1 == NS ? 0 : stage + 1;
        if (lkb == stages) next_loads();
      }
      if constexpr (KG > 1) asm volatile("s_barrier" ::: "memory");  // of the sums
      young = 0;
      continue;
    }

    // A stage is FM steps of FN MFMAs: a step reads the next one's rows, and a
    // result's multiply-adds run FN MFMAs after it.  The stage's barrier stands
    // before the last step, once every wavefront has its last rows of the stage
    // in registers; behind it the stage's buffer is refilled, and each column
    // operand is replaced by the next stage's after its last use.  With more
    // than two steps a second barrier, behind the first step, says that every
    // wavefront has the stage's columns in registers, and their buffer is
    // refilled from there on (4096 x 4096 x 12288: 190 us without, 187 with;
    // 8192^3 478 and 467).  The scheduling barriers keep the compiler from
    // undoing this order.
    f32x4_t acc[FM][FN], d[FN];
    i32x8_t wf[FN], xf[2];
    float sx[2], sd = 0.0f, sw;
    auto add = [&](int i, int f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][f][j] = fmaf(d[f][j], sd, acc[i][f][j]);
    };
    auto columns = [&](const uint8_t* st, int f) {
      const int o = 4096 * (f >> 1) + 512 * (f & 1);
      wf[f] = join(*reinterpret_cast<const uint4*>(st + wo + o),
                   *reinterpret_cast<const uint4*>(st + (wo ^ 64) + o));
    };
    auto rows = [&](const uint8_t* st, int i) {
      xf[i & 1] = join(*reinterpret_cast<const uint4*>(st + xo + 2048 * i),
                       *reinterpret_cast<const uint4*>(st + (xo ^ 64) + 2048 * i));
      sx[i & 1] = *reinterpret_cast<const float*>(st + ko + kS + 4 * (xrow + 16 * i));
    };
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      columns(lds + stage * kStage, f);
      d[f] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i][f] = f32x4_t{0, 0, 0, 0};
    }
    rows(lds + stage * kStage, 0);
    sw = *reinterpret_cast<const float*>(lds + stage * kStage + so);
    for (int kb = 0; kb < stages;) {
      // the stages until the loads change their tile
      const int n = std::min(stages - kb, stages - lkb);
      for (int r = 0; r < n; ++r) {
        const uint8_t* st = lds + stage * kStage;
        stage = stage + 1 == NS ? 0 : stage + 1;
        const uint8_t* nx = lds + stage * kStage;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const float s = sx[i & 1] * sw;
          if (kEarly && i == 1) asm volatile("s_barrier" ::: "memory");
          if (i < FM - 1) {
            rows(st, i + 1);
          } else {
            if constexpr (kEarly) {
              ring_barrier<kWait, FM * FN / 2>(__builtin_amdgcn_readfirstlane(young));
              young = std::max(young - 1, 0);
            } else {
              stage_barrier<kWait>();
            }
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
              for (int l = kLoads * f / FN; l < kLoads * (f + 1) / FN; ++l)
                if (!kEarly || l < XI || l == kLoads - 1) load(l);
            }
            if (kEarly && i >= 1 && i < FM - 1) {
              constexpr int kSlots = kEarly ? (FM - 2) * FN : 1;
              const int slot = (i - 1) * FN + f;
#pragma unroll
              for (int l = WI * slot / kSlots; l < WI * (slot + 1) / kSlots; ++l) load(XI + l);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          sd = s;
        }
        loaded();
      }
      kb += n;
      if (lkb == stages) next_loads();
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) add(FM - 1, f);

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
    const int nl = n0 + wn * FN * 16 + 8 * g;  // this lane's columns: 8 of each 32
    int stores = 0;  // of this wavefront
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
      uint16_t* out = p.y + y * (int64_t(p.S) * p.Ns) + int64_t(slice) * p.Ns + nl;
#pragma unroll
      for (int f = 0; f < FN; f += 2) {
        const f32x4_t u = acc[i][f] * wt, v = acc[i][f + 1] * wt;
        const bool in = y >= 0 && nl + 16 * f < p.Ns;
        stores += __ballot(in) != 0;
        if (in)
          *reinterpret_cast<uint4*>(out + 16 * f) =
              make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]),
                         pack_bf16x2(v[2], v[3]));
      }
    }
    young = stores == FM * FN / 2 ? NS - 1 : 0;
  }
  // no load into LDS outlives its workgroup
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KG = 1>
hipError_t tile_launch(GemmParams p, hipStream_t st) {
  using T = Tile<WM, WN, FM, FN, NS, KG>;
  const int ntiles = (p.Ns + T::BN - 1) / T::BN;
  const int64_t resident = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * T::groups(GROUPED);
  const int32_t all = GROUPED ? p.blocks : int32_t((p.M + T::BM - 1) / T::BM);
  const int32_t most = GROUPED ? kTileBlocks : all;
  for (p.block0 = 0; p.block0 < all; p.block0 += most) {
    p.blocks = std::min(most, all - p.block0);
    const int64_t grid = std::min(int64_t(p.blocks) * p.S * ntiles, resident);
    hipLaunchKernelGGL((fp8_gemm_tile_kernel<WM, WN, FM, FN, NS, GROUPED, KG>), dim3(unsigned(grid)),
                       dim3(T::NW * kWave), 0, st, p, ntiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Pieces of an align block that start at once: as many as an expert has on
// average, a block's workgroups take the others in turn.  Starting every piece
// would leave most workgroups to find padding: 64 experts of 256 x 512, 8 rows
// each in blocks of 64, 8.5 us, so 4.9; 8 of 2048 x 4096 29.3 and 17.2.
template <int MT>
int64_t parts_of(const GemmParams& p) {
  const int64_t each = p.numel / (int64_t(p.E) * 12) + 1;
  return std::min<int64_t>(each, p.block_m / (16 * MT));
}

template <int MT, int NT, bool GROUPED>
int64_t rows_grid(const GemmParams& p) {
  const int64_t pieces = GROUPED ? p.blocks * parts_of<MT>(p) : (p.M + 16 * MT - 1) / (16 * MT);
  return pieces * p.S * ((p.Ns + 16 * NT - 1) / (16 * NT));
}

// Whether one launch takes so many workgroups of the rows kernel: it has fewer
// than 2^32 threads.  (The tiles' workgroups go from tile to tile, any number.)
bool rows_fit(int64_t grid) { return grid < (int64_t(1) << 32) / (kSplit * kWave); }

template <int MT, int NT, bool GROUPED>
hipError_t rows_of(const GemmParams& p, hipStream_t st) {
  const int ntiles = (p.Ns + 16 * NT - 1) / (16 * NT);
  const int64_t grid = rows_grid<MT, NT, GROUPED>(p);
  hipLaunchKernelGGL((fp8_gemm_rows_kernel<MT, NT, GROUPED>), dim3(unsigned(grid)),
                     dim3(kSplit * kWave), 0, st, p, ntiles, GROUPED ? int(parts_of<MT>(p)) * 16 * MT : 0);
  return hipGetLastError();
}

}  // namespace

// Estimates in microseconds.  The tiles above 32 x 32: 3 us, and for each 128 of K
// the hundredths that a round over the device takes (measured at K = 4096 with
// every CU busy: 64 x 64 30, or 50 with two on a CU; 64 x 128 43; 128 x 128 63; 128 x
// 256 98; 256 x 256 175).  The 32 x 32 tile, where there is a CU for each.  Few rows
// or columns straight from memory: all of W for every 32 rows, or 1.6 ns a
// workgroup.
//
// Measured, with W from memory, not from the cache in front of it, straight, 32 x
// 32 and 64 x 64: 16 rows of 4096 x 4096 6.9, 8.9 and 11.6 us, of 8192 x 8192 16.5,
// 15.4 and 21.5; 32 rows of 4096 x 4096 8.8, 9.4 and 11.8, of 4096 x 7840 14.5, 10.6
// and 12.8; 64 rows of 4096 x 4096 14.3, 9.5 and 13.2, of 4096 x 12288 36, 22 and
// 16; 100 of 8192 x 2048 24.6, 13.5 and 22.1; 482 of 32 x 3512 7.5, - and 4.5; 1463
// of 4016 x 32 6.3, - and 10.5.
hipError_t launch_fp8_gemm(GemmParams p, hipStream_t st) {
  const int64_t cus = int64_t(std::max(xcd_compute_units(), 1)) * kXcds;
  auto rounds = [&](int bm, int bn, int64_t at_once) {
    const int64_t tiles = (p.M + bm - 1) / bm * p.S * ((p.Ns + bn - 1) / bn);
    return (tiles + at_once - 1) / at_once;
  };
  const bool once32 = rounds(32, 32, cus) == 1, once64 = rounds(64, 64, cus) == 1;
  const int64_t cost[5] = {once64 ? 30 : 50 * rounds(64, 64, 2 * cus), 43 * rounds(64, 128, cus),
                           63 * rounds(128, 128, cus), 98 * rounds(128, 256, cus),
                           175 * rounds(256, 256, cus)};
  const int best = int(std::min_element(cost, cost + 5) - cost);
  const int64_t groups = int64_t(p.S) * ((p.Ns + 15) / 16), passes = (p.M + 31) / 32;
  const double mb = 1e-6 * p.S * p.Ns * p.K;
  const double by_rows = 1.8 + 5e-4 * p.K + std::max(mb * (p.M <= 16 ? 0.18 : 0.3 * double(passes)),
                                                     (p.M <= 16 ? 8e-4 : 1.6e-3) * double(groups * passes));
  const double by_32 = once32 ? 3.5 + 1.4e-3 * p.K : INFINITY;
  const double by_tile = 3 + 0.01 * p.KB * double(cost[best]);
  const int64_t grid = p.M > 16         ? rows_grid<2, 1, false>(p)
                       : groups <= cus ? rows_grid<1, 1, false>(p)
                                       : rows_grid<1, 2, false>(p);
  if (by_rows < std::min(by_32, by_tile) && rows_fit(grid)) {
    // (16 rows: up to a CU's worth of groups of 16 columns 6.1 us, in 32s 7.8, 4096
    // x 4096; beyond, 2880 x 5120, 6.0 and 4.9)
    if (p.M > 16) return rows_of<2, 1, false>(p, st);
    return groups <= cus ? rows_of<1, 1, false>(p, st) : rows_of<1, 2, false>(p, st);
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

// Estimates in microseconds, with the pairs spread evenly: `stream`, one expert's
// weights at 5.5 TB/s.  The rows kernel takes 3 us, and for each piece of 16 rows
// those weights or 4 ns a workgroup; the tiles take 10 us, of which most is
// finding them, and each expert's weights once, or, with few of them, the
// latency of their K.  Measured with W from memory, rows and tiles: 8 experts of
// 512 x 1024, 8 rows each, 4.5 and 12.1, 96 rows 9.6 and 13.6; 8 of 2048 x 4096,
// 8 rows 17.2 and 31.8, 48 rows 40 and 36; 128 of 2880 x 2880, 4 rows 178 and 193,
// 8 rows 197 and 201, 16 rows 260 and 210.  Routing that leaves most pairs to few
// experts is not seen: the rows kernel then reads their weights once for every 16
// rows, whatever the tiles would take.
hipError_t launch_fp8_moe_gemm(GemmParams p, hipStream_t st) {
  const int64_t cus = int64_t(std::max(xcd_compute_units(), 1)) * kXcds;
  const int64_t E = p.E, used = std::min<int64_t>(p.numel, E);
  // tiles of `rows` rows
  auto tiles = [&](int rows) { return std::min<int64_t>(p.numel, std::max(used, p.numel / rows + E / 2)); };
  const double stream = double(p.S) * p.Ns * p.K / 5.5e6;
  const double groups = double(p.S) * ((p.Ns + 31) / 32);
  const double by_rows = 3 + double(tiles(16)) * std::max(stream, 0.004 * groups);
  const double by_tiles = 10 + std::max(0.45 * p.KB, 0.2 * p.KB + double(used) * stream);
  if (by_rows <= by_tiles && rows_fit(rows_grid<1, 2, true>(p))) {
    // 64 columns a workgroup read X half as often as 32, which is worth it from a
    // few rows an expert on and with a workgroup for every CU (64 experts of 1024
    // x 4096: 1 row each 38.0 us and 35.6, 8 rows 56.0 and 53.4; 128 of 2880 x
    // 2880, 4 rows 178 and 182, 8 rows 197 and 214; 8 of 512 x 1024, 8 rows 5.4
    // and 4.5)
    if (p.numel >= 3 * E && used * p.S * ((p.Ns + 63) / 64) >= cus) return rows_of<1, 4, true>(p, st);
    return rows_of<1, 2, true>(p, st);
  }
  // The tile whose rounds over the device cost least, the largest only with enough
  // rows to fill it whatever the routing.  (64 x 256, 128 x 256 and 256 x 256) 128
  // experts of 1536 x 2048: 32 rows each 82, 83 and 87 us, 64 rows 106, 91 and
  // 95, 128 rows 132, 122 and 112; of 2880 x 2880, 128 rows 408, 319 and 298; 16 of
  // 2048 x 4096: 96 rows 45, 50 and 52, 192 rows 68, 51 and 63, 256 rows 87, 82
  // and 68; skewed routing over 64 of 1024 x 1024, 96 rows: 30, 30 and 39.
  const int64_t cols = p.S * ((p.Ns + 255) / 256);
  auto rounds = [&](int rows) { return (tiles(rows) * cols + cus - 1) / cus; };
  const int64_t cost64 = 80 * rounds(64), cost128 = 98 * rounds(128), cost256 = 140 * rounds(256);
  if (p.block_m <= 64 && cost64 <= cost128) return tile_launch<2, 4, 2, 4, 3, true>(p, st);
  if (p.numel <= 96 * E || cost128 <= cost256) return tile_launch<2, 4, 4, 4, 2, true>(p, st);
  return tile_launch<2, 4, 8, 4, 2, true>(p, st);
}

}  // namespace mlr
