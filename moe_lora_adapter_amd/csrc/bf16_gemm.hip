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
#include <utility>

#include "base.h"
#include "common.h"
#include "dma.h"
#include "internal.h"
#include "tiles.h"

namespace mlr {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));


// f(0), f(1), ..., f(N - 1) with constants as arguments: arrays that only constants
// index are registers, however much code there is (a loop that is unrolled late
// leaves them in memory).
template <class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}

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

__device__ __forceinline__ f32x4_t silu(f32x4_t v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= sigmoid(v[j]);
  return v;
}
// (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
__device__ __forceinline__ f32x4_t gelu_tanh(f32x4_t v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= sigmoid(1.5957691216057308f * (v[j] + 0.044715f * v[j] * v[j] * v[j]));
  return v;
}
// (the clamps keep NaN)
__device__ __forceinline__ f32x4_t swiglu_clamp(f32x4_t g, f32x4_t u) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = g[j] > 7.0f ? 7.0f : g[j];
    const float b = u[j] > 7.0f ? 7.0f : (u[j] < -7.0f ? -7.0f : u[j]);
    g[j] = a * sigmoid(1.702f * a) * (b + 1.0f);
  }
  return g;
}
__device__ __forceinline__ f32x4_t activate(f32x4_t v, f32x4_t u, int act) {
  switch (act) {
    case kActSilu: return silu(v);
    case kActGeluTanh: return gelu_tanh(v);
    case kActSiluMul: return silu(v) * u;
    case kActSwigluClamp: return swiglu_clamp(v, u);
    default: return v;
  }
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
  v = activate(v, u, p.act);
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

// The same for a wavefront's part of a tile, one step of the epilogue after the
// other over all of it.  at(i) is the row of Y or -1, wt(i) its weight, `col` the
// first column of this lane; acc[i][f] and acc[i][f + 1] are columns col + 16 f ..
// + 7, or, gated, gate and up of columns col + 8 f .. + 3.  Operands are read at a
// place that is there, whether or not the row and the column are, and only stores
// are left out; the loads of kAtOnce rows are in flight together.
template <int FM, int FN, bool GROUPED, class At, class Weight>
__device__ __forceinline__ void finish_tile(const ProductParams& p, f32x4_t (&acc)[FM][FN], At at, Weight wt,
                                            const uint16_t* bias, int col) {
  constexpr int kAtOnce = FM < 4 ? FM : FN > 2 ? 2 : 4;
  static_assert(FM % kAtOnce == 0, "rows");
  const bool gated = p.gated;
  const int wide = gated ? 8 : 16;
  // a pair of sums' eight values of an operand whose rows have gate and up
  auto eight = [&](const uint16_t* from, int f) {
    const uint16_t* a = from + min(col + wide * f, p.No - (gated ? 4 : 8));
    if (!gated) return *reinterpret_cast<const uint4*>(a);
    const uint2 g = *reinterpret_cast<const uint2*>(a), u = *reinterpret_cast<const uint2*>(a + p.No);
    return make_uint4(g.x, g.y, u.x, u.y);
  };
  auto four = [&](const uint16_t* from, int f) {  // of one whose rows have not
    const uint16_t* a = from + min(col + wide * f, p.No - (gated ? 4 : 8));
    if (!gated) return *reinterpret_cast<const uint4*>(a);
    const uint2 g = *reinterpret_cast<const uint2*>(a);
    return make_uint4(g.x, g.y, 0, 0);
  };
  if (bias) {
    each<FN / 2>([&](auto h) {
      constexpr int f = 2 * h;
      const uint4 b = eight(bias, f);
      const f32x4_t lo = widen(make_uint2(b.x, b.y)), hi = widen(make_uint2(b.z, b.w));
      each<FM>([&](auto i) { acc[i][f] += lo, acc[i][f + 1] += hi; });
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  if constexpr (GROUPED) {
    if (p.wt)
      each<FM>([&](auto i) {
        const float w = wt(i);
        each<FN>([&](auto f) { acc[i][f] *= w; });
      });
  }
  // adds an operand, read by `get`
  auto add = [&](const uint16_t* from, int width, auto get) {
    asm volatile("" : "+v"(col));  // addresses are not to be kept: the registers are needed
    each<FM / kAtOnce>([&](auto part) {
      constexpr int i0 = part * kAtOnce;
      uint4 d[kAtOnce][FN / 2];
      each<kAtOnce>([&](auto i) {
        const uint16_t* line = from + max(at(i0 + i), int64_t(0)) * width;
        each<FN / 2>([&](auto h) { d[i][h] = get(line, 2 * h); });
      });
      each<kAtOnce>([&](auto i) {
        each<FN / 2>([&](auto h) {
          acc[i0 + i][2 * h] += widen(make_uint2(d[i][h].x, d[i][h].y));
          acc[i0 + i][2 * h + 1] += widen(make_uint2(d[i][h].z, d[i][h].w));
        });
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  if (p.delta) add(p.delta, p.N, eight);
  // without an activation the residual is a second delta
  const bool late = !GROUPED && p.residual && p.act != kActNone;
  if constexpr (!GROUPED) {
    if (p.residual && !late) add(p.residual, p.No, four);
  }
  asm volatile("" : "+v"(col));
  each<FM>([&](auto i) {
    __builtin_amdgcn_sched_barrier(0);
    const int64_t m = at(i);
    each<FN / 2>([&](auto h) {
      const int n = col + wide * 2 * h;
      if (m < 0 || n >= p.No) return;
      f32x4_t v = acc[i][2 * h], u = acc[i][2 * h + 1];
      const int64_t to = m * p.No + n;
      if (gated) {
        v = activate(v, u, p.act);
      } else if (p.act != kActNone) {
        v = activate(v, u, p.act);
        u = activate(u, u, p.act);
      }
      if (late) {
        const uint4 r = four(p.residual + m * p.No, 2 * h);
        v += widen(make_uint2(r.x, r.y));
        u += widen(make_uint2(r.z, r.w));
      }
      if (p.out32) {
        float* y = static_cast<float*>(p.y) + to;
        *reinterpret_cast<f32x4_t*>(y) = v;
        if (!gated) *reinterpret_cast<f32x4_t*>(y + 4) = u;
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.y) + to;
        const uint2 lo = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        if (gated)
          *reinterpret_cast<uint2*>(y) = lo;
        else
          *reinterpret_cast<uint4*>(y) = make_uint4(lo.x, lo.y, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
      }
    });
  });
}

// ---------------------------------------------------------------- few rows
// One workgroup computes 16 rows x 16 NT columns of W: its kSplit wavefronts
// take the stages w, w + kSplit, ... of K straight from memory and add their sums
// in LDS, in order.  Bound by the stream of W: 20b-like decode w13 (64 pairs, 940
// MB) 167 us, 5.6 TB/s, 120b-like decode w2 79 us, 6.0; more stages in flight a
// wavefront are slower there (two 184 us) and no faster where a CU has one
// workgroup (1 row of 4096 x 4096: 8.4 us, two 9.9, four 9.3).  Gated, the even
// groups of 16 columns are gate's and the odd ones the same of up.  Grouped, the
// workgroups of a block take its pieces of 16 rows in steps of `step` rows.
constexpr int kSplit = 8;
template <int NT, bool GROUPED>
__global__ void __launch_bounds__(kSplit * kWave) gemm_rows_kernel(ProductParams p, int ntiles, uint32_t step) {
  __shared__ f32x4_t red[kSplit][NT][kWave];
  const int tile = blockIdx.x % ntiles;
  const int lane = lane_id(), w = wave_id(), a = lane & 15, g = lane >> 4;
  const uint32_t piece = blockIdx.x / ntiles;
  const int64_t first = int64_t(piece) * 16;  // dense: the first row
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
      if ((at < kWave ? held0 : held1) >> (at % kWave) & 0xffff) return true;
    return false;
  };
  // this lane's row of the piece
  auto row_here = [&]() {
    if constexpr (GROUPED)
      return row_of_pair(p, uint32_t(__shfl(at < kWave ? id0 : id1, at % kWave + a)));
    else
      return row_of<false>(p, first, a);
  };
  if constexpr (GROUPED) {
    // a block's workgroups are neighbours; what lies behind the last block comes last
    const uint32_t parts = step / 16, block = piece / parts;
    at = piece % parts * 16;
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
    const int64_t xrows = GROUPED ? p.rows : std::min<int64_t>(p.rows - first, 16);
    const auto xr = make_rsrc(p.x + x0 * p.K, uint32_t(xrows * K2));
    const int64_t x_row = row_here().x_row;
    const uint32_t xoff = x_row >= 0 ? uint32_t((x_row - x0) * K2) + 16 * g : kOob;

    f32x4_t acc[NT];
#pragma unroll
    for (int f = 0; f < NT; ++f) acc[f] = f32x4_t{0, 0, 0, 0};

    for (int kb = w; kb < p.KB; kb += kSplit) {
      const uint32_t k = uint32_t(kb) * (2 * kStageK);
      const uint32_t lo = k + 16 * g < K2 ? k : kOob;
      const uint32_t hi = k + 64 + 16 * g < K2 ? k + 64 : kOob;
      uint4 wl[NT], wh[NT];
#pragma unroll
      for (int f = 0; f < NT; ++f) {
        wl[f] = buf_ld16(wr, woff[f] + lo, 0);
        wh[f] = buf_ld16(wr, woff[f] + hi, 0);
      }
      __builtin_amdgcn_sched_barrier(0);  // the columns' loads first, a line's two halves together
      const uint4 xl = buf_ld16(xr, xoff + lo, 0), xh = buf_ld16(xr, xoff + hi, 0);
#pragma unroll
      for (int f = 0; f < NT; ++f) {
        acc[f] = mfma_bf16(wl[f], xl, acc[f]);
        acc[f] = mfma_bf16(wh[f], xh, acc[f]);
      }
    }
#pragma unroll
    for (int f = 0; f < NT; ++f) red[w][f][lane] = acc[f];
    __syncthreads();
    const uint16_t* bias = p.bias ? p.bias + e * p.N : nullptr;
#pragma unroll
    for (int f = 0; f < NT; ++f) {
      // gated, the wavefront of the even group takes both
      if (f % kSplit != w || (p.gated && (f & 1))) continue;
      auto sum = [&](int f) {
        f32x4_t s = red[0][f][lane];
#pragma unroll
        for (int v = 1; v < kSplit; ++v) s += red[v][f][lane];
        return s;
      };
      const RowMap r = row_here();
      const f32x4_t s = sum(f);
      f32x4_t u = {0, 0, 0, 0};
      if (NT > 1 && p.gated) u = sum(NT > 1 ? f + 1 : f);
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
// Large products are bound by the card's power and by this loop: 4096 x 4096 x
// 12288 takes 289 to 300 us (1.37 to 1.43 PFLOP/s), the matrix cores 68 % busy at
// 1.94 GHz.  Matrix instructions alone, on random operands in registers, reach 1.97
// PFLOP/s at 2.1 GHz; this loop without its loads, on zeros, takes 217 us at 2.45
// GHz.  No LDS bank conflicts.  A 128 x 64 tile a wavefront reads 192 KB of LDS a
// stage; 128 x 128 with four wavefronts reads 128 KB and was no faster.
//
// KS > 1: a stage has KS blocks of 64, which share its barrier.  KG > 1, for few
// tiles: KG groups of WM x WN wavefronts multiply a block each, and their sums meet
// in LDS.
template <int WM, int WN, int FM, int FN, int NS, int KS = 1, int KG = 1>
struct Tile {
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN * KG;
  static constexpr int XI = BM / 8 / NW, WI = BN / 8 / NW;  // 1 KiB loads a wavefront and K block
  static constexpr int kEach = XI + WI, kLoads = KS * KG * kEach;
  static constexpr int kX = 0, kW = BM * 128, kBlock = kW + BN * 128;
  static constexpr int kStage = KS * KG * kBlock;
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

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KS, int KG>
__global__ void __launch_bounds__(WM * WN * KG * kWave, 2)
    gemm_tile_kernel(ProductParams p, int ntiles) {
  using T = Tile<WM, WN, FM, FN, NS, KS, KG>;
  constexpr int BM = T::BM, BN = T::BN, XI = T::XI, WI = T::WI, kLoads = T::kLoads;
  constexpr bool kPhases = KS == 1;  // (below)
  static_assert(!GROUPED || KS * KG == 1, "a stage of several K blocks");
  constexpr int kX = T::kX, kW = T::kW, kStage = T::kStage;
  const int stages = (p.KB + KS * KG - 1) / (KS * KG);  // of a tile
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
  uint32_t xoff[XI], woff[WI];  // of each of a block's loads
  auto chunk_flip = [&](int l) { return 16 * swizzle(8 * (w * WI + l)); };  // of a load of columns
  const uint32_t xstep = 8 * K2, wstep = gated ? 4 * K2 : 8 * K2;
  const uint32_t base = lds_address(lds);
  int2* pairs = reinterpret_cast<int2*>(lds + T::kPairs);

  auto set_tile = [&]() {
    uint32_t nx = kOob, nw = kOob;  // nothing left: loads from nowhere
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
    }
    each<XI>([&](auto l) {
      xoff[l] = GROUPED ? __builtin_amdgcn_ds_bpermute(4 * (8 * l + rl), nx) + xc : nx + uint32_t(l) * xstep;
    });
    each<WI>([&](auto l) { woff[l] = nw + uint32_t(l) * wstep + (wc ^ chunk_flip(l)); });
  };
  // One of a stage's loads.  Chunks past K in a short last block read as
  // zeros; behind the last tile everything does, so that every stage counts the
  // same loads.
  auto load = [&](auto at) {
    constexpr int block = at / T::kEach, l = at % T::kEach;
    const int kb = lkb * (KS * KG) + block;
    const uint32_t st = base + uint32_t(lstage) * kStage + uint32_t(block * T::kBlock);
    // (a stage's later blocks may be past K)
    const uint32_t k = KS * KG == 1 || kb < p.KB ? uint32_t(kb) * (2 * kStageK) : 0;
    const int have = KS * KG == 1 || kb < p.KB ? int(K2 - k) : 0;
    if constexpr (l < XI)
      tile_dma16(xr, st + kX + 1024 * (w * XI + l), xc < have ? xoff[l] : kOob, k);
    else
      tile_dma16(wr, st + kW + 1024 * (w * WI + l - XI), (wc ^ chunk_flip(l - XI)) < have ? woff[l - XI] : kOob, k);
  };
  constexpr int kXLoads = KS * KG * XI, kWLoads = KS * KG * WI;
  // (with phases a stage's columns are loaded before its rows)
  auto load_x = [&](auto q) { load(std::integral_constant<int, q / XI * T::kEach + q % XI>{}); };
  auto load_w = [&](auto q) { load(std::integral_constant<int, q / WI * T::kEach + XI + q % WI>{}); };
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
  constexpr int kWait = (NS - 2) * kLoads;  // younger loads at a stage's barrier

  set_tile();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    each<kWLoads>(load_w);
    each<kXLoads>(load_x);
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
        if constexpr (kPhases) {
          stage_barrier<kWait + kXLoads>();
          each<kWLoads>(load_w);
          stage_barrier<kWait + kWLoads>();
          each<kXLoads>(load_x);
        } else {
          stage_barrier<kWait>();
          each<kLoads>([&](auto l) { load(l); });
        }
        loaded();
        stage = stage + 1 == NS ? 0 : stage + 1;
        if (lkb == stages) next_loads();
      }
      if constexpr (KG > 1) asm volatile("s_barrier" ::: "memory");  // of the sums
      continue;
    }

    f32x4_t acc[FM][FN];
    each<FM * FN>([&](auto j) { acc[j / FN][j % FN] = f32x4_t{0, 0, 0, 0}; });
    // The scheduling barriers keep the compiler from undoing the order below.
    if constexpr (kPhases) {
      // A stage is two phases of 32 of K, each FM steps of FN MFMAs.  The rows of a
      // step are read kAhead steps before it, the other phase's columns during this
      // one.  At the stage's middle every wavefront has all its columns in
      // registers: the columns' buffer is refilled from there on, and the next
      // stage's have to be there.  kAhead steps before its end the same holds for
      // the rows.  So LDS reads and loads are spread evenly over the MFMAs, and a
      // load has a whole stage to arrive.  4096 x 4096 x 12288: 289 us, 301 with one
      // barrier a stage and the columns' reads behind it; 1 step ahead 295; four
      // wavefronts of 128 x 128 each 303.
      constexpr int kAhead = FM > 2 ? 2 : 1, kHeld = 4, kSteps = 2 * FM;
      uint4 wf[2][FN], xf[kHeld];
      auto columns = [&](const uint8_t* st, auto h, auto f) {
        constexpr int o = 4096 * (f >> 1) + 512 * (f & 1);
        wf[h][f] = *reinterpret_cast<const uint4*>(st + (h ? wo ^ 64 : wo) + o);
      };
      auto rows = [&](const uint8_t* st, auto s) {  // of step s of a stage
        xf[s % kHeld] = *reinterpret_cast<const uint4*>(st + (s >= FM ? xo ^ 64 : xo) + 2048 * (s % FM));
      };
      each<FN>([&](auto f) { columns(lds + stage * kStage, std::integral_constant<int, 0>{}, f); });
      each<kAhead>([&](auto s) { rows(lds + stage * kStage, s); });
      for (int kb = 0; kb < stages;) {
        // the stages until the loads change their tile
        const int n = std::min(stages - kb, stages - lkb);
        for (int r = 0; r < n; ++r) {
          const uint8_t* st = lds + stage * kStage;
          stage = stage + 1 == NS ? 0 : stage + 1;
          const uint8_t* nx = lds + stage * kStage;
          each<kSteps>([&](auto step) {
            constexpr int s = step, h = s / FM, i = s % FM, ahead = s + kAhead;
            if constexpr (s == FM) stage_barrier<kWait + kXLoads>();
            if constexpr (ahead == kSteps) stage_barrier<kWait + kWLoads>();
            rows(ahead < kSteps ? st : nx, std::integral_constant<int, ahead % kSteps>{});
            each<FN>([&](auto f) {
              acc[i][f] = mfma_bf16(wf[h][f], xf[s % kHeld], acc[i][f]);
              // reads and loads, each behind an MFMA of its own
              constexpr int slot = i * FN + f, kRead = (FM - kAhead) * FN;
              each<FN>([&](auto c) {
                if constexpr (slot == kRead * c / FN) columns(h ? nx : st, std::integral_constant<int, 1 - h>{}, c);
              });
              if constexpr (h == 1) {
                each<kWLoads>([&](auto l) {
                  if constexpr (slot == 1 + (kRead - 1) * l / kWLoads) load_w(l);
                });
                each<kXLoads>([&](auto l) {
                  if constexpr (slot == kRead + kAhead * FN * l / kXLoads) load_x(l);
                });
              }
              __builtin_amdgcn_sched_barrier(0);
            });
          });
          loaded();
        }
        kb += n;
        if (lkb == stages) next_loads();
      }
    } else {
      // A wavefront has the operands of a K block in registers and reads those of the
      // next while it multiplies.  Before the last block of a stage stands the
      // stage's barrier: every wavefront has read it, and the next one has to be
      // there; behind it the stage's buffer is refilled.  What a stage costs besides
      // its MFMAs is that barrier and the latency behind it: KS > 1 blocks share it.
      uint4 wf[2][2][FN], xf[2][2][FM];
      auto read = [&](const uint8_t* st, auto set, auto block) {
        each<2 * FN>([&](auto j) {
          constexpr int h = j / FN, f = j % FN, o = block * T::kBlock + 4096 * (f >> 1) + 512 * (f & 1);
          wf[set][h][f] = *reinterpret_cast<const uint4*>(st + (h ? wo ^ 64 : wo) + o);
        });
        each<2 * FM>([&](auto j) {
          constexpr int h = j / FM, i = j % FM, o = block * T::kBlock + 2048 * i;
          xf[set][h][i] = *reinterpret_cast<const uint4*>(st + (h ? xo ^ 64 : xo) + o);
        });
      };
      static_assert(KG == 1 && KS % 2 == 0, "one group of wavefronts, and the sets take turns");
      read(lds + stage * kStage, std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
      for (int kb = 0; kb < stages;) {
        const int n = std::min(stages - kb, stages - lkb);
        for (int r = 0; r < n; ++r) {
          const uint8_t* st = lds + stage * kStage;
          stage = stage + 1 == NS ? 0 : stage + 1;
          const uint8_t* nx = lds + stage * kStage;
          each<KS>([&](auto block) {
            constexpr int set = block % 2;
            constexpr bool last = block == KS - 1;
            constexpr std::integral_constant<int, 1 - set> other;
            if constexpr (last) {
              stage_barrier<kWait>();
              read(nx, other, std::integral_constant<int, 0>{});
            } else {
              read(st, other, std::integral_constant<int, block + 1>{});
            }
            __builtin_amdgcn_sched_barrier(0);
            constexpr int kAll = 2 * FM * FN;
            each<kAll>([&](auto j) {
              constexpr int h = j / (FM * FN), i = j / FN % FM, f = j % FN;
              acc[i][f] = mfma_bf16(wf[set][h][f], xf[set][h][i], acc[i][f]);
              if constexpr (last)
                each<kLoads>([&](auto l) {
                  if constexpr (l >= kLoads * j / kAll && l < kLoads * (j + 1) / kAll) load(l);
                });
              __builtin_amdgcn_sched_barrier(0);
            });
          });
          loaded();
        }
        kb += n;
        if (lkb == stages) next_loads();
      }
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
    const int2* own = pairs + ring * BM + xrow;
    auto at = [&](int i) -> int64_t {
      if constexpr (GROUPED) return own[16 * i].x;
      int r = xrow + 16 * i;
      asm volatile("" : "+v"(r));  // not to be kept: the registers are needed
      const int64_t y = int64_t(row) * BM + r;
      return y < p.M ? y : -1;
    };
    auto wt = [&](int i) { return __int_as_float(own[16 * i].y); };
    finish_tile<FM, FN, GROUPED>(p, acc, at, wt, bias, gated ? n0 + 4 * g : n0 + 8 * g);
  }
  // no load into LDS outlives its workgroup
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

// Columns of Y of a tile of `cols` columns of W.
int own_columns(const ProductParams& p, int cols) { return p.gated ? cols / 2 : cols; }
int column_tiles(const ProductParams& p, int cols) { return (p.No + own_columns(p, cols) - 1) / own_columns(p, cols); }

template <int WM, int WN, int FM, int FN, int NS, bool GROUPED, int KS = 1, int KG = 1>
hipError_t tile_launch(ProductParams p, hipStream_t st) {
  using T = Tile<WM, WN, FM, FN, NS, KS, KG>;
  const int ntiles = column_tiles(p, T::BN);
  const int64_t resident = int64_t(std::max(xcd_compute_units(), 1)) * kXcds * T::groups(GROUPED);
  const int32_t all = GROUPED ? p.blocks : int32_t((p.M + T::BM - 1) / T::BM);
  const int32_t most = GROUPED ? kTileBlocks : all;
  for (p.block0 = 0; p.block0 < all; p.block0 += most) {
    p.blocks = std::min(most, all - p.block0);
    const int64_t grid = std::min(int64_t(p.blocks) * ntiles, resident);
    hipLaunchKernelGGL((gemm_tile_kernel<WM, WN, FM, FN, NS, GROUPED, KS, KG>), dim3(unsigned(grid)),
                       dim3(T::NW * kWave), 0, st, p, ntiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Pieces of an align block that start at once: as many as an expert has on
// average, a block's workgroups take the others in turn (starting every piece
// would leave most workgroups to find padding).
int64_t parts_of(const ProductParams& p) {
  const int64_t each = p.numel / (int64_t(p.E) * 12) + 1;
  return std::min<int64_t>(each, p.block_m / 16);
}

template <int NT, bool GROUPED>
int64_t rows_grid(const ProductParams& p) {
  const int64_t pieces = GROUPED ? p.blocks * parts_of(p) : (p.M + 15) / 16;
  return pieces * column_tiles(p, 16 * NT);
}

// Whether one launch takes so many workgroups of the rows kernel: it has fewer
// than 2^32 threads.  (The tiles' workgroups go from tile to tile, any number.)
bool rows_fit(int64_t grid) { return grid < (int64_t(1) << 32) / (kSplit * kWave); }

template <int NT, bool GROUPED>
hipError_t rows_of(const ProductParams& p, hipStream_t st) {
  hipLaunchKernelGGL((gemm_rows_kernel<NT, GROUPED>), dim3(unsigned(rows_grid<NT, GROUPED>(p))),
                     dim3(kSplit * kWave), 0, st, p, column_tiles(p, 16 * NT), GROUPED ? int(parts_of(p)) * 16 : 0);
  return hipGetLastError();
}

// The current device's; without one, as when a kernel's name is asked for on a host
// that has none, an MI355X's.
int64_t compute_units() {
  const int per = xcd_compute_units();
  return int64_t(per > 0 ? per : 32) * kXcds;
}

// Kernels of the dense product, and their rows x columns of W.
enum DenseForm { kRows16, kRows32, kTile32, kTile32x128, kTile64, kTile64x128, kTile128, kTile128x256, kTile256 };
constexpr const char* kDenseNames[] = {
    "gemm_rows_kernel 16x16", "gemm_rows_kernel 16x32", "gemm_tile_kernel 32x32",
    "gemm_tile_kernel 32x128", "gemm_tile_kernel 64x64", "gemm_tile_kernel 64x128",
    "gemm_tile_kernel 128x128", "gemm_tile_kernel 128x256", "gemm_tile_kernel 256x256"};

// Estimates in microseconds, fitted to measured shapes with W from memory.  A tile
// takes `block` for each 64 of K and each round over the device (one workgroup a
// CU; with fewer tiles than CUs up to a fifth less), `once` a round and `base` a
// call.  Few rows straight from memory: a wavefront's latency over K, for each
// round.
//
// Measured: rows, 32 x 32, 64 x 64, 32 x 128 and 64 x 128: 1 row of 2880 x 2880 5.7,
// 8.5, 11.8, 13.5 and 13.3; 16 rows of 4096 x 4096 9.7, 10.1, 15.2, 17.4 and 17.2; 64 -,
// 10.5, 16.7, 18.0 and 21.6; 256 -, 32.5, 17.5, 19.8 and 21.8; 333 of 2880 x 2880 -, 30,
// 25.6, 16.4 and 18.7.  64 x 128, 128 x 128, 128 x 256 and 256 x 256: 512 of 4096 x 4096
// 26, 30, 45 and 74; 1024 46, 37, 45 and 75; 2048 89, 69, 59 and 76; 4000 of 512 x 4096
// 33, 26, 23 and 21; 4096 of 4096 x 12288 -, -, 333 and 289.
DenseForm dense_form(const ProductParams& p) {
  const int64_t cus = compute_units();
  struct Shape {
    DenseForm form;
    int rows, cols;
    double block, once, base;
  };
  constexpr Shape shapes[] = {{kTile32, 32, 32, 0.1, 0, 3.8},         {kTile32x128, 32, 128, 0.27, 0, 2.5},
                              {kTile64, 64, 64, 0.222, 0, 2.5},       {kTile64x128, 64, 128, 0.34, 0, 2.5},
                              {kTile128, 128, 128, 0.53, 0, 3.0},     {kTile128x256, 128, 256, 0.85, 1.5, 3.0},
                              {kTile256, 256, 256, 1.45, 3.0, 4.0}};
  DenseForm best = kTile32;
  double least = INFINITY;
  for (const Shape& s : shapes) {
    const int64_t tiles = (p.M + s.rows - 1) / s.rows * column_tiles(p, s.cols);
    const double rounds = double((tiles + cus - 1) / cus), part = std::min(1.0, double(tiles) / double(cus));
    const double cost = s.base + rounds * (s.block * p.KB * (0.8 + 0.2 * part) + s.once);
    if (cost < least) least = cost, best = s.form;
  }
  if (p.M <= 16) {
    // (gated, gate and up of 16 columns)
    const int64_t grid = p.gated ? rows_grid<2, false>(p) : rows_grid<1, false>(p);
    const double rounds = double((grid + cus - 1) / cus);
    const double by_rows = p.gated ? 2.0 + 2.9e-3 * p.K * rounds : 1.0 + 1.8e-3 * p.K * rounds;
    if (by_rows < least && rows_fit(grid)) return p.gated ? kRows32 : kRows16;
  }
  return best;
}

// Kernels of the grouped product.
enum GroupedForm { kPairs32, kPairs64, kExperts64, kExperts128, kExperts256 };
constexpr const char* kGroupedNames[] = {"gemm_rows_kernel 16x32", "gemm_rows_kernel 16x64",
                                         "gemm_tile_kernel 64x256", "gemm_tile_kernel 128x256",
                                         "gemm_tile_kernel 256x256"};

// Estimates in microseconds, with the pairs spread evenly: `stream`, one expert's
// weights at 5.5 TB/s.  The rows kernel takes 3 us, and for each piece of 16 rows
// those weights or 4 ns a workgroup; the tiles take 10 us, of which most is
// finding them, and each expert's weights once, or, with few of them, the
// latency of their K.  Measured, rows and tiles: 8 experts of 512 x 1024, 8 rows each,
// 5.7 and 13.5, 96 rows 12.3 and 15.8; 8 of 2048 x 4096, 8 rows 30 and 54, 48 rows 75
// and 59; 128 of 2880 x 2880, 8 rows 361 and 363, 16 rows 477 and 370; 64 of 1536 x
// 1024, 4 rows 38 and 45.  Routing that leaves most pairs to few experts is not
// seen: the rows kernel then reads their weights once for every 16 rows, but reaches
// fewer experts (64 tokens x 4 over 32 experts of 5760 x 2880: even 193 us, one expert
// with 40 rows 205, with 64 and 19 experts reached 154).
GroupedForm grouped_form(const ProductParams& p) {
  const int64_t cus = compute_units();
  const int64_t E = p.E, used = std::min<int64_t>(p.numel, E);
  // tiles of `rows` rows
  auto tiles = [&](int rows) { return std::min<int64_t>(p.numel, std::max(used, p.numel / rows + E / 2)); };
  const double stream = 2.0 * p.N * p.K / 5.5e6;
  const double groups = double((p.N + 31) / 32);
  const double by_rows = 3 + double(tiles(16)) * std::max(stream, 0.004 * groups);
  const double by_tiles = 10 + std::max(0.45 * p.KB, 0.2 * p.KB + double(used) * stream);
  if (by_rows <= by_tiles && rows_fit(rows_grid<2, true>(p))) {
    // 64 columns a workgroup read X half as often as 32, where that leaves a
    // workgroup for every CU (32 experts of 5760 x 2880, 2 rows each, 167.5 us and
    // 171; 8 of 512 x 1024, 96 rows 12.3 and 14.9, 8 rows 7.6 and 5.8)
    return tiles(16) * column_tiles(p, 64) >= cus ? kPairs64 : kPairs32;
  }
  // The tile whose rounds over the device cost least, the largest only with enough
  // rows to fill it whatever the routing.  (64 x 256, 128 x 256 and 256 x 256) 128
  // experts of 1536 x 2048: 32 rows each 155, 155 and 157 us, 64 rows 191, 175 and
  // 180, 128 rows 233, 205 and 196, 512 rows 606, 462 and 437; of 2880 x 2880, 128
  // rows 656, 547 and 483; 16 of 2048 x 4096: 96 rows 73, 80 and 87, 192 rows 115, 79
  // and 99, 256 rows 157, 125 and 102; skewed routing over 64 of 1024 x 1024, 96 rows:
  // 51, 45 and 57; 8 of 512 x 512, 300 rows: 12, 15 and 20.
  const int64_t cols = column_tiles(p, 256);
  auto rounds = [&](int rows) { return (tiles(rows) * cols + cus - 1) / cus; };
  const int64_t cost64 = 80 * rounds(64), cost128 = 98 * rounds(128), cost256 = 140 * rounds(256);
  if (p.block_m <= 64 && cost64 <= cost128) return kExperts64;
  return p.numel <= 96 * E || cost128 <= cost256 ? kExperts128 : kExperts256;
}

}  // namespace

const char* gemm_name(const ProductParams& p) { return kDenseNames[dense_form(p)]; }
const char* moe_gemm_name(const ProductParams& p) { return kGroupedNames[grouped_form(p)]; }

hipError_t launch_gemm(ProductParams p, hipStream_t st) {
  switch (dense_form(p)) {
    case kRows16: return rows_of<1, false>(p, st);
    case kRows32: return rows_of<2, false>(p, st);
    case kTile32: return tile_launch<1, 1, 2, 2, 3, false, 1, 4>(p, st);
    case kTile32x128: return tile_launch<1, 4, 2, 2, 3, false, 2>(p, st);
    case kTile64: return tile_launch<2, 2, 2, 2, 3, false, 2>(p, st);
    case kTile64x128: return tile_launch<2, 4, 2, 2, 3, false, 2>(p, st);
    case kTile128: return tile_launch<2, 4, 4, 2, 4, false>(p, st);
    case kTile128x256: return tile_launch<2, 4, 4, 4, 3, false>(p, st);
    default: return tile_launch<2, 4, 8, 4, 2, false>(p, st);
  }
}

hipError_t launch_moe_gemm(ProductParams p, hipStream_t st) {
  switch (grouped_form(p)) {
    case kPairs32: return rows_of<2, true>(p, st);
    case kPairs64: return rows_of<4, true>(p, st);
    case kExperts64: return tile_launch<2, 4, 2, 4, 3, true>(p, st);
    case kExperts128: return tile_launch<2, 4, 4, 4, 3, true>(p, st);
    default: return tile_launch<2, 4, 8, 4, 2, true>(p, st);
  }
}

}  // namespace mlr
