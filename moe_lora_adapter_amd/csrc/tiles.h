// What the tiled products share: where a block's rows lie, the loads of a ring
// of stages in LDS, and the order and the lists of tiles.
#pragma once

#include <algorithm>

#include "common.h"
#include "dma.h"

namespace mlr {

// Where a block's rows come from and go to.
struct RowMap {
  int64_t x_row;  // row of X, or -1
  int64_t y_row;  // row of Y, or -1
};
template <class Params>
__device__ __forceinline__ RowMap row_of_pair(const Params& p, uint32_t pair) {
  if (pair >= uint32_t(p.numel)) return {-1, -1};
  return {int64_t(p.x_per_pair ? pair : pair / uint32_t(p.topk)), int64_t(pair)};
}
template <bool GROUPED, class Params>
__device__ __forceinline__ RowMap row_of(const Params& p, int64_t first, int i) {
  if constexpr (GROUPED) {
    return row_of_pair(p, uint32_t(p.sorted[first + i]));
  } else {
    const int64_t r = first + i;
    return r < p.M ? RowMap{r, r} : RowMap{-1, -1};
  }
}

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

// stage_barrier<VM>, or, where `young` is not 0, one that also leaves the ST
// stores of the last tile in flight.  They are younger than the loads waited
// for, and memory operations complete in order, so waiting for VM would wait
// for them too.  One asm statement, to keep the loop around it one block.
template <int VM, int ST>
__device__ __forceinline__ void ring_barrier(int young) {
  static_assert(VM + ST < 64, "vmcnt is a 6-bit field");
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\t"
      "s_cbranch_scc1 0f\n\t"
      "s_waitcnt vmcnt(%2) lgkmcnt(0)\n\t"
      "s_branch 1f\n"
      "0:\n\t"
      "s_waitcnt vmcnt(%1) lgkmcnt(0)\n"
      "1:\n\t"
      "s_barrier"
      :
      : "s"(young), "n"(VM), "n"(VM + ST)
      : "memory", "scc");
}

// Work item -> (tile of rows, tile of columns).  Workgroups go to the XCDs in
// turn, so each XCD takes one contiguous run of items, its workgroups in turn;
// its L2 then holds that run's operands.  Within the run G tiles of rows share
// each column tile before the next one: 4 for dense rows (4096 x 4096 x 12288:
// 182 us, alone 192, 16 of them 187), 1 for grouped ones, whose tiles seldom
// have the same weights (120b-like w2, 32768 pairs: 458 us, 4 of them 489).
template <int G>
struct Items {
  uint32_t rows, cols;  // tiles of rows, tiles of columns (of all slices)
  uint32_t first, end;  // this XCD's run
  uint32_t step;        // its workgroups

  __device__ __forceinline__ Items(uint32_t r, uint32_t c) : rows(r), cols(c) {
    const uint32_t total = r * c, per = total / kXcds, rem = total % kXcds;
    const uint32_t xcd = blockIdx.x % kXcds;
    first = xcd * per + min(xcd, rem);
    end = first + per + (xcd < rem ? 1 : 0);
    step = (gridDim.x - xcd + kXcds - 1) / kXcds;
  }
  __device__ __forceinline__ void at(uint32_t t, uint32_t* row, uint32_t* col) const {
    const uint32_t grp = t / (G * cols), base = grp * G;
    const uint32_t size = min(uint32_t(G), rows - base), in = t - base * cols;
    *row = base + in % size;
    *col = in / size;
  }
};

// Grouped: a tile of BM rows takes up to BM / block_m consecutive blocks of one
// expert, so that its weights are read once for all of them.  The first block
// of each tile is found on chip: in every run of blocks with the same expert,
// each (BM / block_m)-th.  Each 64 blocks keep their first blocks as a mask and
// the count of those before them; a launch takes at most kTileBlocks blocks.
constexpr int kTileChunks = 256;
constexpr int kTileBlocks = kTileChunks * kWave;
struct TileList {
  uint64_t lead[kTileChunks];
  uint32_t before[kTileChunks];

  // The whole workgroup; `starts` is LDS scratch of kTileChunks masks.
  // Returns the number of tiles.
  __device__ inline uint32_t build(const int32_t* eids, int blocks, int E, int per, uint64_t* starts,
                                   int nw) {
    const int lane = lane_id(), w = wave_id(), chunks = (blocks + kWave - 1) / kWave;
    // where a run begins, and the blocks whose expert is one; eight chunks' loads
    // in flight (16384 blocks: 24 us with one)
    constexpr int kAtOnce = 8;
    for (int c0 = w; c0 < chunks; c0 += nw * kAtOnce) {
      int e[kAtOnce], before_it[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = std::min((c0 + j * nw) * kWave + lane, blocks - 1);
        e[j] = eids[i];
        before_it[j] = eids[std::max(i - 1, 0)];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int c = c0 + j * nw, i = c * kWave + lane;
        const uint64_t m = __ballot(i < blocks && (i == 0 || e[j] != before_it[j]));
        const uint64_t v = __ballot(i < blocks && uint32_t(e[j]) < uint32_t(E));
        if (lane == 0 && c < chunks) {
          starts[c] = m;
          lead[c] = v;
        }
      }
    }
    __syncthreads();
    for (int c = w; c < kTileChunks; c += nw) {
      uint64_t m = 0;
      if (c < chunks) {
        int run = 0;  // where the run that reaches into this chunk began
        for (int b = c - 1; b >= 0; --b) {
          if (starts[b]) {
            run = b * kWave + 63 - __builtin_clzll(starts[b]);
            break;
          }
        }
        const uint64_t own = starts[c] & (lanes_below(lane) | (uint64_t(1) << lane));
        if (own) run = c * kWave + 63 - __builtin_clzll(own);
        m = lead[c] & __ballot((c * kWave + lane - run) % per == 0);
      }
      if (lane == 0) lead[c] = m;
    }
    __syncthreads();
    constexpr int kEach = kTileChunks / kWave;
    uint32_t n[kEach], sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      n[j] = sum;
      sum += __builtin_popcountll(lead[lane * kEach + j]);
    }
    const uint32_t incl = uint32_t(wave_incl_scan(int(sum)));
    if (w == 0) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) before[lane * kEach + j] = incl - sum + n[j];
    }
    const uint32_t total = uint32_t(lane_value(int(incl), kWave - 1));
    __syncthreads();
    return total;
  }
  // Block of tile t.
  __device__ __forceinline__ int block(uint32_t t) const {
    constexpr int kEach = kTileChunks / kWave;
    const int lane = lane_id();
    const int hi = __builtin_popcountll(__ballot(before[lane * kEach] <= t)) - 1;
    const int lo = __builtin_popcountll(__ballot(lane < kEach && before[hi * kEach + lane % kEach] <= t)) - 1;
    const int c = hi * kEach + lo;
    const uint64_t m = lead[c];
    const bool here = (m >> lane & 1) && __builtin_popcountll(m & lanes_below(lane)) == int(t - before[c]);
    return c * kWave + __builtin_ctzll(__ballot(here));
  }
};

}  // namespace mlr
