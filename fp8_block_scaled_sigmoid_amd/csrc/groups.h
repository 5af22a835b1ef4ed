// Helpers of the grouped products (bf16 and 4-bit): waits and buffer resources of
// direct-to-LDS copies, the row tiles of ragged groups, and which workgroup takes
// which tile.  There is one workgroup per compute unit.
#pragma once

#include "rows.h"

namespace moe {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef const __attribute__((address_space(4))) int32_t* uniform_int_t;

constexpr int kMaxGroups = 1025;
constexpr int kTileRows = 256;             // of a tile, and up to kUnit more
constexpr int kUnit = 32;                  // row tiles are multiples of this
constexpr uint32_t kOut = 0x80000000u;     // an offset past every buffer (all are below 2^31)

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The groups of a call, and the columns of its result.
struct Groups {
  const int32_t* offsets;
  int n, rows, columns;
};

// A tile: rows m0 .. m0 + m_rows - 1 of group g (which starts at row row0),
// columns n0 .. n0 + cols - 1.
struct TileAt {
  int g, row0, m0, m_rows, n0, cols;
};

// Rows of group gi (0 for a group past the last).
__device__ __forceinline__ int group_rows(const Groups& of, int gi, int& lo) {
  lo = 0;
  if (gi < 0 || gi >= of.n) return 0;
  lo = clampi(of.offsets[gi], 0, of.rows);
  return max(clampi(of.offsets[gi + 1], 0, of.rows) - lo, 0);
}

// Row tiles of a group of `rows` rows: its units of kUnit rows are spread
// evenly over as few tiles of at most kTileRows + kUnit rows as hold them.  A tile of
// a few rows takes 0.6 of a full one's time, for it streams the same
// weights: with tiles of 256 rows and a rest, 32 groups of 4096 x 7168 take 428 us at
// 256 rows, 726 at 288, 712 at 300 and 1058 at 600; spread evenly 427, 466, 568
// and 908 (at most 256 rows each: 428, 462, 571, 913, and 851 against 807 at 530).
__device__ __forceinline__ int units_of(int rows) { return (rows + kUnit - 1) / kUnit; }
constexpr int kMostUnits = (kTileRows + kUnit) / kUnit;
__device__ __forceinline__ int row_tiles_of(int rows, int most) { return (units_of(rows) + most - 1) / most; }

// Exclusive prefix of v over the workgroup's threads, and the total.
template <int THREADS>
__device__ __forceinline__ int prefix(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int n = __shfl_up(incl, o, 64);
    if (lane >= o) incl += n;
  }
  if (lane == 63) tmp[wave] = incl;
  __syncthreads();
  int before = incl - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    const int n = tmp[w];
    if (w < wave) before += n;
    total += n;
  }
  __syncthreads();
  return before;
}

// The tile list of the large-batch kernel.  A group's row tiles go in bands of
// up to kBand, column tile by column tile, so that tiles which share a weight tile
// follow one another.  kRun consecutive tiles, one round of an XCD's compute
// units (fewer where that would leave XCDs without any), form a run; run j of
// the dispatch order belongs to XCD j % 8, and its tiles share a few row and
// column tiles through that XCD's L2.  Runs are dispatched in the order of a
// golden-ratio stride over the list: a group with many rows needs the matrix
// cores and hardly any memory, one with few rows the reverse, and this way
// every moment has some of both (33 groups of together 16384 rows, even and
// uneven, timed in turn on two cards: in list order 1.0 % and 1.0 to 1.8 % more, 858
// and 867 us, 933 and 945).  Runs of 16, 32 and 64 tiles
// take 858, 852 and 840 us and 935, 910 and 909; bands of 2, 4 and 8 row tiles 840,
// 852 and 853, and 923, 910 and 917 (on a card whose clock was lower).
//
// The grid is one workgroup per compute unit.  A workgroup's first tile is its
// own by position; further ones come from its XCD's counter and, when that
// XCD's runs are all taken, from the next XCD's: tiles differ in time, and
// workgroups that the hardware hands out one per tile leave a tenth of the
// compute units waiting.
constexpr int kXcds = 8;
constexpr int kBand = 4;
constexpr int kRun = 32;
template <int THREADS>
constexpr int kPer = (kMaxGroups + THREADS - 1) / THREADS;        // groups of a thread
constexpr int kCounterStride = 16;                                // ints between the XCDs' counters
constexpr int kListBytes = (kMaxGroups - 1) * 4;                  // LDS: row tiles before group g, g from 1 on

static __global__ void tile_counters_kernel(unsigned* next, unsigned first) {
  if (threadIdx.x < kXcds) next[threadIdx.x * kCounterStride] = first;
}

// WIDTH: columns of a tile.  `list` is LDS that stays, `tmp` LDS that only the
// members' calls use (all waves are done with it when they return).
template <int WIDTH, int THREADS>
struct TileList {
  const Groups of;
  int* const list;
  int* const tmp;
  unsigned* const next;    // [8] counters, NULL when the first tiles are all
  int n_tiles, all, tiles, run, runs, stride;      // all: row tiles; run: its tiles
  int home, xcd;           // the workgroup's XCD; the one whose list it takes from

  // most: units of a tile
  __device__ __forceinline__ TileList(const Groups& groups, uint8_t* list_at, uint8_t* tmp_at, unsigned* counters,
                                      int most = kMostUnits)
      : of(groups), list(reinterpret_cast<int*>(list_at)), tmp(reinterpret_cast<int*>(tmp_at)), next(counters) {
    const int G = of.n, per = (G + THREADS - 1) / THREADS;
    int lo, mt[kPer<THREADS>], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer<THREADS>; ++i) {
      mt[i] = i < per ? row_tiles_of(group_rows(of, (int)threadIdx.x * per + i, lo), most) : 0;
      sum += mt[i];
    }
    int at = prefix<THREADS>(sum, tmp, all);
#pragma unroll
    for (int i = 0; i < kPer<THREADS>; ++i) {
      const int g = (int)threadIdx.x * per + i;
      if (i < per && g > 0 && g < G) list[g - 1] = at;
      at += mt[i];
    }
    __syncthreads();
    n_tiles = (of.columns + WIDTH - 1) / WIDTH;
    tiles = all * n_tiles;
    run = min(kRun, max((tiles + kXcds - 1) / kXcds, 1));
    runs = (tiles + run - 1) / run;
    stride = max((int)(0.618034f * runs), 1);
    for (;; ++stride) {               // the next one that has no factor in common with the runs
      int x = runs, y = stride;
      while (y) {
        const int r = x % y;
        x = y;
        y = r;
      }
      if (x <= 1) break;
    }
    home = xcd = blockIdx.x & (kXcds - 1);
  }
  // Row tiles before group g.
  __device__ __forceinline__ int before(int g) const { return g == 0 ? 0 : g == of.n ? all : list[g - 1]; }
  // The tile at position `slot` of the current XCD's list, or at a later one
  // of this list and the others; false when there is none.
  __device__ __forceinline__ bool find(int slot, TileAt& t) {
    for (;;) {
      const int j = slot / run * kXcds + xcd;
      if (j < runs) {
        const int want = (int)((long long)j * stride % runs) * run + slot % run;
        if (want < tiles) {
          const int row_tile = want / n_tiles;
          for (int g = threadIdx.x; g < of.n; g += THREADS)
            if (before(g) <= row_tile && row_tile < before(g + 1)) tmp[1] = g;
          __syncthreads();
          t.g = __builtin_amdgcn_readfirstlane(tmp[1]);
          const int first = __builtin_amdgcn_readfirstlane(before(t.g));
          const int mt = __builtin_amdgcn_readfirstlane(before(t.g + 1)) - first;
          __syncthreads();
          const int in = want - first * n_tiles;
          const int band = in / (kBand * n_tiles), rest = in - band * kBand * n_tiles;
          const int height = min(kBand, mt - band * kBand);
          const int n_tile = rest / height;
          const uniform_int_t offsets = (uniform_int_t)(uintptr_t)of.offsets;
          t.row0 = clampi(offsets[t.g], 0, of.rows);
          const int rows = clampi(offsets[t.g + 1], 0, of.rows) - t.row0;
          const int i = band * kBand + rest - n_tile * height, units = units_of(rows);
          t.m0 = (int)((long long)units * i / mt) * kUnit;
          t.m_rows = min(rows, (int)((long long)units * (i + 1) / mt) * kUnit) - t.m0;
          t.n0 = n_tile * WIDTH;
          t.cols = min(WIDTH, of.columns - t.n0);
          return true;
        }
      } else {
        xcd = (xcd + 1) & (kXcds - 1);
        if (xcd == home) return false;
      }
      if (!next) return false;
      slot = pop_now();
    }
  }
  __device__ __forceinline__ unsigned pop() {
    // (an increment, because the compiler wraps a wave-wide reduction around an
    // addition, and that would wait for the result at once)
    return next && threadIdx.x == 0 ? atomicInc(next + xcd * kCounterStride, 0x7FFFFFFFu) : 0u;
  }
  __device__ __forceinline__ int publish(unsigned position) {
    __syncthreads();
    if (threadIdx.x == 0) tmp[0] = (int)position;
    __syncthreads();
    const int got = __builtin_amdgcn_readfirstlane(tmp[0]);
    __syncthreads();
    return got;
  }
  __device__ __forceinline__ int pop_now() { return publish(pop()); }
};

// Small groups: the time is the weights' stream, so every workgroup (one per
// compute unit) streams the same number of weight columns.  Each group with
// rows counts its columns once per 128 rows, in units of PIECE; workgroup b takes
// units [U b / blocks, U (b + 1) / blocks), in tiles of at most WIDTH columns and
// about equal width inside one group, each passed to `f`.  tmp: LDS that f may
// use as well.
template <int WIDTH, int PIECE, int THREADS, typename F>
__device__ __forceinline__ void stream_tiles(const Groups& of, uint8_t* tmp_at, F f) {
  int* tmp = reinterpret_cast<int*>(tmp_at);
  const int units = (of.columns + PIECE - 1) / PIECE;
  const int per = (of.n + THREADS - 1) / THREADS;
  int sum = 0, lo;
#pragma unroll
  for (int i = 0; i < kPer<THREADS>; ++i)
    if (i < per) sum += (group_rows(of, (int)threadIdx.x * per + i, lo) + 127) / 128;
  int all;
  const int at = prefix<THREADS>(sum, tmp, all);
  // row tiles in 64 bits: units of the whole list pass 2^31
  const long long first = (long long)all * units * blockIdx.x / gridDim.x;
  const long long last = (long long)all * units * (blockIdx.x + 1) / gridDim.x;
  if (first >= last) return;
  const int want = (int)(first / units);      // the row tile that the range starts in
  int u = (int)(first - (long long)want * units);
  if (want >= at && want < at + sum) {
    int m = want - at;
    for (int i = 0; i < per; ++i) {
      const int g = (int)threadIdx.x * per + i;
      const int tiles = (group_rows(of, g, lo) + 127) / 128;
      if (m < tiles) {
        tmp[8] = g, tmp[9] = m;
        break;
      }
      m -= tiles;
    }
  }
  __syncthreads();
  int g = __builtin_amdgcn_readfirstlane(tmp[8]), m = __builtin_amdgcn_readfirstlane(tmp[9]);
  for (long long left = last - first; left > 0;) {
    TileAt t;
    const int rows = group_rows(of, g, t.row0);
    if (m * 128 >= rows) {        // the group is done, or has no rows
      ++g, m = 0;
      continue;
    }
    t.g = g;
    t.m0 = m * 128;
    t.m_rows = min(rows - t.m0, 128);
    const int here = (int)min((long long)(units - u), left);      // units of this row tile
    const int pieces = (here + WIDTH / PIECE - 1) / (WIDTH / PIECE);
    const int take = (here + pieces - 1) / pieces;
    t.n0 = u * PIECE;
    t.cols = min(take * PIECE, of.columns - t.n0);
    __syncthreads();              // LDS is free again
    f(t);
    left -= take;
    u += take;
    if (u >= units) u = 0, ++m;
  }
}

}  // namespace moe

// ---------------------------------------------------------------------------
// host side
namespace moe {

// Row tiles that the groups can make at most.
inline long long row_tiles(int num_groups, int total_rows, int tile_rows = kTileRows) {
  return (long long)total_rows / tile_rows + (num_groups < total_rows ? num_groups : total_rows);
}
// Workgroups of an XCD: one per compute unit (of the whole chip without a device).
inline int places() {
  const int cus = cu_count();
  return cus < kXcds ? 32 : cus / kXcds;
}
// Bytes of the XCDs' counters; 0 when every tile is some workgroup's first.
inline size_t counter_bytes(long long tiles) {
  return tiles <= kXcds * kRun && places() >= kRun ? 0 : kXcds * kCounterStride * sizeof(unsigned);
}

}  // namespace moe
