// Grouped bf16 products of the experts over ragged row groups:
//   forward and input gradient   C[r, c] = s[r] sum_k A[src(r), k] B[g](c, k)
//   weight gradient              dW[g][i, j] = sum_{r in g} A[srcA(r), i] B[srcB(r), j]
// bf16 operands, float sums (v_mfma_f32_16x16x32_bf16), bf16 or float results.
//
// One K loop serves all three (tile_product below).  An operand is either
// "straight" (the contraction index runs along its rows in memory: both
// operands of the forward product, the A of the input gradient) or "crossed"
// (it runs across rows: the weights of the input gradient, both operands of
// the weight gradient); they differ in how a tile is laid into LDS and read
// back into MFMA fragments, not in the schedule.
//
//   * A workgroup of 8 waves computes a 256 x 256 tile in steps of 64 along
//     the contraction.  Wave (wm, wn) owns 16-row subtiles 2 i + wm of each
//     128-row half of A and columns 32 wn .. + 31 of each 128-column half of
//     B: four quadrants (half of A x half of B) of 16 MFMAs a step, 128 float
//     accumulators.
//   * LDS holds two steps of both operands as eight 16 KB half tiles, filled
//     by direct-to-LDS buffer loads.  Each quadrant is one phase; a phase
//     reads the fragments that its successor needs and requests one half
//     tile into the slot that was last read two phases ago, four to five
//     phases (1 us) before its first use.
//   * Waves 0-3 and 4-7 (one of each per SIMD) run half a phase apart: while
//     one group issues its MFMAs the other reads LDS and requests copies.
//   * Straight half tile: [128 rows][64 k], 16-byte chunks XOR-swizzled by row
//     so that ds_read_b128 has no bank conflicts.  Crossed half tile: [64 k]
//     [128 columns], swizzled for ds_read_b64_tr_b16, which hands each lane
//     four k values of its column.
//   * A tile of fewer than 256 rows skips the MFMAs of its empty subtiles (the
//     loop is compiled for each count); one of up to 288 carries 32 rows behind
//     A's halves; one of at most 128 has no second half of A, and runs two
//     phases a step over three steps in LDS (ShortProduct).
//   * Rows past a group's end, columns past the matrix and the tail of k are
//     given offsets beyond the buffer resource's size and read as zero, so
//     they never meet the group's data, whatever they hold.
//
// Measured, in bf16 with weights of 4096 x 7168, over several cards: one group of 8192
// rows runs at 1260 to 1350 TFLOP/s forward, 1070 to 1180 for the input gradient and 1330
// to 1440 for the weight gradient (the library's products of these shapes: 1490 to
// 1600, 1150 to 1280 and 940 to 980).  33 groups of together 16384 rows: forward 805 to
// 860 us (1120 to 1195 TFLOP/s), input gradient 868 to 945 us with uneven groups, bound
// by the matrix cores (75 and 67 % busy) and, for the groups of 256 rows and fewer,
// by the weights' stream as well; weight gradient to float 1250 to 1320 us, bound by
// its 3.9 GB of stores for the short groups and by the matrix cores for the long
// one.  144 rows over 33 groups: 315 to 335 us, 5.9 TB/s of weights.
#include <type_traits>

#include "rows.h"

namespace {

using namespace moe;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef const __attribute__((address_space(4))) int32_t* uniform_int_t;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;

constexpr int kMaxGroups = 1025;
constexpr int kThreads = 512;
constexpr int kTile = 256;                 // rows and columns of a tile
constexpr int kUnit = 32;                  // row tiles are multiples of this, up to kTile + kUnit
constexpr int kStep = 64;                  // contraction depth of a step
constexpr int kHalf = 128 * kStep * 2;     // bytes of a half tile
// [A, B][half][step parity] and 32 more rows of A twice, or 3 x [A, B0, B1]
constexpr int kLds = 9 * kHalf;
constexpr uint32_t kOut = 0x80000000u;     // an offset past every buffer (all are below 2^31)

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// One operand of a tile, as a lane sees it.
struct Operand {
  const uint8_t* base;     // straight: the tile's first element; crossed: the step's first row
  uint32_t bytes;          // straight, gathered: size of the resource
  uint32_t off[2][2];      // [half][j]: this lane's offsets of its two loads of a half tile
  uint32_t tail;           // straight: added to the offsets in the last step
  uint32_t extra;          // straight: the offset of the load of the extra rows
  // crossed
  const int32_t* index;    // gather, from the group's first row
  int rows, max_row;       // contraction length; last row of a gathered operand
  uint32_t ld2;            // row stride in bytes
};

// Transposing LDS read: the 16 lanes of a group read four rows of 16 values
// (lane i the values 4 (i & 3) .. + 3 of row i >> 2), and lane c receives column
// c.  Through a restrict parameter the compiler sees that no copy in flight
// aliases it; without that it would wait for all of them before every read.
// The waits that these reads need are the explicit ones of the K loop.
__device__ __forceinline__ s16x4 read_tr(lds_s16x4_t __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
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

// Copies and fragment reads.  A_X / B_X: crossed operand.
template <bool A_X, bool B_X>
struct Tile {
  f32x4 acc[2][4][2][2];        // [A half][subtile][B half][subtile]
  f32x4 more[2][2];             // [B half][subtile] of the rows past A's halves
  uint8_t* smem;
  int wave, lane, n_steps;
  const Operand &A, &B;

  __device__ __forceinline__ Tile(uint8_t* s, int w, int l, int n, const Operand& a, const Operand& b)
      : smem(s), wave(w), lane(l), n_steps(n), A(a), B(b) {}

  template <bool X, bool G>
  __device__ __forceinline__ void copy(const Operand& o, uint8_t* slot, int h, int step, const int (&idx)[2]) {
    step = min(step, n_steps - 1);       // steps past the end repeat the last one, unread
    uint8_t* dst = slot + wave * 1024;
    if constexpr (!X) {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(o.base, o.bytes);
      const uint32_t t = step == n_steps - 1 ? o.tail : 0u;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(dst + j * 8192), 16,
                                                 (int)(o.off[h][j] | t), step * (kStep * 2), 0, 0);
    } else if constexpr (!G) {
      const int left = min(o.rows - step * kStep, kStep);
      const __amdgpu_buffer_rsrc_t r =
          make_rsrc(o.base + (long long)step * kStep * o.ld2, (uint32_t)left * o.ld2);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(dst + j * 8192), 16,
                                                 (int)o.off[h][j], 0, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(o.base, o.bytes);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool live = step * kStep + 4 * wave + (lane >> 4) + 32 * j < o.rows;
        int row = idx[j];
        asm volatile("" : "+v"(row));      // keeps the arithmetic here, phases after the load
        const uint32_t at = live ? (uint32_t)clampi(row, 0, o.max_row) * o.ld2 : kOut;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(dst + j * 8192), 16,
                                                 (int)(at + o.off[h][j]), 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void load_index(const Operand& o, int step, int (&idx)[2]) {
    const int first = step * kStep + 4 * wave + (lane >> 4);
#pragma unroll
    for (int j = 0; j < 2; ++j) idx[j] = o.index[min(first + 32 * j, o.rows - 1)];
  }

  // MFMA fragment of 16 rows (columns) and 32 k values
  __device__ __forceinline__ bf16x8 crossed(const uint8_t* s, int blk, int kk) {
    const int lk = lane >> 4, a = (lane & 15) >> 2, q = lane & 3;
    const int x = a | ((lk & 1) << 2);
    const uint8_t* p = s + (kk * 32 + lk * 8 + a) * 256 + (blk ^ x) * 32 + (q >> 1) * 16 + (q & 1) * 8;
    const s16x4 lo = read_tr((lds_s16x4_t)p);
    const s16x4 hi = read_tr((lds_s16x4_t)(p + 1024));
    const bf16x4 l4 = __builtin_bit_cast(bf16x4, lo), h4 = __builtin_bit_cast(bf16x4, hi);
    return __builtin_shufflevector(l4, h4, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ bf16x8 read_a(const uint8_t* s, int i, int kk) {
    const int blk = 2 * i + (wave & 1);
    if constexpr (A_X) {
      return crossed(s, blk, kk);
    } else {
      const int r = lane & 15, lk = lane >> 4;
      return *reinterpret_cast<const bf16x8*>(s + (blk * 16 + r) * 128 + (((lk + 4 * kk) ^ (r >> 1)) << 4));
    }
  }
  __device__ __forceinline__ bf16x8 read_b(const uint8_t* s, int t, int kk) {
    const int wn = wave >> 1;
    if constexpr (B_X) {
      return crossed(s, 2 * wn + t, kk);
    } else {
      // fragment row i holds column 8 (i >> 2) + 4 t + (i & 3): the two
      // subtiles give a lane eight consecutive columns
      const int a = (lane & 15) >> 2, b = lane & 3, lk = lane >> 4;
      return *reinterpret_cast<const bf16x8*>(s + (wn * 32 + a * 8 + t * 4 + b) * 128 +
                                              (((lk + 4 * kk) ^ ((b >> 1) | (a << 1))) << 4));
    }
  }

  template <int H, int L>
  __device__ __forceinline__ void quadrant(const bf16x8 (&a)[4][2], const bf16x8 (&b)[2][2], int hb) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < L; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[H][i][hb][t] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t][kk], a[i][kk], acc[H][i][hb][t], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  }

  __device__ __forceinline__ void extra(const bf16x8 (&a)[2], const bf16x8 (&b)[2][2], int hb) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        more[hb][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t][kk], a[kk], more[hb][t], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  }

  template <int H, int L>
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) acc[H][i][u][v] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
};

// The K loop.  A_G / B_G: gathered crossed operand; L0, L1: 16-row subtiles per
// wave with rows in A's first and second half.  EXTRA: kUnit more rows of a
// straight A, copied together with its second half and multiplied in phase 2.
// (Their 16 accumulators and fragments make the compiler put seven loop
// invariants into scratch; with their second half of the work in phase 3 it is
// 15, and the time the same.)
template <bool A_X, bool B_X, bool A_G, bool B_G, int L0, int L1, bool EXTRA = false>
struct Product : Tile<A_X, B_X> {
  using T = Tile<A_X, B_X>;
  using T::A, T::B, T::smem, T::wave, T::n_steps;
  static constexpr int kIdx = 2 * (A_G ? 1 : 0) + 2 * (B_G ? 1 : 0);   // index loads a step
  static constexpr int kMore = EXTRA ? 1 : 0;                          // copies of the extra rows
  bf16x8 a0[4][2], a1[4][2], a2[2], b0[2][2], b1[2][2];
  int ia[2][2], ib[2][2];       // gathered rows of the two steps ahead, [step parity][j]
  using T::T;

  __device__ __forceinline__ uint8_t* slot(int op, int h, int par) {
    return smem + ((op * 2 + h) * 2 + par) * kHalf;
  }

  __device__ __forceinline__ uint8_t* extra_slot(int par) { return smem + 8 * kHalf + par * (kHalf / 2); }
  __device__ __forceinline__ void copy_extra(int par, int step) {
    step = min(step, n_steps - 1);
    const uint32_t t = step == n_steps - 1 ? A.tail : 0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A.base, A.bytes), (lds_ptr_t)(extra_slot(par) + wave * 1024), 16,
                                             (int)(A.extra | t), step * (kStep * 2), 0, 0);
  }

  // One step in four phases.  PAR: parity of the step's slots.
  template <int PAR>
  __device__ __forceinline__ void step(int s) {
    // phase 0: rest of A0 and all of B0; quadrant (A0, B0)
    if constexpr (L0 > 3) {
      a0[3][0] = this->read_a(slot(0, 0, PAR), 3, 0);
      a0[3][1] = this->read_a(slot(0, 0, PAR), 3, 1);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b0[t][kk] = this->read_b(slot(1, 0, PAR), t, kk);
    this->template copy<A_X, A_G>(A, slot(0, 1, PAR ^ 1), 1, s + 1, ia[PAR ^ 1]);
    if constexpr (EXTRA) copy_extra(PAR ^ 1, s + 1);
    wait_vm<6 + kIdx + kMore>();
    barrier();
    this->template quadrant<0, L0>(a0, b0, 0);
    barrier();
    // phase 1: B1, first of A1; quadrant (A0, B1)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b1[t][kk] = this->read_b(slot(1, 1, PAR), t, kk);
    if constexpr (L1 > 0) {
      a1[0][0] = this->read_a(slot(0, 1, PAR), 0, 0);
      a1[0][1] = this->read_a(slot(0, 1, PAR), 0, 1);
    }
    this->template copy<B_X, B_G>(B, slot(1, 1, PAR ^ 1), 1, s + 1, ib[PAR ^ 1]);
    barrier();
    this->template quadrant<0, L0>(a0, b1, 1);
    barrier();
    // phase 2: rest of A1; quadrant (A1, B1)
#pragma unroll
    for (int i = 1; i < L1; ++i) {
      a1[i][0] = this->read_a(slot(0, 1, PAR), i, 0);
      a1[i][1] = this->read_a(slot(0, 1, PAR), i, 1);
    }
    if constexpr (EXTRA) {
      a2[0] = this->read_a(extra_slot(PAR), 0, 0);
      a2[1] = this->read_a(extra_slot(PAR), 0, 1);
    }
    this->template copy<A_X, A_G>(A, slot(0, 0, PAR), 0, s + 2, ia[PAR]);
    wait_vm<8 + kIdx + kMore>();
    barrier();
    this->template quadrant<1, L1>(a1, b1, 1);
    if constexpr (EXTRA) this->extra(a2, b1, 1);
    if constexpr (EXTRA) this->extra(a2, b0, 0);
    barrier();
    // phase 3: most of the next step's A0; quadrant (A1, B0)
#pragma unroll
    for (int i = 0; i < (L0 < 3 ? L0 : 3); ++i) {
      a0[i][0] = this->read_a(slot(0, 0, PAR ^ 1), i, 0);
      a0[i][1] = this->read_a(slot(0, 0, PAR ^ 1), i, 1);
    }
    if constexpr (A_G) this->load_index(A, s + 3, ia[PAR ^ 1]);
    if constexpr (B_G) this->load_index(B, s + 3, ib[PAR ^ 1]);
    __builtin_amdgcn_sched_barrier(0);
    this->template copy<B_X, B_G>(B, slot(1, 0, PAR), 0, s + 2, ib[PAR]);
    wait_vm<8 + kIdx + kMore>();
    barrier();
    this->template quadrant<1, L1>(a1, b0, 0);
    barrier();
  }

  __device__ __forceinline__ void run() {
    this->template clear<0, L0>();
    this->template clear<1, L1>();
    if constexpr (EXTRA) {
#pragma unroll
      for (int u = 0; u < 4; ++u) this->more[u >> 1][u & 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (n_steps == 0) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (A_G) this->load_index(A, s, ia[s]);
      if constexpr (B_G) this->load_index(B, s, ib[s]);
    }
    this->template copy<A_X, A_G>(A, slot(0, 0, 0), 0, 0, ia[0]);
    this->template copy<B_X, B_G>(B, slot(1, 0, 0), 0, 0, ib[0]);
    this->template copy<A_X, A_G>(A, slot(0, 1, 0), 1, 0, ia[0]);
    if constexpr (EXTRA) copy_extra(0, 0);
    this->template copy<B_X, B_G>(B, slot(1, 1, 0), 1, 0, ib[0]);
    if constexpr (A_G) this->load_index(A, 2, ia[0]);
    if constexpr (B_G) this->load_index(B, 2, ib[0]);
    __builtin_amdgcn_sched_barrier(0);
    this->template copy<A_X, A_G>(A, slot(0, 0, 1), 0, 1, ia[1]);
    this->template copy<B_X, B_G>(B, slot(1, 0, 1), 0, 1, ib[1]);
    wait_vm<8 + kMore>();    // A0 and B0 of step 0
    barrier();
#pragma unroll
    for (int i = 0; i < (L0 < 3 ? L0 : 3); ++i) {
      a0[i][0] = this->read_a(slot(0, 0, 0), i, 0);
      a0[i][1] = this->read_a(slot(0, 0, 0), i, 1);
    }
    if (wave >= 4) barrier();     // half a phase behind
    int s = 0;
    for (; s + 2 <= n_steps; s += 2) {
      step<0>(s);
      step<1>(s + 1);
    }
    if (s < n_steps) step<0>(s);
    if (wave < 4) barrier();
    wait_vm<0>();            // copies in flight would land in the next user's LDS
  }
};

// The K loop of a tile of at most 128 rows (straight A): two phases a step,
// [A, B0, B1] of three steps in LDS, each requested two steps ahead into
// the slots that were last read two phases ago.  L: 16-row subtiles per wave.
template <bool B_X, int L>
struct ShortProduct : Tile<false, B_X> {
  using T = Tile<false, B_X>;
  using T::A, T::B, T::smem, T::wave, T::n_steps;
  static constexpr int kAhead = L < 2 ? L : 2;     // subtiles of A read a phase early
  bf16x8 a0[4][2], b0[2][2], b1[2][2];
  int none[2];
  using T::T;

  __device__ __forceinline__ uint8_t* slot(int which, int stage) { return smem + (stage * 3 + which) * kHalf; }
  __device__ __forceinline__ void read_a_part(int stage, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < lo || i >= hi) continue;
      a0[i][0] = this->read_a(slot(0, stage), i, 0);
      a0[i][1] = this->read_a(slot(0, stage), i, 1);
    }
  }

  // STAGE: the step's slots.
  template <int STAGE>
  __device__ __forceinline__ void step(int s) {
    constexpr int kNext = (STAGE + 1) % 3, kRefill = (STAGE + 2) % 3;
    // phase 0: rest of A and all of B0; quadrant (A, B0)
    read_a_part(STAGE, kAhead, L);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b0[t][kk] = this->read_b(slot(1, STAGE), t, kk);
    this->template copy<false, false>(A, slot(0, kRefill), 0, s + 2, none);
    this->template copy<B_X, false>(B, slot(1, kRefill), 0, s + 2, none);
    wait_vm<8>();
    barrier();
    this->template quadrant<0, L>(a0, b0, 0);
    barrier();
    // phase 1: B1; quadrant (A, B1).  The next step's first subtiles of A are
    // read into their registers behind the MFMAs.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b1[t][kk] = this->read_b(slot(2, STAGE), t, kk);
    this->template copy<B_X, false>(B, slot(2, kRefill), 1, s + 2, none);
    wait_vm<8>();
    barrier();
    this->template quadrant<0, L>(a0, b1, 1);
    read_a_part(kNext, 0, kAhead);
    barrier();
  }

  __device__ __forceinline__ void run() {
    this->template clear<0, L>();
    if (n_steps == 0) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      this->template copy<false, false>(A, slot(0, s), 0, s, none);
      this->template copy<B_X, false>(B, slot(1, s), 0, s, none);
      this->template copy<B_X, false>(B, slot(2, s), 1, s, none);
    }
    wait_vm<8>();            // A and B0 of step 0
    barrier();
    read_a_part(0, 0, kAhead);
    if (wave >= 4) barrier();     // half a phase behind
    int s = 0;
    for (; s + 3 <= n_steps; s += 3) {
      step<0>(s);
      step<1>(s + 1);
      step<2>(s + 2);
    }
    if (s < n_steps) step<0>(s);
    if (s + 1 < n_steps) step<1>(s + 1);
    if (wave < 4) barrier();
    wait_vm<0>();
  }
};

// This lane's offsets of a straight operand (rows[h][j]: the row, relative to
// the operand's base, of load j of half h; negative: nothing there).
__device__ __forceinline__ void straight_offsets(Operand& o, const long long (&rows)[2][2], long long ld,
                                                 int chunk, int K) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o.off[h][j] = rows[h][j] < 0 ? kOut : (uint32_t)(rows[h][j] * ld * 2) + chunk * 16;
  const int last = (K - 1) / kStep * kStep;
  o.tail = last + chunk * 8 < K ? 0u : kOut;
}
// and of a crossed operand of `cols` columns from the tile's first one
__device__ __forceinline__ void crossed_offsets(Operand& o, int wave, int lane, uint32_t ld2, int cols,
                                                bool gathered) {
  const int k = 4 * wave + (lane >> 4);
  const int chunk = (lane & 15) ^ (2 * ((lane >> 4) | (((wave >> 1) & 1) << 2)));
  o.ld2 = ld2;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o.off[h][j] = h * 128 + chunk * 8 >= cols
                        ? kOut
                        : (gathered ? 0u : (uint32_t)(k + 32 * j) * ld2) + h * 256 + chunk * 16;
}

// ---- forward product and input gradient.

// A tile: rows m0 .. m0 + m_rows - 1 of group g (which starts at row row0),
// columns n0 .. n0 + cols - 1.
struct TileAt {
  int g, row0, m0, m_rows, n0, cols;
};

template <bool KN, int L0, int L1, bool EXTRA = false>
__device__ __forceinline__ void gemm_tile(const moe_gemm_bf16_args& a, const TileAt& t, uint8_t* smem) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int K = a.k_dim, N = a.n_out;
  Operand A, B;
  {
    // straight A: load j of wave w fills rows 8 (w + 8 j) .. + 7 of a half tile
    const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    long long rows[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = h * 128 + 8 * (wave + 8 * j) + (lane >> 3);
        rows[h][j] = -1;
        if (r < t.m_rows && (h == 0 || L1 > 0))
          rows[h][j] = a.a_row_index ? clampi(a.a_row_index[t.row0 + t.m0 + r], 0, a.a_rows - 1) : r;
      }
    const uint8_t* base = static_cast<const uint8_t*>(a.a);
    A.base = a.a_row_index ? base : base + (long long)(t.row0 + t.m0) * a.lda * 2;
    A.bytes = (uint32_t)((a.a_row_index ? a.a_rows : t.m_rows) * a.lda * 2);
    straight_offsets(A, rows, a.lda, chunk, K);
    A.extra = kOut;
    if constexpr (EXTRA) {
      const int r = kTile + 8 * wave + (lane >> 3);
      if (r < t.m_rows)
        A.extra = (uint32_t)((a.a_row_index ? (long long)clampi(a.a_row_index[t.row0 + t.m0 + r], 0, a.a_rows - 1) : r) *
                             a.lda * 2) + chunk * 16;
    }
  }
  const uint8_t* b = static_cast<const uint8_t*>(a.b) + (long long)t.g * N * K * 2;
  if constexpr (KN) {
    B.base = b + (long long)t.n0 * 2;
    B.index = nullptr;
    B.rows = K;
    crossed_offsets(B, wave, lane, (uint32_t)N * 2, t.cols, false);
  } else {
    const int chunk = (lane & 7) ^ (((lane >> 4) & 1) | ((wave & 3) << 1));
    long long rows[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = h * 128 + 8 * (wave + 8 * j) + (lane >> 3);
        rows[h][j] = r < t.cols ? r : -1;
      }
    B.base = b + (long long)t.n0 * K * 2;
    B.bytes = (uint32_t)t.cols * (uint32_t)K * 2;
    straight_offsets(B, rows, K, chunk, K);
  }
  typename std::conditional<(L1 > 0), Product<false, KN, false, false, L0, L1, EXTRA>,
                            ShortProduct<KN, L0>>::type p(smem, wave, lane, (K + kStep - 1) / kStep, A, B);
  p.run();

  // A lane holds 4 consecutive columns of one row in each accumulator; with a
  // straight B its two subtiles make 8 consecutive columns.
  const int wm = wave & 1, wn = wave >> 1, lk = lane >> 4;
  auto put = [&](int subtile, const f32x4 (&acc)[2][2]) {
    const int r = (subtile + wm) * 16 + (lane & 15);
    if (r >= t.m_rows) return;
    const long long row = t.row0 + t.m0 + r;
    const float s = a.row_scale ? a.row_scale[row] : 1.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int c = u * 128 + wn * 32 + (KN ? v * 16 + lk * 4 : lk * 8 + v * 4);
        if (c >= t.cols) continue;
        const long long at = row * a.ldo + t.n0 + c;
        const f32x4 x = acc[u][v] * s;
        if (a.out_dtype == MOE_F32) {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = x;
        } else {
          bf16x4 y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = (__bf16)x[e];
          *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.out) + at) = y;
        }
      }
  };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < (h ? L1 : L0); ++i) put(h * 8 + 2 * i, p.acc[h][i]);
  if constexpr (EXTRA) put(16, p.more);
}

template <bool KN>
__device__ __forceinline__ void short_tile(const moe_gemm_bf16_args& a, const TileAt& t, uint8_t* smem) {
  const int l0 = (t.m_rows + 31) / 32;
  if (l0 > 2) l0 > 3 ? gemm_tile<KN, 4, 0>(a, t, smem) : gemm_tile<KN, 3, 0>(a, t, smem);
  else l0 > 1 ? gemm_tile<KN, 2, 0>(a, t, smem) : gemm_tile<KN, 1, 0>(a, t, smem);
}

// Rows of group gi (0 for a group past the last).
__device__ __forceinline__ int group_rows(const int32_t* offsets, int gi, int G, int total, int& lo) {
  lo = 0;
  if (gi < 0 || gi >= G) return 0;
  lo = clampi(offsets[gi], 0, total);
  return max(clampi(offsets[gi + 1], 0, total) - lo, 0);
}

// Row tiles of a group of `rows` rows: its units of kUnit rows are spread
// evenly over as few tiles of at most kTile + kUnit rows as hold them.  A tile of
// a few rows takes 0.6 of a full one's time, for it streams the same
// weights: with tiles of 256 rows and a rest, 32 groups of 4096 x 7168 take 428 us at
// 256 rows, 726 at 288, 712 at 300 and 1058 at 600; spread evenly 427, 466, 568
// and 908 (at most 256 rows each: 428, 462, 571, 913, and 851 against 807 at 530).
__device__ __forceinline__ int units_of(int rows) { return (rows + kUnit - 1) / kUnit; }
__device__ __forceinline__ int row_tiles_of(int rows) {
  constexpr int kMost = (kTile + kUnit) / kUnit;
  return (units_of(rows) + kMost - 1) / kMost;
}

// Exclusive prefix of v over the workgroup's threads, and the total.
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
  for (int w = 0; w < kThreads / 64; ++w) {
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
constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;      // groups of a thread
constexpr int kCounterStride = 16;                                // ints between the XCDs' counters
constexpr int kListAt = kLds;                                     // behind the half tiles: row tiles before group g
constexpr int kNextAt = kListAt + (kMaxGroups + 1) * 4;           // and the next position, the group found
constexpr int kListLds = (kNextAt + 16 + 15) / 16 * 16;

struct GemmParams {
  moe_gemm_bf16_args a;
  unsigned* next;          // [8] counters, NULL when the first tiles are all
};

__global__ void tile_counters_kernel(unsigned* next, unsigned first) {
  if (threadIdx.x < kXcds) next[threadIdx.x * kCounterStride] = first;
}

struct TileList {
  const moe_gemm_bf16_args& a;
  const int* before;       // LDS
  int* shared;             // LDS: the next position, the group found
  unsigned* next;
  int n_tiles, tiles, run, runs, stride;      // run: its tiles
  int home, xcd;           // the workgroup's XCD; the one whose list it takes from

  __device__ __forceinline__ TileList(const GemmParams& p, uint8_t* smem, int* tmp)
      : a(p.a), before(reinterpret_cast<int*>(smem + kListAt)), shared(reinterpret_cast<int*>(smem + kNextAt)),
        next(p.next) {
    const int G = a.num_groups, per = (G + kThreads - 1) / kThreads;
    int* list = reinterpret_cast<int*>(smem + kListAt);
    int lo, mt[kPer], sum = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mt[i] = i < per ? row_tiles_of(group_rows(a.group_offsets, (int)threadIdx.x * per + i, G, a.total_rows, lo)) : 0;
      sum += mt[i];
    }
    int at = prefix(sum, tmp, all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i < per && (int)threadIdx.x * per + i < G) list[(int)threadIdx.x * per + i] = at;
      at += mt[i];
    }
    if (threadIdx.x == 0) list[G] = all;
    __syncthreads();
    n_tiles = (a.n_out + kTile - 1) / kTile;
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
  // The tile at position `slot` of the current XCD's list, or at a later one
  // of this list and the others; false when there is none.
  __device__ __forceinline__ bool find(int slot, TileAt& t) {
    for (;;) {
      const int j = slot / run * kXcds + xcd;
      if (j < runs) {
        const int want = (int)((long long)j * stride % runs) * run + slot % run;
        if (want < tiles) {
          const int row_tile = want / n_tiles;
          for (int g = threadIdx.x; g < a.num_groups; g += kThreads)
            if (before[g] <= row_tile && row_tile < before[g + 1]) shared[1] = g;
          __syncthreads();
          t.g = __builtin_amdgcn_readfirstlane(shared[1]);
          const int first = __builtin_amdgcn_readfirstlane(before[t.g]);
          const int mt = __builtin_amdgcn_readfirstlane(before[t.g + 1]) - first;
          const int in = want - first * n_tiles;
          const int band = in / (kBand * n_tiles), rest = in - band * kBand * n_tiles;
          const int height = min(kBand, mt - band * kBand);
          const int n_tile = rest / height;
          const uniform_int_t offsets = (uniform_int_t)(uintptr_t)a.group_offsets;
          t.row0 = clampi(offsets[t.g], 0, a.total_rows);
          const int rows = clampi(offsets[t.g + 1], 0, a.total_rows) - t.row0;
          const int i = band * kBand + rest - n_tile * height, units = units_of(rows);
          t.m0 = (int)((long long)units * i / mt) * kUnit;
          t.m_rows = min(rows, (int)((long long)units * (i + 1) / mt) * kUnit) - t.m0;
          t.n0 = n_tile * kTile;
          t.cols = min(kTile, a.n_out - t.n0);
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
    if (threadIdx.x == 0) shared[0] = (int)position;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(shared[0]);
  }
  __device__ __forceinline__ int pop_now() { return publish(pop()); }
};

template <bool KN>
__global__ __launch_bounds__(kThreads, 2) void grouped_gemm_bf16_kernel(GemmParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  TileList list(p, smem, reinterpret_cast<int*>(smem));
  TileAt t;
  for (int slot = blockIdx.x / kXcds; list.find(slot, t);) {
    const unsigned popped = list.pop();
    const int l1 = (t.m_rows - 128 + 31) / 32;
    if (t.m_rows > kTile) gemm_tile<KN, 4, 4, true>(p.a, t, smem);
    else if (t.m_rows <= 128) short_tile<KN>(p.a, t, smem);
    else if (l1 > 2) l1 > 3 ? gemm_tile<KN, 4, 4>(p.a, t, smem) : gemm_tile<KN, 4, 3>(p.a, t, smem);
    else l1 > 1 ? gemm_tile<KN, 4, 2>(p.a, t, smem) : gemm_tile<KN, 4, 1>(p.a, t, smem);
    if (!p.next) return;
    slot = list.publish(popped);      // and all waves are done with LDS
  }
}

// Small groups: the time is the weights' stream, so every workgroup (one per
// compute unit) streams the same number of weight columns.  Each group with
// rows counts its columns once per 128 rows, in units of 16, or 64 (a cache
// line) where a weight row is cut at a unit's edge; workgroup b takes units
// [U b / blocks, U (b + 1) / blocks), in pieces of at most 256 columns and
// about equal width inside one group.
template <bool KN>
__global__ __launch_bounds__(kThreads, 2) void grouped_gemm_bf16_stream_kernel(GemmParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const moe_gemm_bf16_args& a = p.a;
  int* tmp = reinterpret_cast<int*>(smem);
  constexpr int kPiece = KN ? 64 : 16;
  const int G = a.num_groups, units = (a.n_out + kPiece - 1) / kPiece;
  const int per = (G + kThreads - 1) / kThreads;
  int sum = 0, lo;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < per) sum += (group_rows(a.group_offsets, (int)threadIdx.x * per + i, G, a.total_rows, lo) + 127) / 128;
  int all;
  const int at = prefix(sum, tmp, all);
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
      const int tiles = (group_rows(a.group_offsets, g, G, a.total_rows, lo) + 127) / 128;
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
    const int rows = group_rows(a.group_offsets, g, G, a.total_rows, t.row0);
    if (m * 128 >= rows) {        // the group is done, or has no rows
      ++g, m = 0;
      continue;
    }
    t.g = g;
    t.m0 = m * 128;
    t.m_rows = min(rows - t.m0, 128);
    const int here = (int)min((long long)(units - u), left);      // units of this row tile
    const int pieces = (here + kTile / kPiece - 1) / (kTile / kPiece);
    const int take = (here + pieces - 1) / pieces;
    t.n0 = u * kPiece;
    t.cols = min(take * kPiece, a.n_out - t.n0);
    __syncthreads();              // LDS is free again
    short_tile<KN>(a, t, smem);
    left -= take;
    u += take;
    if (u >= units) u = 0, ++m;
  }
}

// ---- weight gradient: one workgroup per 256 x 256 tile of one group's dW.
//
// Most groups have a few hundred rows, so a tile is a few steps and then 256 KB
// of float results, whose way to memory bounds it.  What that asks for:
//   * results go through LDS and leave as whole rows of the tile, with
//     non-temporal stores that do not push the operands out of L2 (straight from
//     the accumulators, in 64-byte pieces, stores reach 3.8 TB/s; whole cache
//     lines 5.5, whole rows 5.8);
//   * an XCD takes an eighth of a group's tiles, column tiles in bands of
//     kWBand, so that its L2 fetches an eighth of B and A once a band; the
//     eighths rotate with the group, for groups with fewer than 8 tiles; groups
//     go from the last (the shared expert, whose tiles are the longest) to the
//     first.
// Where there are few tiles, each group's rows are cut into `splits` parts,
// whose partial sums (float, in the workspace) a second kernel adds in order.
constexpr int kWBand = 4;
constexpr int kOutStride = kTile * 4 + 16;      // bytes between rows staged in LDS, off the banks' period
static_assert(128 * kOutStride <= kLds, "half a tile of float rows fits");

struct WgradParams {
  moe_wgrad_bf16_args a;
  int splits;
  float* part;             // [splits][G][n][k] when splits > 1
};

// One row piece of 16 bytes, `old` being what accumulation adds to.
__device__ __forceinline__ void put16(float* o, const uint8_t* s, bool accumulate) {
  f32x4 x = *reinterpret_cast<const f32x4*>(s);
  if (accumulate) x += *reinterpret_cast<const f32x4*>(o);
  __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(o));
}
__device__ __forceinline__ void put16(__bf16* o, const uint8_t* s, bool accumulate) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(s), hi = *reinterpret_cast<const f32x4*>(s + 16);
  bf16x8 old = {}, y;
  if (accumulate) old = *reinterpret_cast<const bf16x8*>(o);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = (__bf16)(accumulate ? lo[e] + (float)old[e] : lo[e]);
    y[4 + e] = (__bf16)(accumulate ? hi[e] + (float)old[4 + e] : hi[e]);
  }
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, y), reinterpret_cast<u32x4*>(o));
}

template <typename OUT, typename P>
__device__ __forceinline__ void store_tile(const P& p, uint8_t* smem, int wave, int lane, OUT* out, long long ld,
                                           int rows, int cols, bool accumulate) {
  const int wm = wave & 1, wn = wave >> 1, lk = lane >> 4;
  constexpr int kLanes = kTile * (int)sizeof(OUT) / 16;      // lanes that a row takes
  constexpr int kRows = 64 / kLanes;                         // rows of a wave's store
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h * 128 >= rows) break;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v)
          *reinterpret_cast<f32x4*>(smem + ((2 * i + wm) * 16 + (lane & 15)) * kOutStride +
                                    (u * 128 + wn * 32 + v * 16 + lk * 4) * 4) = p.acc[h][i][u][v];
    __syncthreads();
    const int c = lane % kLanes * (16 / (int)sizeof(OUT));
#pragma unroll 4
    for (int r = wave * kRows + lane / kLanes; r < 128; r += 8 * kRows)
      if (h * 128 + r < rows && c < cols)
        put16(out + (h * 128 + r) * ld + c, smem + r * kOutStride + c * 4, accumulate);
  }
}

template <bool A_G, bool B_G>
__global__ __launch_bounds__(kThreads, 2) void grouped_wgrad_bf16_kernel(WgradParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const moe_wgrad_bf16_args& a = p.a;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int nt = (a.n + kTile - 1) / kTile, kt = (a.k + kTile - 1) / kTile, tiles = nt * kt * p.splits;
  const int per = (tiles + kXcds - 1) / kXcds, slot = blockIdx.x / kXcds;
  const int g = a.num_groups - 1 - slot / per;
  const int at = ((blockIdx.x + g) & (kXcds - 1)) * per + slot % per;
  if (at >= tiles) return;
  const int split = at / (nt * kt), in = at - split * nt * kt;
  const int band = in / (kWBand * nt), r = in - band * kWBand * nt, width = min(kWBand, kt - band * kWBand);
  const int m0 = r / width * kTile, n0 = (band * kWBand + r % width) * kTile;
  int row0 = clampi(a.group_offsets[g], 0, a.total_rows);
  int rows = max(clampi(a.group_offsets[g + 1], 0, a.total_rows) - row0, 0);
  if (p.splits > 1) {          // this part of the rows, in whole steps
    const int steps = (rows + kStep - 1) / kStep;
    const int lo = (int)((long long)steps * split / p.splits) * kStep;
    const int hi = min((int)((long long)steps * (split + 1) / p.splits) * kStep, rows);
    row0 += lo;
    rows = hi - lo;
  }
  Operand A, B;
  const uint8_t* ab = static_cast<const uint8_t*>(a.a) + (long long)m0 * 2;
  const uint8_t* bb = static_cast<const uint8_t*>(a.b) + (long long)n0 * 2;
  A.base = A_G ? ab : ab + (long long)row0 * a.lda * 2;
  B.base = B_G ? bb : bb + (long long)row0 * a.ldb * 2;
  A.bytes = (uint32_t)((long long)a.a_rows * a.lda * 2 - m0 * 2);
  B.bytes = (uint32_t)((long long)a.b_rows * a.ldb * 2 - n0 * 2);
  A.index = A_G ? a.a_row_index + row0 : nullptr;
  B.index = B_G ? a.b_row_index + row0 : nullptr;
  A.rows = B.rows = rows;
  A.max_row = a.a_rows - 1;
  B.max_row = a.b_rows - 1;
  crossed_offsets(A, wave, lane, (uint32_t)a.lda * 2, a.n - m0, A_G);
  crossed_offsets(B, wave, lane, (uint32_t)a.ldb * 2, a.k - n0, B_G);
  Product<true, true, A_G, B_G, 4, 4> product(smem, wave, lane, (rows + kStep - 1) / kStep, A, B);
  product.run();

  const int out_rows = min(a.n - m0, kTile), out_cols = min(a.k - n0, kTile);
  if (p.splits > 1)
    store_tile(product, smem, wave, lane, p.part + (((long long)split * a.num_groups + g) * a.n + m0) * a.k + n0, a.k,
               out_rows, out_cols, false);
  else if (a.out_dtype == MOE_F32)
    store_tile(product, smem, wave, lane, static_cast<float*>(a.out) + ((long long)g * a.n + m0) * a.k + n0, a.k,
               out_rows, out_cols, a.accumulate);
  else
    store_tile(product, smem, wave, lane, static_cast<__bf16*>(a.out) + ((long long)g * a.n + m0) * a.k + n0, a.k,
               out_rows, out_cols, a.accumulate);
}

// out = (out +) the sum of the parts, eight values a thread.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* part, int splits, long long values, void* out,
                                                          moe_dtype_t dt, int accumulate) {
  const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= values) return;
  f32x4 x[2] = {};
  for (int s = 0; s < splits; ++s) {
    const f32x4* q = reinterpret_cast<const f32x4*>(part + s * values + at);
    x[0] += q[0];
    x[1] += q[1];
  }
  if (dt == MOE_F32) {
    put16(static_cast<float*>(out) + at, reinterpret_cast<const uint8_t*>(x), accumulate);
    put16(static_cast<float*>(out) + at + 4, reinterpret_cast<const uint8_t*>(x + 1), accumulate);
  } else {
    put16(static_cast<__bf16*>(out) + at, reinterpret_cast<const uint8_t*>(x), accumulate);
  }
}

// Parts that a group's rows are cut into: with fewer tiles than half the
// compute units, as many as fill them, of at least 512 rows on average.
int wgrad_splits(int num_groups, int total_rows, int n, int k) {
  const long long tiles = (long long)num_groups * ((n + kTile - 1) / kTile) * ((k + kTile - 1) / kTile);
  if (tiles == 0 || tiles > 128) return 1;
  const long long fill = 256 / tiles, deep = total_rows / num_groups / 512;
  const long long s = fill < deep ? fill : deep;
  return s > 1 ? (int)s : 1;
}

// Row tiles of 256 that the groups can make at most.
long long row_tiles(int num_groups, int total_rows) {
  return (long long)total_rows / kTile + (num_groups < total_rows ? num_groups : total_rows);
}
// Up to 48 rows a group on average the weights' stream decides.  32 groups of
// 4096 x 7168 take, in the stream kernel and in row tiles: at 2 rows a group 307 and
// 317 us (317 and 323 in the other layout), at 48 328 and 326 (330, 332), at 96
// 366 and 344 (372, 342), at 160 775 and 374 (787, 358); 33 groups of 48 rows, which do
// not fill whole rounds of row tiles, 368 and 404 (378, 369).  The host knows the
// mean alone, and a group of hundreds of rows among small ones is streamed once for
// each 128 of them: 32 groups of 9 and one of 300 rows take 455 and 386 us (421, 346), 30
// of 10 and three of 400 rows 500 and 411 (476, 360).
bool streams_weights(int num_groups, int total_rows) { return total_rows <= 48LL * num_groups; }
// Workgroups of an XCD: one per compute unit (of the whole chip without a device).
int places() {
  const int cus = cu_count();
  return cus < kXcds ? 32 : cus / kXcds;
}

// element rows that 32-bit byte offsets of a gathered operand can reach
bool fits31(long long rows, long long ld) { return rows * ld * 2 < (1LL << 31); }
// a tile's or a step's rows of an operand that is not gathered
bool tile_fits31(long long ld) { return fits31(kTile + kUnit, ld); }

}  // namespace

extern "C" size_t moe_grouped_gemm_bf16_workspace_bytes(int num_groups, int total_rows, int n_out,
                                                        int k_dim) {
  (void)k_dim;
  if (num_groups < 1 || total_rows < 1 || n_out < 1 || streams_weights(num_groups, total_rows)) return 0;
  const long long tiles = row_tiles(num_groups, total_rows) * ((n_out + kTile - 1) / kTile);
  if (tiles <= kXcds * kRun && places() >= kRun) return 0;      // every tile is some workgroup's first
  return kXcds * kCounterStride * sizeof(unsigned);
}

extern "C" moe_status_t moe_grouped_gemm_bf16(const moe_gemm_bf16_args* args, void* ws, size_t ws_bytes,
                                              hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_gemm_bf16_args& a = *args;
  if (a.total_rows < 0 || a.n_out < 0 || a.k_dim < 0 || a.n_out % 8 || a.k_dim % 8 ||
      a.num_groups < 1 || a.lda < a.k_dim || a.lda % 8 || a.ldo < a.n_out || a.ldo % 8 || a.a_rows < 0)
    return MOE_ERR_SHAPE;
  if (a.num_groups > kMaxGroups || !valid_dtype(a.out_dtype) ||
      (a.b_layout != MOE_B_NK && a.b_layout != MOE_B_KN) ||
      !fits31(a.n_out, a.k_dim) || !tile_fits31(a.lda) ||
      (a.b_layout == MOE_B_KN && !fits31(kStep, a.n_out)))
    return MOE_ERR_UNSUPPORTED;
  if (a.a_row_index && !fits31(a.a_rows, a.lda)) return MOE_ERR_UNSUPPORTED;
  if (!a.a_row_index && a.a_rows < a.total_rows) return MOE_ERR_SHAPE;
  if (a.total_rows == 0 || a.n_out == 0) return MOE_OK;
  if (a.a_rows == 0) return MOE_ERR_SHAPE;
  if (!a.group_offsets || !a.out || (a.k_dim > 0 && (!a.a || !a.b))) return MOE_ERR_NULL;
  if (!aligned16(a.a) || !aligned16(a.b) || !aligned16(a.out)) return MOE_ERR_ALIGN;
  const size_t need = moe_grouped_gemm_bf16_workspace_bytes(a.num_groups, a.total_rows, a.n_out, a.k_dim);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return MOE_ERR_ALIGN;
  if (row_tiles(a.num_groups, a.total_rows) * ((a.n_out + kTile - 1) / kTile) > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (moe_status_t s = check_device()) return s;
  const bool kn = a.b_layout == MOE_B_KN, stream_weights = streams_weights(a.num_groups, a.total_rows);
  const int grid = places() * kXcds;
  const GemmParams p{a, need ? static_cast<unsigned*>(ws) : nullptr};
  if (need) {
    hipLaunchKernelGGL(tile_counters_kernel, dim3(1), dim3(64), 0, stream, p.next, (unsigned)grid / kXcds);
    if (moe_status_t s = launch_status()) return s;
  }
  static void (*const table[2][2])(GemmParams) = {
      {grouped_gemm_bf16_kernel<false>, grouped_gemm_bf16_kernel<true>},
      {grouped_gemm_bf16_stream_kernel<false>, grouped_gemm_bf16_stream_kernel<true>}};
  static std::atomic<uint64_t> lds_set[2][2] = {};
  const auto kernel = table[stream_weights][kn];
  if (moe_status_t st = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), kListLds, lds_set[stream_weights][kn]))
    return st;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), kListLds, stream, p);
  return launch_status();
}

extern "C" size_t moe_grouped_wgrad_bf16_workspace_bytes(int num_groups, int total_rows, int n,
                                                         int k) {
  if (num_groups < 1 || total_rows < 0 || n < 0 || k < 0) return 0;
  const int s = wgrad_splits(num_groups, total_rows, n, k);
  return s > 1 ? (size_t)s * num_groups * n * k * sizeof(float) : 0;
}

extern "C" moe_status_t moe_grouped_wgrad_bf16(const moe_wgrad_bf16_args* args, void* ws,
                                               size_t ws_bytes, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_wgrad_bf16_args& a = *args;
  if (a.total_rows < 0 || a.n < 0 || a.k < 0 || a.n % 8 || a.k % 8 || a.num_groups < 1 ||
      a.lda < a.n || a.lda % 8 || a.ldb < a.k || a.ldb % 8 || a.a_rows < 0 || a.b_rows < 0)
    return MOE_ERR_SHAPE;
  if (a.num_groups > kMaxGroups || !valid_dtype(a.out_dtype)) return MOE_ERR_UNSUPPORTED;
  if ((a.a_row_index && !fits31(a.a_rows, a.lda)) || (a.b_row_index && !fits31(a.b_rows, a.ldb)) ||
      !tile_fits31(a.lda) || !tile_fits31(a.ldb))
    return MOE_ERR_UNSUPPORTED;
  if ((!a.a_row_index && a.a_rows < a.total_rows) || (!a.b_row_index && a.b_rows < a.total_rows) ||
      (a.total_rows > 0 && (a.a_rows == 0 || a.b_rows == 0)))
    return MOE_ERR_SHAPE;
  if (a.n == 0 || a.k == 0) return MOE_OK;
  if (!a.group_offsets || !a.out || (a.total_rows > 0 && (!a.a || !a.b))) return MOE_ERR_NULL;
  if (!aligned16(a.a) || !aligned16(a.b) || !aligned16(a.out)) return MOE_ERR_ALIGN;
  const int splits = wgrad_splits(a.num_groups, a.total_rows, a.n, a.k);
  if (splits > 1) {
    if (!ws || ws_bytes < moe_grouped_wgrad_bf16_workspace_bytes(a.num_groups, a.total_rows, a.n, a.k))
      return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_ALIGN;
  }
  const long long tiles = (long long)((a.n + kTile - 1) / kTile) * ((a.k + kTile - 1) / kTile) * splits;
  const long long grid = a.num_groups * ((tiles + kXcds - 1) / kXcds * kXcds);
  if (grid > 0x7FFFFFFFLL) return MOE_ERR_UNSUPPORTED;
  if (moe_status_t s = check_device()) return s;
  static void (*const table[2][2])(WgradParams) = {
      {grouped_wgrad_bf16_kernel<false, false>, grouped_wgrad_bf16_kernel<false, true>},
      {grouped_wgrad_bf16_kernel<true, false>, grouped_wgrad_bf16_kernel<true, true>}};
  const int ga = a.a_row_index && a.total_rows > 0, gb = a.b_row_index && a.total_rows > 0;
  static std::atomic<uint64_t> lds_set[2][2] = {};
  if (moe_status_t st = allow_dynamic_lds(reinterpret_cast<const void*>(table[ga][gb]), kLds, lds_set[ga][gb]))
    return st;
  const WgradParams p{a, splits, static_cast<float*>(ws)};
  hipLaunchKernelGGL(table[ga][gb], dim3((unsigned)grid), dim3(kThreads), kLds, stream, p);
  if (moe_status_t s = launch_status()) return s;
  if (splits > 1) {
    const long long values = (long long)a.num_groups * a.n * a.k;
    hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)((values / 8 + 255) / 256)), dim3(256), 0, stream,
                       static_cast<const float*>(ws), splits, values, a.out, a.out_dtype, a.accumulate);
    return launch_status();
  }
  return MOE_OK;
}
