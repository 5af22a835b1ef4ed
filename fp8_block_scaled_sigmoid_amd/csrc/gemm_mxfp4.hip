// Grouped product of the experts in microscaled 4-bit floating point
// (include/moe_fp8.h gives formula and layout).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 128 columns of 16 rows of each operand;
// lane l holds the 16 bytes of block l >> 4 of row l & 15 and, in one byte of a
// register that its op_sel picks, that block's scale.  Its sums are exact up to a
// rounding or two of the float result (measured: 2^-24 of the sum of
// magnitudes), whatever the scales.
//
// At 16 cycles it takes as long as the bf16 instruction for a quarter of the columns, from
// the same 16 bytes a lane, so the bf16 product's schedule carries over with
// steps of 256 columns (128 bytes of a row):
//   * A workgroup of 8 waves computes a 256 x 256 tile.  Wave (wm, wn) owns 16-row
//     subtiles 2 i + wm of each 128-row half of A and rows 32 wn .. + 31 of each
//     128-row half of B: four quadrants (half of A x half of B) of 16 MFMAs a step,
//     128 float accumulators.
//   * LDS holds two steps of both operands as eight 16 KB half tiles, filled
//     by direct-to-LDS buffer loads.  Each quadrant is one phase; a phase
//     reads the fragments that its successor needs and requests one half
//     tile into the slot that was last read two phases ago.
//   * Waves 0-3 and 4-7 (one of each per SIMD) run half a phase apart: while
//     one group issues its MFMAs the other reads LDS and requests copies.
//   * Scales: a row's 16 bytes for 512 columns are one lane's copy, so all rows of
//     both operands take one load a wave every second step; a lane's four scales
//     of a row are then one ds_read_b32, and the MFMA picks the byte.
//   * A tile of fewer than 256 rows skips the MFMAs of its empty subtiles (the
//     loop is compiled for each count); one of up to 288 carries 32 rows behind
//     A's halves; one of at most 128 has no second half of A, and runs two
//     phases a step over three steps in LDS (ShortProduct).
//   * For the gated epilogue B's halves are the gate rows and the up rows of the
//     same 128 columns, so a lane holds both products of each of its columns and,
//     with the three lanes that share its row, one block of the result: activation,
//     scale and codes need two lane exchanges and no LDS.
//   * Rows past a group's end, rows of B past the matrix and blocks past k are
//     given offsets beyond the buffer resource's size and read as zero.
//
// Measured, weights of 4096 x 7168, over several cards: one group of 8192 rows takes 132 to
// 143 us (3370 to 3650 TFLOP/s; the instruction alone, on random operands, reaches 7000 at
// the clock that its power leaves), 33 groups of together 16384 rows 275 to 290 us
// (gated 270 to 275, to float 305 to 312), 32 groups of 256 rows 157 to 163, 144 rows over
// 33 groups 98 us, 5.2 TB/s of weights.  The matrix cores are busy 41 % of the large
// call's time.  Per step of 256 columns and tile (from the slope over k): 1.8 us where the
// weights are in L2, of which the copies alone take 1.1 and everything but them 1.5;
// 2.4 us at 16 groups of 256 rows, copies alone 2.2.
#include <type_traits>

#include "groups.h"
#include "mx.h"

namespace {

using namespace moe;

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kTile = kTileRows;           // rows and columns of a tile
constexpr int kStepBlocks = 8;             // blocks of 32 columns in a step
constexpr int kStepBytes = 16 * kStepBlocks;
constexpr int kHalf = 128 * kStepBytes;    // bytes of a half tile
// Rows of B from which tiles have more than 128 rows of A: their loads add up to 192 rows to
// a scalar offset, which may not pass the resource.  At k 7168 a matrix of 192 rows in short
// tiles and one of 193 in tall ones take 28 and 40 us for 300 rows of A, 32 and 59 for 8192, 81
// and 82 for 65536, but 68 and 57 for 33 groups of 1024.
constexpr int kLeastRows = 193;
// LDS of a tile: [A, B][half][step parity], 32 more rows of A twice, a place for loads
// that are not wanted, and twice the scales of 256 rows of A and of B and of 64 more of
// A; or 3 x [A, B0, B1] and twice the scales of 128 rows of A and 256 of B
constexpr int kWaveBytes = 1024;           // what a wave's load fills
constexpr int kExtraAt = 8 * kHalf, kExtra = kUnit * kStepBytes;
constexpr int kUnwantedAt = kExtraAt + 2 * kExtra;
constexpr int kScaleAt = kUnwantedAt + kWaveBytes, kScales = (2 * kTile + 64) * 16;
constexpr int kShortScaleAt = 9 * kHalf, kShortScales = (128 + kTile) * 16;
constexpr int kLds = kShortScaleAt + 2 * kShortScales;
static_assert(kScaleAt + 2 * kScales <= kLds && kLds + kListBytes <= 160 * 1024, "LDS of a compute unit");

// One operand of a tile, as a lane sees it.
struct Operand {
  const uint8_t* base;     // codes
  uint32_t bytes;          // size of the resource
  uint32_t off[2][2];      // [half][j]: this lane's offsets of its two loads of a half tile
  uint32_t tail;           // kOut where the last step has no such block
  uint32_t extra;          // the offset of the load of the extra rows
  uint32_t row_bytes;
};
// The scales: a wave loads 64 rows of one operand.
struct Scales {
  const uint8_t* base;
  uint32_t bytes, off;
  int at;                  // where in LDS
  const uint8_t* a_base;   // and of the extra rows
  uint32_t a_bytes, extra;
};

template <int J>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, J, (int)sa, J, (int)sb);
}

// Copies and fragment reads.
struct Tile {
  f32x4 acc[2][4][2][2];        // [A half][subtile][B half][subtile]
  f32x4 more[2][2];             // [B half][subtile] of the rows past A's halves
  uint8_t* smem;
  int wave, lane, n_steps;
  uint32_t a_at[2], b_at[2], sa_at, sb_at;      // this lane's part of its reads' addresses
  const Operand &A, &B;
  const Scales& S;

  // b_slots, a_sc, b_sc: where B's half tiles and the scales of either operand start, so that
  // what is left of a slot's place fits a read instruction's 16 bits.
  __device__ __forceinline__ Tile(uint8_t* s, int w, int l, int n, const Operand& a, const Operand& b, const Scales& sc,
                                  int b_slots, int a_sc, int b_sc)
      : smem(s), wave(w), lane(l), n_steps(n), A(a), B(b), S(sc) {
    const int r = l & 15, lk = l >> 4, wn = w >> 1;
    const int a_row = (w & 1) * 16 + r, b_row = wn * 32 + (r >> 2) * 8 + (r & 3);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      a_at[kk] = a_row * kStepBytes + (((lk + 4 * kk) ^ (r >> 1)) << 4);
      b_at[kk] = b_slots + b_row * kStepBytes + (((lk + 4 * kk) ^ (((r & 3) >> 1) | ((r >> 2) << 1))) << 4);
    }
    sa_at = a_sc + a_row * 16 + lk * 4;
    sb_at = b_sc + b_row * 16 + lk * 4;
    // one register each, to which the slots are constants: otherwise the wave's part
    // joins the slot's and takes an addition, or a register, for every slot
    asm volatile("" : "+v"(a_at[0]), "+v"(a_at[1]), "+v"(b_at[0]), "+v"(b_at[1]), "+v"(sa_at), "+v"(sb_at));
  }

  // No copy stands under a condition: the compiler would move the matrix
  // instructions of earlier phases past the branch.

  // TAIL: the last step may have fewer blocks than the others.
  template <bool TAIL>
  __device__ __forceinline__ void copy(const Operand& o, int slot, int h, int step) {
    step = min(step, n_steps - 1);       // steps past the end repeat the last one, unread
    const __amdgpu_buffer_rsrc_t r = make_rsrc(o.base, o.bytes);
    const uint32_t t = TAIL && step == n_steps - 1 ? o.tail : 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(smem + slot + wave * kWaveBytes + j * 8192), 16,
                                               (int)(o.off[h][j] | t), step * kStepBytes, 0, 0);
  }

  // The same for rows at one stride (row_bytes), the offset of the first of which is
  // off[0][0]; rows past the matrix lie past the resource.  The bounds check compares a
  // lane's offset with the resource's bytes less the scalar offset, which is below them: it
  // is less than kLeastRows rows, and narrower matrices take short tiles.  A lane's own offset
  // is less than 64 rows past the matrix, below 2^32 because 288 rows are below 2^31 bytes.
  template <bool TAIL>
  __device__ __forceinline__ void copy_rows(const Operand& o, int slot, int h, int step) {
    step = min(step, n_steps - 1);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(o.base, o.bytes);
    const uint32_t t = TAIL && step == n_steps - 1 ? o.tail : 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(smem + slot + wave * kWaveBytes + j * 8192), 16,
                                               (int)(o.off[0][0] | t),
                                               (h * 128 + j * 64) * (int)o.row_bytes + step * kStepBytes, 0, 0);
  }

  // Fragment of 16 rows of the half tile at `slot`: block lk + 4 kk of each row's step.
  __device__ __forceinline__ u32x4 read_a(int slot, int i, int kk) {
    return *reinterpret_cast<const u32x4*>(smem + a_at[kk] + (slot + i * 32 * kStepBytes));
  }
  // Fragment row i holds column 8 (i >> 2) + 4 t + (i & 3): the two subtiles
  // give a lane eight consecutive columns.
  __device__ __forceinline__ u32x4 read_b(int slot, int t, int kk) {
    return *reinterpret_cast<const u32x4*>(smem + b_at[kk] + (slot + t * 4 * kStepBytes));
  }
  // This lane's scales of two steps.
  __device__ __forceinline__ uint32_t a_scales(int slot, int i) {
    return *reinterpret_cast<const uint32_t*>(smem + sa_at + (slot + i * 32 * 16));
  }
  __device__ __forceinline__ uint32_t b_scales(int slot, int t) {
    return *reinterpret_cast<const uint32_t*>(smem + sb_at + (slot + t * 4 * 16));
  }

  // Subtiles LO .. HI - 1 of a half of A.  PAR: the step's parity, which picks the scale
  // byte together with kk.
  template <int H, int LO, int HI, int PAR>
  __device__ __forceinline__ void quadrant(const u32x4 (&a)[4][2], const u32x4 (&b)[2][2], int hb,
                                           const uint32_t (&sa)[4], const uint32_t (&sb)[2]) {
#pragma unroll
    for (int i = LO; i < HI; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc[H][i][hb][t] = mfma<2 * PAR>(b[t][0], a[i][0], acc[H][i][hb][t], sb[t], sa[i]);
#pragma unroll
    for (int i = LO; i < HI; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc[H][i][hb][t] = mfma<2 * PAR + 1>(b[t][1], a[i][1], acc[H][i][hb][t], sb[t], sa[i]);
  }
  template <int PAR>
  __device__ __forceinline__ void extra(const u32x4 (&a)[2], const u32x4 (&b)[2][2], int hb, uint32_t sa,
                                        const uint32_t (&sb)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) more[hb][t] = mfma<2 * PAR>(b[t][0], a[0], more[hb][t], sb[t], sa);
#pragma unroll
    for (int t = 0; t < 2; ++t) more[hb][t] = mfma<2 * PAR + 1>(b[t][1], a[1], more[hb][t], sb[t], sa);
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

// The K loop.  L0, L1: 16-row subtiles per wave with rows in A's first and second
// half.  EXTRA: kUnit more rows of A, copied together with its second half; only
// for whole steps, because the last step's offsets would not fit the registers.
template <int L0, int L1, bool EXTRA = false>
struct Product : Tile {
  static constexpr int kMore = EXTRA ? 1 : 0;        // copies of the extra rows
  // subtiles of A0 and A1 read a phase early: what the registers hold (a K loop that
  // reloads a value from scratch memory waits for every copy in flight there: 32
  // groups of 288 rows took 195 us in a build with one reload, 251 in one with four, on
  // different cards, and take 168 to 174 without)
  static constexpr int kMost = EXTRA ? 0 : 3, kAhead = L0 < kMost ? L0 : kMost;
  static constexpr int kFirst = EXTRA || L1 == 0 ? 0 : 1;
  u32x4 a0[4][2], a1[4][2], a2[2], b0[2][2], b1[2][2];
  uint32_t sa0[4], sa1[4], sa2, sb0[2], sb1[2];      // scales of this step and its successor
  __device__ __forceinline__ Product(uint8_t* s, int w, int l, int n, const Operand& a, const Operand& b, const Scales& sc)
      : Tile(s, w, l, n, a, b, sc, slot(1, 0, 0), kScaleAt, kScaleAt + kScaleB) {}

  static constexpr int slot(int op, int h, int par) { return ((op * 2 + h) * 2 + par) * kHalf; }
  static constexpr int extra_slot(int par) { return kExtraAt + par * kExtra; }
  // Scales of the pair of steps: A's halves, B's halves, A's extra rows.
  static constexpr int scale_slot(int which) { return kScaleAt + which * kScales; }
  static constexpr int kScaleB = kTile * 16, kScaleExtra = 2 * kTile * 16;

  // Waves 0-3 load eight of the extra rows each; the others' loads are not wanted.
  __device__ __forceinline__ void copy_extra(int par, int step) {
    step = min(step, n_steps - 1);
    uint8_t* to = smem + (wave < 4 ? extra_slot(par) + wave * kWaveBytes : kUnwantedAt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A.base, A.bytes), (lds_ptr_t)to, 16, (int)A.extra,
                                             step * kStepBytes, 0, 0);
  }
  // Waves 0-3 load the scales of A's rows, waves 4-7 those of B's, wave 0 also those of
  // the extra rows.
  __device__ __forceinline__ void copy_scales(int which, int pair) {
    const int from = min(pair, (n_steps - 1) >> 1) * 16;
    const int s = scale_slot(which);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(S.base, S.bytes), (lds_ptr_t)(smem + s + S.at), 16,
                                             (int)S.off, from, 0, 0);
    if constexpr (EXTRA) {
      uint8_t* to = smem + (wave == 0 ? s + kScaleExtra : kUnwantedAt);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(S.a_base, S.a_bytes), (lds_ptr_t)to, 16, (int)S.extra, from, 0, 0);
    }
  }

  // One step in four phases.  PAR: parity of the step's slots, PAIR: of its scales'.
  template <int PAR, int PAIR>
  __device__ __forceinline__ void step(int s) {
    constexpr int sc = PAIR * kScales;
    // an even step requests the scales of the next pair
    constexpr int kScaleLoads = PAR == 0 ? 1 + kMore : 0;
    // phase 0: rest of A0 and all of B0; quadrant (A0, B0)
#pragma unroll
    for (int i = kAhead; i < L0; ++i) {
      a0[i][0] = read_a(slot(0, 0, PAR), i, 0);
      a0[i][1] = read_a(slot(0, 0, PAR), i, 1);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b0[t][kk] = read_b(slot(0, 0, PAR), t, kk);
    if constexpr (PAR == 0) {
#pragma unroll
      for (int i = 0; i < L0; ++i) sa0[i] = a_scales(sc, i);
#pragma unroll
      for (int t = 0; t < 2; ++t) sb0[t] = b_scales(sc, t);
    }
    copy<!EXTRA>(A, slot(0, 1, PAR ^ 1), 1, s + 1);
    if constexpr (EXTRA) copy_extra(PAR ^ 1, s + 1);
    if constexpr (PAR == 0) copy_scales(PAIR ^ 1, (s >> 1) + 1);
    wait_vm<6 + kMore + kScaleLoads>();
    barrier();
    __builtin_amdgcn_s_setprio(1);
    quadrant<0, 0, L0, PAR>(a0, b0, 0, sa0, sb0);
    __builtin_amdgcn_s_setprio(0);
    barrier();
    // phase 1: B1, first of A1; quadrant (A0, B1).  The extra rows are read and
    // multiplied here, into registers that the first of A0 leaves.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b1[t][kk] = read_b(slot(0, 1, PAR), t, kk);
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
      a1[i][0] = read_a(slot(0, 1, PAR), i, 0);
      a1[i][1] = read_a(slot(0, 1, PAR), i, 1);
    }
    if constexpr (PAR == 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t) sb1[t] = b_scales(sc + 128 * 16, t);
      if constexpr (EXTRA) sa2 = a_scales(sc + kScaleExtra, 0);
    }
    copy_rows<!EXTRA>(B, slot(1, 1, PAR ^ 1), 1, s + 1);
    barrier();
    __builtin_amdgcn_s_setprio(1);
    if constexpr (EXTRA) {
      quadrant<0, 0, 2, PAR>(a0, b1, 1, sa0, sb1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t at = a_at[kk];
        asm volatile("" : "+v"(at));      // added here, not kept
        a2[kk] = *reinterpret_cast<const u32x4*>(smem + at + extra_slot(PAR));
      }
      __builtin_amdgcn_sched_barrier(0);
      quadrant<0, 2, L0, PAR>(a0, b1, 1, sa0, sb1);
      extra<PAR>(a2, b1, 1, sa2, sb1);
      extra<PAR>(a2, b0, 0, sa2, sb0);
    } else {
      quadrant<0, 0, L0, PAR>(a0, b1, 1, sa0, sb1);
    }
    __builtin_amdgcn_s_setprio(0);
    barrier();
    // phase 2: rest of A1; quadrant (A1, B1)
#pragma unroll
    for (int i = kFirst; i < L1; ++i) {
      a1[i][0] = read_a(slot(0, 1, PAR), i, 0);
      a1[i][1] = read_a(slot(0, 1, PAR), i, 1);
    }
    if constexpr (PAR == 0) {
#pragma unroll
      for (int i = 0; i < L1; ++i) sa1[i] = a_scales(sc + 128 * 16, i);
    }
    copy<!EXTRA>(A, slot(0, 0, PAR), 0, s + 2);
    wait_vm<8 + kMore + kScaleLoads>();
    barrier();
    __builtin_amdgcn_s_setprio(1);
    quadrant<1, 0, L1, PAR>(a1, b1, 1, sa1, sb1);
    __builtin_amdgcn_s_setprio(0);
    barrier();
    // phase 3: most of the next step's A0; quadrant (A1, B0)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a0[i][0] = read_a(slot(0, 0, PAR ^ 1), i, 0);
      a0[i][1] = read_a(slot(0, 0, PAR ^ 1), i, 1);
    }
    copy_rows<!EXTRA>(B, slot(1, 0, PAR), 0, s + 2);
    wait_vm<8 + kMore + kScaleLoads>();
    barrier();
    __builtin_amdgcn_s_setprio(1);
    quadrant<1, 0, L1, PAR>(a1, b0, 0, sa1, sb0);
    __builtin_amdgcn_s_setprio(0);
    barrier();
  }

  __device__ __forceinline__ void run() {
    clear<0, L0>();
    clear<1, L1>();
    if constexpr (EXTRA) {
#pragma unroll
      for (int u = 0; u < 4; ++u) more[u >> 1][u & 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (n_steps == 0) return;
    copy_scales(0, 0);
    copy<!EXTRA>(A, slot(0, 0, 0), 0, 0);
    copy_rows<!EXTRA>(B, slot(1, 0, 0), 0, 0);
    copy<!EXTRA>(A, slot(0, 1, 0), 1, 0);
    if constexpr (EXTRA) copy_extra(0, 0);
    copy_rows<!EXTRA>(B, slot(1, 1, 0), 1, 0);
    copy<!EXTRA>(A, slot(0, 0, 1), 0, 1);
    copy_rows<!EXTRA>(B, slot(1, 0, 1), 0, 1);
    wait_vm<8 + kMore>();    // the first scales, A0 and B0 of step 0
    barrier();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a0[i][0] = read_a(slot(0, 0, 0), i, 0);
      a0[i][1] = read_a(slot(0, 0, 0), i, 1);
    }
    if (wave >= 4) barrier();     // half a phase behind
    int s = 0;
    for (; s + 4 <= n_steps; s += 4) {
      step<0, 0>(s);
      step<1, 0>(s + 1);
      step<0, 1>(s + 2);
      step<1, 1>(s + 3);
    }
    if (s < n_steps) step<0, 0>(s);
    if (s + 1 < n_steps) step<1, 0>(s + 1);
    if (s + 2 < n_steps) step<0, 1>(s + 2);
    if (wave < 4) barrier();
    wait_vm<0>();            // copies in flight would land in the next user's LDS
  }
};

// The K loop of a tile of at most 128 rows: two phases a step, [A, B0, B1] of
// three steps in LDS, each requested two steps ahead into the slots that were
// last read two phases ago.  L: 16-row subtiles per wave.
template <int L>
struct ShortProduct : Tile {
  static constexpr int kAhead = L < 2 ? L : 2;     // subtiles of A read a phase early
  u32x4 a0[4][2], b0[2][2], b1[2][2];
  uint32_t sa[4], sb0[2], sb1[2];
  __device__ __forceinline__ ShortProduct(uint8_t* s, int w, int l, int n, const Operand& a, const Operand& b,
                                          const Scales& sc)
      : Tile(s, w, l, n, a, b, sc, 0, kShortScaleAt, kShortScaleAt + kScaleB) {}

  static constexpr int slot(int which, int stage) { return (stage * 3 + which) * kHalf; }
  __device__ __forceinline__ int scale_slot(int pair) { return kShortScaleAt + (pair & 1) * kShortScales; }
  static constexpr int kScaleB = 128 * 16;
  __device__ __forceinline__ void read_a_part(int stage, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < lo || i >= hi) continue;
      a0[i][0] = read_a(slot(0, stage), i, 0);
      a0[i][1] = read_a(slot(0, stage), i, 1);
    }
  }
  // Waves 0 and 1 load the scales of A's rows, the others those of B's (waves 5 to 7
  // the same ones).
  __device__ __forceinline__ void copy_scales(int pair) {
    const int from = min(pair, (n_steps - 1) >> 1) * 16;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(S.base, S.bytes), (lds_ptr_t)(smem + scale_slot(pair) + S.at), 16,
                                             (int)S.off, from, 0, 0);
  }

  // STAGE: the step's slots, PAR: its parity.
  template <int STAGE, int PAR>
  __device__ __forceinline__ void step(int s) {
    constexpr int kNext = (STAGE + 1) % 3, kRefill = (STAGE + 2) % 3;
    const int sc = ((s >> 1) & 1) * kShortScales;
    constexpr int kScaleLoads = PAR == 0 ? 1 : 0;      // of the next pair of steps
    // phase 0: rest of A and all of B0; quadrant (A, B0)
    read_a_part(STAGE, kAhead, L);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b0[t][kk] = read_b(slot(1, STAGE), t, kk);
    if constexpr (PAR == 0) {
#pragma unroll
      for (int i = 0; i < L; ++i) sa[i] = a_scales(sc, i);
#pragma unroll
      for (int t = 0; t < 2; ++t) sb0[t] = b_scales(sc, t);
    }
    copy<true>(A, slot(0, kRefill), 0, s + 2);
    copy<true>(B, slot(1, kRefill), 0, s + 2);
    if constexpr (PAR == 0) copy_scales((s >> 1) + 1);
    wait_vm<8 + kScaleLoads>();
    barrier();
    __builtin_amdgcn_s_setprio(1);
    quadrant<0, 0, L, PAR>(a0, b0, 0, sa, sb0);
    __builtin_amdgcn_s_setprio(0);
    barrier();
    // phase 1: B1; quadrant (A, B1).  The next step's first subtiles of A are
    // read into their registers behind the MFMAs.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) b1[t][kk] = read_b(slot(2, STAGE), t, kk);
    if constexpr (PAR == 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t) sb1[t] = b_scales(sc + 128 * 16, t);
    }
    copy<true>(B, slot(2, kRefill), 1, s + 2);
    wait_vm<8 + kScaleLoads>();
    barrier();
    __builtin_amdgcn_s_setprio(1);
    quadrant<0, 0, L, PAR>(a0, b1, 1, sa, sb1);
    __builtin_amdgcn_s_setprio(0);
    read_a_part(kNext, 0, kAhead);
    barrier();
  }

  __device__ __forceinline__ void run() {
    clear<0, L>();
    if (n_steps == 0) return;
    copy_scales(0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      copy<true>(A, slot(0, s), 0, s);
      copy<true>(B, slot(1, s), 0, s);
      copy<true>(B, slot(2, s), 1, s);
    }
    wait_vm<8>();            // the first scales, A and B0 of step 0
    barrier();
    read_a_part(0, 0, kAhead);
    if (wave >= 4) barrier();     // half a phase behind
    int s = 0;
    for (; s + 6 <= n_steps; s += 6) {
      step<0, 0>(s);
      step<1, 1>(s + 1);
      step<2, 0>(s + 2);
      step<0, 1>(s + 3);
      step<1, 0>(s + 4);
      step<2, 1>(s + 5);
    }
    if (s < n_steps) step<0, 0>(s);
    if (s + 1 < n_steps) step<1, 1>(s + 1);
    if (s + 2 < n_steps) step<2, 0>(s + 2);
    if (s + 3 < n_steps) step<0, 1>(s + 3);
    if (s + 4 < n_steps) step<1, 0>(s + 4);
    if (wave < 4) barrier();
    wait_vm<0>();
  }
};

// silu(g) from e = exp(-|g|), which cannot overflow; the square of exp(-|g| / 2), so
// that it goes down through the subnormal floats as the exponential itself does
// not.  Rounded at most (12 + 2 |g|) times 2^-24.
__device__ __forceinline__ float silu(float g) {
  const float half = __builtin_amdgcn_exp2f(fabsf(g) * -0.72134752f);      // log2(e) / 2
  const float e = half * half, p = __builtin_amdgcn_rcpf(1.0f + e);
  return g * (g >= 0.0f ? p : e * p);
}

struct GemmParams {
  moe_gemm_mxfp4_args a;
  unsigned* next;          // [8] counters, NULL when the first tiles are all
};

// Columns of the result; a tile has 256 of them, or 128 where each is made of two
// rows of B.
template <bool GATED>
__device__ __forceinline__ Groups groups_of(const moe_gemm_mxfp4_args& a) {
  return {a.group_offsets, a.num_groups, a.total_rows, GATED ? a.n_out / 2 : a.n_out};
}
template <bool GATED>
constexpr int kWidth = GATED ? 128 : 256;

// The row of B behind column c of the result, in half h of a tile.
template <bool GATED>
__device__ __forceinline__ int row_of_b(int n0, int h, int r) {
  if (!GATED) return n0 + h * 128 + r;
  const int c = n0 + r;
  return (c >> 7) * 256 + h * 128 + (c & 127);
}
template <bool GATED>
__device__ __forceinline__ bool has_row_of_b(int cols, int h, int r) {
  return (GATED ? r : h * 128 + r) < cols;
}

template <int EPI, int L0, int L1, bool EXTRA = false>
__device__ __forceinline__ void gemm_tile(const moe_gemm_mxfp4_args& a, const TileAt& t, uint8_t* smem) {
  constexpr bool kGated = EPI == MOE_EPI_SWIGLU_MXFP4;
  // The lane goes through an asm statement here and behind the K loop, so that no
  // address is formed before its own part of the tile: kept across the K loop it would go
  // to scratch memory, whose loads wait for every copy in flight (32 groups of 288 rows:
  // 240 -> 195 us, gated 337 -> 195).
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int blocks = (a.k_dim + 31) / 32;
  const long long bq = mx_code_bytes(a.k_dim), be = mx_scale_bytes(a.k_dim);
  const int last = (blocks - 1) / kStepBlocks * kStepBlocks;
  constexpr int kScaleWavesA = L1 > 0 ? 4 : 2;
  Operand A, B;
  Scales S;
  {
    // load j of wave w fills rows 8 (w + 8 j) .. + 7 of a half tile
    const long long first = t.row0 + t.m0;
    auto source = [&](int r) -> long long {       // the row, relative to the operand's base
      return a.a_row_index ? clampi(a.a_row_index[first + r], 0, a.a_rows - 1) : r;
    };
    const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = h * 128 + 8 * (wave + 8 * j) + (lane >> 3);
        A.off[h][j] = r < t.m_rows && (h == 0 || L1 > 0) ? (uint32_t)(source(r) * a.lda) + chunk * 16 : kOut;
      }
    A.tail = last + chunk < blocks ? 0u : kOut;
    A.base = a.a_row_index ? a.a_q : a.a_q + first * a.lda;
    const long long rows = a.a_row_index ? a.a_rows : t.m_rows;
    A.bytes = (uint32_t)(rows * a.lda);
    S.a_base = a.a_row_index ? a.a_e : a.a_e + first * a.lde;
    S.a_bytes = (uint32_t)(rows * a.lde);
    A.extra = S.extra = kOut;
    if constexpr (EXTRA) {
      const int x = kTile + 8 * (wave & 3) + (lane >> 3), y = kTile + lane;
      if (x < t.m_rows) A.extra = (uint32_t)(source(x) * a.lda) + chunk * 16;
      if (y < t.m_rows) S.extra = (uint32_t)(source(y) * a.lde);
    }
    const int r = wave * 64 + lane;
    if (wave < kScaleWavesA) {
      S.base = S.a_base;
      S.bytes = S.a_bytes;
      S.at = wave * kWaveBytes;
      S.off = r < t.m_rows ? (uint32_t)(source(r) * a.lde) : kOut;
    }
  }
  {
    const int chunk = (lane & 7) ^ (((lane >> 4) & 1) | ((wave & 3) << 1));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * (wave + 8 * j) + (lane >> 3);
        B.off[h][j] = has_row_of_b<kGated>(t.cols, h, r) ? (uint32_t)(row_of_b<kGated>(t.n0, h, r) * bq) + chunk * 16 : kOut;
      }
    B.tail = last + chunk < blocks ? 0u : kOut;
    B.row_bytes = (uint32_t)bq;
    if constexpr (L1 > 0)
      B.off[0][0] = (uint32_t)(row_of_b<kGated>(t.n0, 0, 8 * wave + (lane >> 3)) * bq) + chunk * 16;
    B.base = a.b_q + (long long)t.g * a.n_out * bq;
    B.bytes = (uint32_t)(a.n_out * bq);
    if (wave >= kScaleWavesA) {
      const int w = min(wave - kScaleWavesA, 3), h = w >> 1, r = (w & 1) * 64 + lane;
      S.base = a.b_e + (long long)t.g * a.n_out * be;
      S.bytes = (uint32_t)(a.n_out * be);
      S.at = (kScaleWavesA + w) * kWaveBytes;
      S.off = has_row_of_b<kGated>(t.cols, h, r) ? (uint32_t)(row_of_b<kGated>(t.n0, h, r) * be) : kOut;
    }
  }
  typename std::conditional<(L1 > 0), Product<L0, L1, EXTRA>, ShortProduct<L0>>::type p(
      smem, wave, lane, (blocks + kStepBlocks - 1) / kStepBlocks, A, B, S);
  p.run();

  // A lane holds 8 consecutive columns of one row in each half of B.
  int l = lane;
  asm volatile("" : "+v"(l));
  const int wm = wave & 1, wn = wave >> 1, lk = l >> 4;
  auto put = [&](int subtile, const f32x4 (&acc)[2][2]) {
    const int r = (subtile + wm) * 16 + (l & 15);
    const long long row = t.row0 + t.m0 + r;
    if constexpr (kGated) {
      float h[8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = silu(acc[0][i >> 2][i & 3]) * acc[1][i >> 2][i & 3];
        m = max(m, __float_as_uint(h[i]) & 0x7FFFFFFFu);
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if (r >= t.m_rows || wn * 32 >= t.cols) return;
      const uint32_t byte = mx_scale_byte(m);
      const int block = (t.n0 >> 5) + wn, all = a.n_out / 64;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + row * a.ldo + block * 16 + lk * 4) = mx_encode(h, byte);
      uint8_t* e = a.out_e + row * mx_scale_bytes(a.n_out / 2);
      if (lk == 0) e[mx_scale_at(block)] = (uint8_t)byte;
      // blocks that are not there: the last one's lanes fill their piece
      if (block == all - 1)
        for (int b = all + lk; b < ((all + 15) & ~15); b += 4) e[mx_scale_at(b)] = (uint8_t)kMxOne;
    } else {
      if (r >= t.m_rows) return;
      const float s = a.row_scale ? a.row_scale[row] : 1.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = u * 128 + wn * 32 + lk * 8;
        if (c >= t.cols) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[u][i >> 2][i & 3] * s;
        const long long at = row * a.ldo + t.n0 + c;
        if constexpr (EPI == MOE_EPI_F32) Vec8<float>::store(static_cast<float*>(a.out) + at, v, t.cols - c);
        else Vec8<bf16_t>::store(static_cast<bf16_t*>(a.out) + at, v, t.cols - c);
      }
    }
  };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < (h ? L1 : L0); ++i) put(h * 8 + 2 * i, p.acc[h][i]);
  if constexpr (EXTRA) put(16, p.more);
}

template <int EPI>
__device__ __forceinline__ void short_tile(const moe_gemm_mxfp4_args& a, const TileAt& t, uint8_t* smem) {
  const int l0 = (t.m_rows + 31) / 32;
  if (l0 > 2) l0 > 3 ? gemm_tile<EPI, 4, 0>(a, t, smem) : gemm_tile<EPI, 3, 0>(a, t, smem);
  else l0 > 1 ? gemm_tile<EPI, 2, 0>(a, t, smem) : gemm_tile<EPI, 1, 0>(a, t, smem);
}

template <int EPI>
__global__ __launch_bounds__(kThreads, 2) void grouped_gemm_mxfp4_kernel(GemmParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool kGated = EPI == MOE_EPI_SWIGLU_MXFP4;
  const bool whole = (p.a.k_dim + 31) / 32 % kStepBlocks == 0;
  const int most = p.a.n_out < kLeastRows ? 128 / kUnit : whole ? kMostUnits : kMostUnits - 1;
  TileList<kWidth<kGated>, kThreads> list(groups_of<kGated>(p.a), smem + kLds, smem, p.next, most);
  TileAt t;
  for (int slot = blockIdx.x / kXcds; list.find(slot, t);) {
    const unsigned popped = list.pop();
    const int l1 = (t.m_rows - 128 + 31) / 32;
    if (t.m_rows > kTile) gemm_tile<EPI, 4, 4, true>(p.a, t, smem);
    else if (t.m_rows <= 128) short_tile<EPI>(p.a, t, smem);
    else if (l1 > 2) l1 > 3 ? gemm_tile<EPI, 4, 4>(p.a, t, smem) : gemm_tile<EPI, 4, 3>(p.a, t, smem);
    else l1 > 1 ? gemm_tile<EPI, 4, 2>(p.a, t, smem) : gemm_tile<EPI, 4, 1>(p.a, t, smem);
    if (!p.next) return;
    slot = list.publish(popped);      // and all waves are done with LDS
  }
}

template <int EPI>
__global__ __launch_bounds__(kThreads, 2) void grouped_gemm_mxfp4_stream_kernel(GemmParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr bool kGated = EPI == MOE_EPI_SWIGLU_MXFP4;
  // units of 16 columns, or of a block of the quantised result
  stream_tiles<kWidth<kGated>, kGated ? 32 : 16, kThreads>(groups_of<kGated>(p.a), smem,
                                                           [&](const TileAt& t) { short_tile<EPI>(p.a, t, smem); });
}

// Up to 64 rows a group on average the weights' stream decides.  32 groups of 4096 x 7168
// take, in the stream kernel and in row tiles: at 2 rows a group 89 and 98 us, at 48 104
// and 110, at 64 110 and 115, at 96 125 and 123, at 128 144 and 130, at 160 271 and 135; 33
// groups of 48 rows, which do not fill whole rounds of row tiles, 114 and 140.  The host
// knows the mean alone, and a group of hundreds of rows among small ones is
// streamed once for each 128 of them: 32 groups of 9 and one of 300 rows take 115 and
// 136 us or 123 and 126 on another card, 30 of 10 and three of 400 rows 147 and 141, one of 2112
// among 32 empty ones 70 and 65.  Worst are many groups: of 256, all of 64 rows 901 and 801 us, one
// of 16129 among single rows 1087 and 920, 32 of 512 among empty ones 541 and 273.
bool streams_weights(int num_groups, int total_rows) { return total_rows <= 64LL * num_groups; }

bool fits31(long long rows, long long bytes) { return rows == 0 || bytes < (1LL << 31) / rows; }

// Tiles of either kind of result (a gated one's are half as wide as B's).
long long tiles_of(int num_groups, int total_rows, int n_out) {
  return row_tiles(num_groups, total_rows, n_out < kLeastRows ? 128 : kTileRows) * ((n_out + 255LL) / 256);
}

}  // namespace

extern "C" size_t moe_grouped_gemm_mxfp4_workspace_bytes(int num_groups, int total_rows, int n_out, int k_dim) {
  (void)k_dim;
  if (num_groups < 1 || total_rows < 1 || n_out < 1 || streams_weights(num_groups, total_rows)) return 0;
  return counter_bytes(tiles_of(num_groups, total_rows, n_out));
}

extern "C" moe_status_t moe_grouped_gemm_mxfp4(const moe_gemm_mxfp4_args* args, void* ws, size_t ws_bytes,
                                               hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_gemm_mxfp4_args& a = *args;
  const bool gated = a.epilogue == MOE_EPI_SWIGLU_MXFP4;
  if (a.total_rows < 0 || a.n_out < 0 || a.k_dim < 0 || a.num_groups < 1 || a.a_rows < 0 ||
      a.lda < mx_code_bytes(a.k_dim) || a.lda % 16 || a.lde < mx_scale_bytes(a.k_dim) || a.lde % 16 ||
      a.ldo < (gated ? a.n_out / 4 : a.n_out) || (gated && (a.n_out % 256 || a.ldo % 4)))
    return MOE_ERR_SHAPE;
  if (a.num_groups > kMaxGroups || (a.epilogue != MOE_EPI_BF16 && a.epilogue != MOE_EPI_F32 && !gated) ||
      (gated && a.row_scale) || !fits31(a.n_out, a.k_dim) || !fits31(a.n_out, mx_code_bytes(a.k_dim)) ||
      !fits31(kTile + kUnit, a.lda) || !fits31(kTile + kUnit, a.lde))
    return MOE_ERR_UNSUPPORTED;
  if (a.a_row_index && (!fits31(a.a_rows, a.lda) || !fits31(a.a_rows, a.lde))) return MOE_ERR_UNSUPPORTED;
  if (!a.a_row_index && a.a_rows < a.total_rows) return MOE_ERR_SHAPE;
  if (a.total_rows == 0 || a.n_out == 0) return MOE_OK;
  if (a.a_rows == 0) return MOE_ERR_SHAPE;
  if (!a.group_offsets || !a.out || (gated && !a.out_e) || (a.k_dim > 0 && (!a.a_q || !a.a_e || !a.b_q || !a.b_e)))
    return MOE_ERR_NULL;
  if (!aligned16(a.a_q) || !aligned16(a.a_e) || !aligned16(a.b_q) || !aligned16(a.b_e) ||
      !element_aligned(a.out, a.epilogue == MOE_EPI_BF16 ? MOE_BF16 : MOE_F32) || (gated && !aligned16(a.out_e)))
    return MOE_ERR_ALIGN;
  const size_t need = moe_grouped_gemm_mxfp4_workspace_bytes(a.num_groups, a.total_rows, a.n_out, a.k_dim);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return MOE_ERR_ALIGN;
  if (tiles_of(a.num_groups, a.total_rows, a.n_out) > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (moe_status_t s = check_device()) return s;
  const int grid = places() * kXcds;
  const GemmParams p{a, need ? static_cast<unsigned*>(ws) : nullptr};
  if (need) {
    hipLaunchKernelGGL(tile_counters_kernel, dim3(1), dim3(64), 0, stream, p.next, (unsigned)grid / kXcds);
    if (moe_status_t s = launch_status()) return s;
  }
  static void (*const table[2][3])(GemmParams) = {
      {grouped_gemm_mxfp4_kernel<MOE_EPI_BF16>, grouped_gemm_mxfp4_kernel<MOE_EPI_F32>,
       grouped_gemm_mxfp4_kernel<MOE_EPI_SWIGLU_MXFP4>},
      {grouped_gemm_mxfp4_stream_kernel<MOE_EPI_BF16>, grouped_gemm_mxfp4_stream_kernel<MOE_EPI_F32>,
       grouped_gemm_mxfp4_stream_kernel<MOE_EPI_SWIGLU_MXFP4>}};
  static std::atomic<uint64_t> lds_set[2][3] = {};
  const int kind = gated ? 2 : a.epilogue == MOE_EPI_F32 ? 1 : 0;
  const bool few = streams_weights(a.num_groups, a.total_rows);
  const int lds = kLds + kListBytes;
  if (moe_status_t st = allow_dynamic_lds(reinterpret_cast<const void*>(table[few][kind]), lds, lds_set[few][kind]))
    return st;
  hipLaunchKernelGGL(table[few][kind], dim3(grid), dim3(kThreads), lds, stream, p);
  return launch_status();
}
