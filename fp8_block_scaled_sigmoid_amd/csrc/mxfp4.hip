// Quantiser and reader of the microscaled 4-bit format (include/moe_fp8.h gives
// the layout): along rows, along columns with the result turned, and back.
//
// Memory bounds all of them: 2 (4) bytes a value in, 0.53 out, and 2 more where
// the values are wanted.  In the row kernels a wave takes pieces of 512 columns, 8
// a lane, so that a quad of lanes owns a block and the piece's scales are 16
// bytes.
//
// Measured at 8192 x 7168 bf16: with the values 38 us (266 MB, 7.0 TB/s: above a
// copy's 4.9, so part of it stays in caches), codes and scales alone 30; 4 x 4096 x 7168
// turned 74 us (54 at best, 297 MB), read back 58 (297 MB).  One token: 2.3 us.
#include "mx.h"

namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kPiece = 512;             // columns of a wave

__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Items, a wave each, go on along a launch's second dimension from 2^24 on (2^22
// workgroups, 2^30 threads; a dimension holds fewer than 2^32).
constexpr uint32_t kMostGroups = 1u << 22;
__device__ __forceinline__ uint32_t item_of_wave() {
  return (blockIdx.y * kMostGroups + blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
}

// One wave per piece of a row.
template <typename E>
__global__ __launch_bounds__(kThreads) void quant_1x32_kernel(const E* x, uint32_t items, uint32_t pieces, int rows,
                                                               int cols, long long ld, int interleave, uint8_t* q,
                                                               uint8_t* e, bf16_t* values) {
  const uint32_t item = item_of_wave();
  if (item >= items) return;
  const int lane = threadIdx.x & 63;
  const uint32_t row = item / pieces, piece = item - row * pieces;
  const int c = (int)piece * kPiece + lane * 8;
  Vec8<E> in;
  in.zero();
  if (c < cols) in.load(x + row * ld + c, cols - c);
  float v[8];
  in.get(v);
  const uint32_t byte = mx_scale_byte(quad_max(largest(v)));
  const uint32_t w = mx_encode(v, byte);
  long long to = row;
  if (interleave) {
    const int r = (int)(row % (uint32_t)rows), block = r >> 7, half = rows >> 8;
    to += ((block < half ? 2 * block : 2 * (block - half) + 1) - block) * 128;
  }
  const bool there = (c >> 5) <= ((cols - 1) >> 5);      // the block holds columns
  if (there) *reinterpret_cast<uint32_t*>(q + to * mx_code_bytes(cols) + (c >> 1)) = w;
  if ((lane & 3) == 0)
    e[to * mx_scale_bytes(cols) + mx_scale_at((int)piece * 16 + (lane >> 2))] = (uint8_t)(there ? byte : kMxOne);
  if (values && c < cols) {
    mx_decode(w, byte, v);
    Vec8<bf16_t>::store(values + (long long)row * cols + c, v, cols - c);
  }
}

// Tiles of 256 rows and 64 columns; a wave takes 32 rows, a row of blocks.  Lane
// (r, c) holds rows 4 r .. 4 r + 3 of columns 8 c .. 8 c + 7, so a column's block is
// eight lanes (c, c + 8, ...), each with two bytes of codes.  Codes and scales go
// through LDS and leave as 128 bytes and 4 x 2 bytes a column (a lane with a whole
// column of a block, whose 16 bytes leave by themselves: 168 us against 74 at
// 4 x 4096 x 7168).
constexpr int kTurnThreads = 512, kTurnRows = 256, kTurnCols = 64;
constexpr int kTurnStride = kTurnRows / 2 + 8;      // bytes between columns in LDS, off the banks' period

// The largest over the lanes that differ in bits 3 to 5.
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false);      // lane ^ 8
  v = v > o ? v : o;
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

template <typename E>
__global__ __launch_bounds__(kTurnThreads) void quant_32x1_kernel(const E* x, int rows, int cols, long long ld,
                                                                   uint8_t* q, uint8_t* e) {
  __shared__ __align__(16) uint8_t codes[kTurnCols * kTurnStride];
  __shared__ uint8_t scales[kTurnCols][8];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int col0 = (int)blockIdx.x * kTurnCols, block0 = (int)blockIdx.y * (kTurnRows / 32);
  const int blocks = (rows + 31) / 32;
  {
    const int c = (lane & 7) * 8, row = (block0 + wave) * 32 + (lane >> 3) * 4;
    const E* at = x + ((long long)blockIdx.z * rows + row) * ld + col0 + c;
    Vec8<E> in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      in[i].zero();
      if (row + i < rows && col0 + c < cols) in[i].load(at + i * ld, cols - col0 - c);
    }
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i].get(v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
      const uint32_t byte = mx_scale_byte(column_max(m));
      const float s = mx_scale_operand(byte);
      uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0][j], v[1][j], s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2][j], v[3][j], s, 1);
      if (byte == kMxNan) w = 0;
      *reinterpret_cast<uint16_t*>(codes + (c + j) * kTurnStride + wave * 16 + (lane >> 3) * 2) = (uint16_t)w;
      // a block that is not there has scale 1, as a block of zeros has
      if (lane < 8) scales[c + j][wave] = (uint8_t)byte;
    }
  }
  __syncthreads();
  {
    const int c = tid >> 3, b = tid & 7;
    const long long to = (long long)blockIdx.z * cols + col0 + c;
    if (col0 + c < cols && block0 + b < blocks) {
      const uint2* from = reinterpret_cast<const uint2*>(codes + c * kTurnStride + b * 16);
      const uint2 lo = from[0], hi = from[1];
      *reinterpret_cast<u32x4*>(q + to * mx_code_bytes(rows) + (block0 + b) * 16) = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
  if (tid < kTurnCols * 4) {        // blocks b and b + 4 of a column are neighbours
    const int c = tid >> 2, b = tid & 3;
    if (col0 + c < cols) {
      const long long to = (long long)blockIdx.z * cols + col0 + c;
      *reinterpret_cast<uint16_t*>(e + to * mx_scale_bytes(rows) + mx_scale_at(block0 + b)) =
          (uint16_t)(scales[c][b] | scales[c][b + 4] << 8);
    }
  }
}

template <typename E>
__global__ __launch_bounds__(kThreads) void dequant_1x32_kernel(const uint8_t* q, const uint8_t* e, uint32_t items,
                                                                 uint32_t pieces, int cols, E* out, long long ldo) {
  const uint32_t item = item_of_wave();
  if (item >= items) return;
  const int lane = threadIdx.x & 63;
  const uint32_t row = item / pieces, piece = item - row * pieces;
  const int c = (int)piece * kPiece + lane * 8;
  if (c >= cols) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + row * mx_code_bytes(cols) + (c >> 1));
  const uint32_t byte = e[row * mx_scale_bytes(cols) + mx_scale_at((int)piece * 16 + (lane >> 2))];
  float v[8];
  mx_decode(w, byte, v);
  Vec8<E>::store(out + row * ldo + c, v, cols - c);
}

// Workgroups for work items of a wave each.
dim3 grid_of(long long items) {
  const long long groups = (items + kThreads / 64 - 1) / (kThreads / 64);
  if (groups <= kMostGroups) return dim3((unsigned)groups);
  return dim3(kMostGroups, (unsigned)((groups + kMostGroups - 1) / kMostGroups));
}
// Items are counted in 31 bits.
bool fits(long long rows, long long pieces) {
  return rows < (1LL << 31) && (rows == 0 || pieces < (1LL << 31) / rows);
}

}  // namespace

extern "C" moe_status_t mxfp4_quant_1x32(const void* x, moe_dtype_t dt, int batch, int rows, int cols, long long ld,
                                         int interleave_gate_up, uint8_t* q, uint8_t* e, void* values_bf16,
                                         hipStream_t stream) {
  if (batch < 0 || rows < 0 || cols < 0 || ld < cols) return MOE_ERR_SHAPE;
  if (interleave_gate_up && rows % 256) return MOE_ERR_SHAPE;
  const long long all = (long long)batch * rows, pieces = (cols + 511LL) / 512;
  if (!valid_dtype(dt) || (interleave_gate_up && values_bf16) || !fits(all, pieces)) return MOE_ERR_UNSUPPORTED;
  if (all == 0 || cols == 0) return MOE_OK;
  if (!x || !q || !e) return MOE_ERR_NULL;
  if (!element_aligned(x, dt) || !aligned16(q) || !aligned16(e) || !element_aligned(values_bf16, MOE_BF16))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const long long items = all * pieces;
  const dim3 grid = grid_of(items), block(kThreads);
  bf16_t* values = static_cast<bf16_t*>(values_bf16);
  if (dt == MOE_F32)
    hipLaunchKernelGGL(quant_1x32_kernel<float>, grid, block, 0, stream, static_cast<const float*>(x), (uint32_t)items,
                       (uint32_t)pieces, rows, cols, ld, interleave_gate_up, q, e, values);
  else
    hipLaunchKernelGGL(quant_1x32_kernel<bf16_t>, grid, block, 0, stream, static_cast<const bf16_t*>(x),
                       (uint32_t)items, (uint32_t)pieces, rows, cols, ld, interleave_gate_up, q, e, values);
  return launch_status();
}

extern "C" moe_status_t mxfp4_quant_32x1(const void* x, moe_dtype_t dt, int batch, int rows, int cols, long long ld,
                                         uint8_t* q, uint8_t* e, hipStream_t stream) {
  if (batch < 0 || rows < 0 || cols < 0 || ld < cols) return MOE_ERR_SHAPE;
  const long long all = (long long)batch * cols, pieces = (rows + 511LL) / 512;
  if (!valid_dtype(dt) || !fits(all, pieces) || !fits((long long)batch * rows, 1)) return MOE_ERR_UNSUPPORTED;
  if (all == 0 || rows == 0) return MOE_OK;
  if (!x || !q || !e) return MOE_ERR_NULL;
  if (!element_aligned(x, dt) || !aligned16(q) || !aligned16(e)) return MOE_ERR_ALIGN;
  if (pieces * 2 > 65535 || batch > 65535 || cols > (1 << 28)) return MOE_ERR_UNSUPPORTED;      // a launch's size
  if (moe_status_t s = check_device()) return s;
  const dim3 grid((unsigned)((cols + 63LL) / kTurnCols), (unsigned)(pieces * 2), (unsigned)batch), block(kTurnThreads);
  if (dt == MOE_F32)
    hipLaunchKernelGGL(quant_32x1_kernel<float>, grid, block, 0, stream, static_cast<const float*>(x), rows, cols, ld, q,
                       e);
  else
    hipLaunchKernelGGL(quant_32x1_kernel<bf16_t>, grid, block, 0, stream, static_cast<const bf16_t*>(x), rows, cols, ld,
                       q, e);
  return launch_status();
}

extern "C" moe_status_t mxfp4_dequant_1x32(const uint8_t* q, const uint8_t* e, int rows, int cols,
                                           moe_dtype_t out_dtype, void* out, long long ldo, hipStream_t stream) {
  if (rows < 0 || cols < 0 || ldo < cols) return MOE_ERR_SHAPE;
  const long long pieces = (cols + 511LL) / 512;
  if (!valid_dtype(out_dtype) || !fits(rows, pieces)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!q || !e || !out) return MOE_ERR_NULL;
  if (!aligned16(q) || !aligned16(e) || !element_aligned(out, out_dtype)) return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const long long items = (long long)rows * pieces;
  const dim3 grid = grid_of(items), block(kThreads);
  if (out_dtype == MOE_F32)
    hipLaunchKernelGGL(dequant_1x32_kernel<float>, grid, block, 0, stream, q, e, (uint32_t)items, (uint32_t)pieces, cols,
                       static_cast<float*>(out), ldo);
  else
    hipLaunchKernelGGL(dequant_1x32_kernel<bf16_t>, grid, block, 0, stream, q, e, (uint32_t)items, (uint32_t)pieces,
                       cols, static_cast<bf16_t*>(out), ldo);
  return launch_status();
}
