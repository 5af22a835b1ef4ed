// Device helpers of the microscaled 4-bit format (MXFP4): 32 values of a row share
// a scale 2^(byte - 127), each a code of 4 bits.  gfx950 converts both ways with
// the block's scale as an operand (a float whose exponent field is the scale
// byte; byte 0 is 2^-127 there too) and rounds to nearest even, saturating at 6,
// exactly as the format asks: checked over every scale, with ties and
// subnormals, on the device.
#pragma once

#include "rows.h"

namespace moe {

constexpr uint32_t kMxOne = 127;      // the scale byte of 2^0
constexpr uint32_t kMxNan = 255;

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Bytes of a row of codes, and of scales.
__host__ __device__ __forceinline__ long long mx_code_bytes(long long cols) { return (cols + 31) / 32 * 16; }
__host__ __device__ __forceinline__ long long mx_scale_bytes(long long cols) { return (cols + 511) / 512 * 16; }
// Where block b's scale stands in its row.
__device__ __forceinline__ int mx_scale_at(int b) { return (b & ~15) + 4 * (b & 3) + ((b & 15) >> 2); }

// The scale byte of a block whose largest |x| has these bits: the exponent of the
// largest value less that of the largest code (6 = 1.5 * 2^2).  bits >> 23 is
// floor(log2) + 127, or 0 below 2^-126, where the byte is 0 either way.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t bits) {
  const uint32_t exponent = bits >> 23;
  if (exponent == 255) return kMxNan;
  if (bits == 0) return kMxOne;
  return exponent > 2 ? exponent - 2 : 0;
}
__device__ __forceinline__ float mx_scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes, value i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t mx_encode(const float (&v)[8], uint32_t byte) {
  if (byte == kMxNan) return 0;
  const float s = mx_scale_operand(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}
__device__ __forceinline__ void mx_decode(uint32_t w, uint32_t byte, float (&v)[8]) {
  const float s = mx_scale_operand(byte);
  f32x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = byte == kMxNan ? __uint_as_float(0x7FC00000u) : p[i >> 1][i & 1];
}

// Largest of a value over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
  return v > o ? v : o;
}

}  // namespace moe
