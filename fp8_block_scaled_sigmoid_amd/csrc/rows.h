// Helpers of the training operators: vector types, and for the row-wise kernels
// (block norms, gated activation, gradient clipping) bf16 and float rows at any
// element alignment, eight elements at a time, held as loaded until they are used.
#pragma once

#include "common.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ float to_float(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }
// round to nearest even; NaN stays NaN
__device__ __forceinline__ void from_float(float v, bf16_t& o) {
  o.bits = __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void from_float(float v, float& o) { o = v; }

// Eight consecutive elements of a row.  gfx950 loads and stores 16 bytes at
// any element alignment, so rows of odd widths and strides take the same path;
// the vector that crosses the end of a row goes element by element.
template <typename E>
struct Vec8;

template <>
struct Vec8<bf16_t> {
  typedef u32x4 __attribute__((aligned(2))) raw_t;
  u32x4 w;
  __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const bf16_t* p, int valid) {
    if (valid >= 8) {
      w = *reinterpret_cast<const raw_t*>(p);
    } else {
      uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < valid) t[i >> 1] |= (uint32_t)p[i].bits << (16 * (i & 1));
      w = u32x4{t[0], t[1], t[2], t[3]};
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store(bf16_t* p, const float (&v)[8], int valid) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
    const u32x4 w = __builtin_bit_cast(u32x4, o);
    if (valid >= 8) {
      *reinterpret_cast<raw_t*>(p) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < valid) p[i].bits = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
};

template <>
struct Vec8<float> {
  typedef f32x4 __attribute__((aligned(4))) raw_t;
  f32x4 a, b;
  __device__ __forceinline__ void zero() { a = b = f32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const float* p, int valid) {
    if (valid >= 8) {
      a = *reinterpret_cast<const raw_t*>(p);
      b = *reinterpret_cast<const raw_t*>(p + 4);
    } else {
      float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < valid) t[i] = p[i];
      a = f32x4{t[0], t[1], t[2], t[3]};
      b = f32x4{t[4], t[5], t[6], t[7]};
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8], int valid) {
    if (valid >= 8) {
      *reinterpret_cast<raw_t*>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<raw_t*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < valid) p[i] = v[i];
    }
  }
};

// Sum over the 16 lanes of each DPP row, in every lane: exchanges with lane ^ 1,
// ^ 2, then the mirrored half and the mirrored row.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row16_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  return dpp_add<0x140>(v);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// Sum over the wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

}  // namespace moe

namespace moe {
inline bool element_aligned(const void* p, moe_dtype_t dt) {
  return (reinterpret_cast<uintptr_t>(p) & (dt == MOE_F32 ? 3u : 1u)) == 0;
}
inline bool valid_dtype(moe_dtype_t dt) { return dt == MOE_BF16 || dt == MOE_F32; }
}  // namespace moe
