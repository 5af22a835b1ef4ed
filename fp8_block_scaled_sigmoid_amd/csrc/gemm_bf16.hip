// Grouped bf16 products of the experts over ragged row groups:
//   forward and input gradient   C[r, c] = s[r] sum_k A[src(r), k] B[g](c, k)
//   weight gradient              dW[g][n, k] = sum_{r in g} A[srcA(r), n] B[srcB(r), k]
// bf16 operands, float sums (v_mfma_f32_16x16x32_bf16), bf16 or float results.
#include "common.h"

namespace {

using namespace moe;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxGroups = 1025;
constexpr int kThreads = 256;
constexpr int BM = 128, BN = 128, BK = 32, kPad = 8;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// The group and the row tile inside it of row tile `want` of the list of all
// groups' row tiles, found by every thread from the device-side offsets.
__device__ __forceinline__ bool find_row_tile(const int32_t* offsets, int G, int total, int tile,
                                              int want, int* s_scan, int& g, int& m, int& row0,
                                              int& rows) {
  int base = 0;
  for (int g0 = 0; g0 < G; g0 += kThreads) {
    const int gi = g0 + threadIdx.x;
    int lo = 0, n = 0;
    if (gi < G) {
      lo = clampi(offsets[gi], 0, total);
      n = clampi(offsets[gi + 1], 0, total) - lo;
      if (n < 0) n = 0;
    }
    const int tiles = (n + tile - 1) / tile;
    s_scan[threadIdx.x] = tiles;
    __syncthreads();
    int before = base, all = base;
    for (int i = 0; i < kThreads; ++i) {
      if (i < (int)threadIdx.x) before += s_scan[i];
      all += s_scan[i];
    }
    __syncthreads();
    if (want >= before && want < before + tiles) {
      s_scan[kThreads] = gi;
      s_scan[kThreads + 1] = want - before;
      s_scan[kThreads + 2] = lo;
      s_scan[kThreads + 3] = n;
    }
    __syncthreads();
    if (want < all) {
      g = s_scan[kThreads];
      m = s_scan[kThreads + 1];
      row0 = s_scan[kThreads + 2];
      rows = s_scan[kThreads + 3];
      return true;
    }
    base = all;
  }
  return false;
}

struct GemmParams {
  moe_gemm_bf16_args a;
};

__device__ __forceinline__ void store_out(void* out, moe_dtype_t dt, long long at, float v) {
  if (dt == MOE_F32) static_cast<float*>(out)[at] = v;
  else static_cast<__bf16*>(out)[at] = (__bf16)v;
}

template <bool KN>
__global__ __launch_bounds__(kThreads) void grouped_gemm_bf16_kernel(GemmParams p) {
  __shared__ __align__(16) uint16_t sa[BM][BK + kPad], sb[BN][BK + kPad];
  __shared__ int s_scan[kThreads + 4];
  const moe_gemm_bf16_args& a = p.a;
  int g, mt, row0, rows;
  if (!find_row_tile(a.group_offsets, a.num_groups, a.total_rows, BM, blockIdx.x, s_scan, g, mt, row0, rows))
    return;
  const int m0 = mt * BM, n0 = blockIdx.y * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave & 1, wn = wave >> 1;
  const uint16_t* A = static_cast<const uint16_t*>(a.a);
  const uint16_t* B = static_cast<const uint16_t*>(a.b) + (long long)g * a.n_out * a.k_dim;
  f32x4 acc[4][4] = {};
  const int K = a.k_dim, N = a.n_out;
  for (int k0 = 0; k0 < K; k0 += BK) {
    for (int i = tid; i < BM * BK / 8; i += kThreads) {
      const int r = i / (BK / 8), c = (i % (BK / 8)) * 8;
      u32x4 v = {0, 0, 0, 0};
      if (m0 + r < rows && k0 + c < K) {
        int src = row0 + m0 + r;
        if (a.a_row_index) src = a.a_row_index[src];
        src = clampi(src, 0, a.a_rows - 1);
        v = *reinterpret_cast<const u32x4*>(A + (long long)src * a.lda + k0 + c);
      }
      *reinterpret_cast<u32x4*>(&sa[r][c]) = v;
    }
    if constexpr (!KN) {
      for (int i = tid; i < BN * BK / 8; i += kThreads) {
        const int r = i / (BK / 8), c = (i % (BK / 8)) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (n0 + r < N && k0 + c < K) v = *reinterpret_cast<const u32x4*>(B + (long long)(n0 + r) * K + k0 + c);
        *reinterpret_cast<u32x4*>(&sb[r][c]) = v;
      }
    } else {
      for (int i = tid; i < BK * BN / 8; i += kThreads) {
        const int r = i / (BN / 8), c = (i % (BN / 8)) * 8;
        u32x4 v = {0, 0, 0, 0};
        if (k0 + r < K && n0 + c < N) v = *reinterpret_cast<const u32x4*>(B + (long long)(k0 + r) * N + n0 + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) sb[c + j][r] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
      }
    }
    __syncthreads();
    bf16x8 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i] = *reinterpret_cast<const bf16x8*>(&sa[wm * 64 + i * 16 + (lane & 15)][(lane >> 4) * 8]);
      fb[i] = *reinterpret_cast<const bf16x8*>(&sb[wn * 64 + i * 16 + (lane & 15)][(lane >> 4) * 8]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = m0 + wm * 64 + i * 16 + (lane >> 4) * 4 + v;
      if (r < rows) {
        const float s = a.row_scale ? a.row_scale[row0 + r] : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = n0 + wn * 64 + j * 16 + (lane & 15);
          if (c < N) store_out(a.out, a.out_dtype, (long long)(row0 + r) * a.ldo + c, acc[i][j][v] * s);
        }
      }
    }
}

__global__ __launch_bounds__(kThreads) void grouped_wgrad_bf16_kernel(moe_wgrad_bf16_args a) {
  __shared__ __align__(16) uint16_t sa[BM][BK + kPad], sb[BN][BK + kPad];
  const int g = blockIdx.z;
  const int row0 = clampi(a.group_offsets[g], 0, a.total_rows);
  const int end = clampi(a.group_offsets[g + 1], 0, a.total_rows);
  const int m0 = blockIdx.x * BM, n0 = blockIdx.y * BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave & 1, wn = wave >> 1;
  const uint16_t* A = static_cast<const uint16_t*>(a.a);
  const uint16_t* B = static_cast<const uint16_t*>(a.b);
  f32x4 acc[4][4] = {};
  for (int r0 = row0; r0 < end; r0 += BK) {
    for (int i = tid; i < BK * BM / 8; i += kThreads) {
      const int r = i / (BM / 8), c = (i % (BM / 8)) * 8;
      u32x4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
      if (r0 + r < end) {
        int ra = r0 + r, rb = r0 + r;
        if (a.a_row_index) ra = a.a_row_index[ra];
        if (a.b_row_index) rb = a.b_row_index[rb];
        ra = clampi(ra, 0, a.a_rows - 1);
        rb = clampi(rb, 0, a.b_rows - 1);
        if (m0 + c < a.n) va = *reinterpret_cast<const u32x4*>(A + (long long)ra * a.lda + m0 + c);
        if (n0 + c < a.k) vb = *reinterpret_cast<const u32x4*>(B + (long long)rb * a.ldb + n0 + c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sa[c + j][r] = (uint16_t)(va[j >> 1] >> (16 * (j & 1)));
        sb[c + j][r] = (uint16_t)(vb[j >> 1] >> (16 * (j & 1)));
      }
    }
    __syncthreads();
    bf16x8 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i] = *reinterpret_cast<const bf16x8*>(&sa[wm * 64 + i * 16 + (lane & 15)][(lane >> 4) * 8]);
      fb[i] = *reinterpret_cast<const bf16x8*>(&sb[wn * 64 + i * 16 + (lane & 15)][(lane >> 4) * 8]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = m0 + wm * 64 + i * 16 + (lane >> 4) * 4 + v;
      if (r < a.n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = n0 + wn * 64 + j * 16 + (lane & 15);
          if (c < a.k) {
            const long long at = ((long long)g * a.n + r) * a.k + c;
            float t = acc[i][j][v];
            if (a.accumulate)
              t += a.out_dtype == MOE_F32 ? static_cast<const float*>(a.out)[at]
                                          : (float)static_cast<const __bf16*>(a.out)[at];
            store_out(a.out, a.out_dtype, at, t);
          }
        }
      }
    }
}

bool valid_dt(moe_dtype_t d) { return d == MOE_BF16 || d == MOE_F32; }
// element rows that 32-bit byte offsets of a gathered operand can reach
bool fits31(long long rows, long long ld) { return rows * ld * 2 < (1LL << 31); }

}  // namespace

extern "C" moe_status_t moe_grouped_gemm_bf16(const moe_gemm_bf16_args* args, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_gemm_bf16_args& a = *args;
  if (a.total_rows < 0 || a.n_out < 0 || a.k_dim < 0 || a.n_out % 8 || a.k_dim % 8 ||
      a.num_groups < 1 || a.lda < a.k_dim || a.lda % 8 || a.ldo < a.n_out || a.ldo % 8 || a.a_rows < 0)
    return MOE_ERR_SHAPE;
  if (a.num_groups > kMaxGroups || !valid_dt(a.out_dtype) ||
      (a.b_layout != MOE_B_NK && a.b_layout != MOE_B_KN) ||
      (long long)a.n_out * a.k_dim * 2 >= (1LL << 31))
    return MOE_ERR_UNSUPPORTED;
  if (a.a_row_index ? !fits31(a.a_rows, a.lda) : a.a_rows < a.total_rows)
    return a.a_row_index ? MOE_ERR_UNSUPPORTED : MOE_ERR_SHAPE;
  if (a.total_rows == 0 || a.n_out == 0) return MOE_OK;
  if (a.a_rows == 0) return MOE_ERR_SHAPE;
  if (!a.group_offsets || !a.out || (a.k_dim > 0 && (!a.a || !a.b))) return MOE_ERR_NULL;
  if (!aligned16(a.a) || !aligned16(a.b) || !aligned16(a.out)) return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  GemmParams p{a};
  const long long tiles = (long long)a.total_rows / BM + (a.num_groups < a.total_rows ? a.num_groups : a.total_rows);
  const dim3 grid((unsigned)tiles, (unsigned)((a.n_out + BN - 1) / BN));
  if (a.b_layout == MOE_B_NK)
    hipLaunchKernelGGL(grouped_gemm_bf16_kernel<false>, grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(grouped_gemm_bf16_kernel<true>, grid, dim3(kThreads), 0, stream, p);
  return launch_status();
}

extern "C" size_t moe_grouped_wgrad_bf16_workspace_bytes(int num_groups, int total_rows, int n,
                                                         int k) {
  return 0;
}

extern "C" moe_status_t moe_grouped_wgrad_bf16(const moe_wgrad_bf16_args* args, void* ws,
                                               size_t ws_bytes, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_wgrad_bf16_args& a = *args;
  if (a.total_rows < 0 || a.n < 0 || a.k < 0 || a.n % 8 || a.k % 8 || a.num_groups < 1 ||
      a.lda < a.n || a.lda % 8 || a.ldb < a.k || a.ldb % 8 || a.a_rows < 0 || a.b_rows < 0)
    return MOE_ERR_SHAPE;
  if (a.num_groups > kMaxGroups || !valid_dt(a.out_dtype)) return MOE_ERR_UNSUPPORTED;
  if ((a.a_row_index && !fits31(a.a_rows, a.lda)) || (a.b_row_index && !fits31(a.b_rows, a.ldb)))
    return MOE_ERR_UNSUPPORTED;
  if ((!a.a_row_index && a.a_rows < a.total_rows) || (!a.b_row_index && a.b_rows < a.total_rows) ||
      (a.total_rows > 0 && (a.a_rows == 0 || a.b_rows == 0)))
    return MOE_ERR_SHAPE;
  if (a.n == 0 || a.k == 0) return MOE_OK;
  if (!a.group_offsets || !a.out || (a.total_rows > 0 && (!a.a || !a.b))) return MOE_ERR_NULL;
  if (!aligned16(a.a) || !aligned16(a.b) || !aligned16(a.out)) return MOE_ERR_ALIGN;
  if (ws_bytes < moe_grouped_wgrad_bf16_workspace_bytes(a.num_groups, a.total_rows, a.n, a.k))
    return MOE_ERR_WORKSPACE;
  if (moe_status_t s = check_device()) return s;
  const dim3 grid((unsigned)((a.n + BM - 1) / BM), (unsigned)((a.k + BN - 1) / BN), (unsigned)a.num_groups);
  hipLaunchKernelGGL(grouped_wgrad_bf16_kernel, grid, dim3(kThreads), 0, stream, a);
  return launch_status();
}
