// The experts' gated activation in bf16 or float, and its backward pass.
//
//   h = silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g)),  a = [g | u]
// Backward of w h with respect to g, u and w (w the row's combine gate, dh the
// gradient of the expert row before the gate):
//   dg = w dh u (s + silu(g) (1 - s)),  du = w dh silu(g),  dw = sum_c h dh
// and w h, the rows that the weight gradient of the second product reads.
//
// Memory bounds both: 3 values an element pair forward (two read, one written),
// 6 backward.  At 73728 x 2048 in bf16 the backward pass moves 1.81 GB in 317 us,
// 5.7 TB/s, the forward pass 0.91 GB in 194 to 200 us, 4.6 TB/s (a large copy: 4.8); the
// forward kernel takes 2.8 us at 9 x 2048.
#include "rows.h"

namespace {

using namespace moe;

// s, 1 - s and silu(g), from e = exp(-|g|), which cannot overflow: s is 1 / (1 + e)
// for g >= 0 and e / (1 + e) below, 1 - s the other one of the two.  silu(g) stays
// a float down to g = -108, and times a large u it counts.
__device__ __forceinline__ void sigmoid_silu(float g, float& s, float& rest, float& silu) {
  const float e = expf(-fabsf(g)), p = 1.0f / (1.0f + e), q = e * p;
  s = g >= 0.0f ? p : q;
  rest = g >= 0.0f ? q : p;
  silu = g * s;
}

// One thread per vector of 8 columns, rows one behind the other.
template <typename E>
__global__ __launch_bounds__(256) void swiglu_kernel(const E* a, long long lda, uint32_t items,
                                                      int vecs, int I, E* h, long long ldh) {
  const uint32_t item = blockIdx.x * 256u + threadIdx.x;
  if (item >= items) return;
  const uint32_t row = item / (uint32_t)vecs;
  const int c = (int)(item - row * (uint32_t)vecs) * 8;
  Vec8<E> gv, uv;
  gv.load(a + row * lda + c, I - c);
  uv.load(a + row * lda + I + c, I - c);
  float g[8], u[8];
  gv.get(g), uv.get(u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float s, rest, silu;
    sigmoid_silu(g[j], s, rest, silu);
    g[j] = silu * u[j];
  }
  Vec8<E>::store(h + row * ldh + c, g, I - c);
}

struct BwdParams {
  const void *a, *dh;
  const float* row_gate;
  void *da, *hg;
  float* dgate;
  long long lda, lddh, ldda, ldhg;
  int R, I, wpr;       // wpr: waves that share a row (1, 2 or 4 of a workgroup's 4)
};

template <typename E>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(BwdParams p) {
  __shared__ float red[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave / p.wpr, first = grp * p.wpr;
  const long long row = (long long)blockIdx.x * (4 / p.wpr) + grp;
  const bool live = row < p.R;
  float sum = 0.0f;
  if (live) {
    const E* a = static_cast<const E*>(p.a) + row * p.lda;
    const E* dh = static_cast<const E*>(p.dh) + row * p.lddh;
    const float w = p.row_gate ? p.row_gate[row] : 1.0f;
    for (int c = (tid - first * 64) * 8; c < p.I; c += p.wpr * 512) {
      Vec8<E> gv, uv, dv;
      gv.load(a + c, p.I - c);
      uv.load(a + p.I + c, p.I - c);
      dv.load(dh + c, p.I - c);
      float g[8], u[8], d[8], hg[8];
      gv.get(g), uv.get(u), dv.get(d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float s, rest, silu;
        sigmoid_silu(g[j], s, rest, silu);
        const float h = silu * u[j], wd = w * d[j];
        sum = __builtin_fmaf(h, d[j], sum);
        hg[j] = w * h;
        g[j] = wd * u[j] * __builtin_fmaf(silu, rest, s);
        u[j] = wd * silu;
      }
      E* da = static_cast<E*>(p.da) + row * p.ldda;
      Vec8<E>::store(da + c, g, p.I - c);
      Vec8<E>::store(da + p.I + c, u, p.I - c);
      if (p.hg) Vec8<E>::store(static_cast<E*>(p.hg) + row * p.ldhg + c, hg, p.I - c);
    }
  }
  if (!p.dgate) return;
  sum = wave_sum(sum);
  if (p.wpr > 1) {
    if (lane == 0) red[wave] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int i = 0; i < p.wpr; ++i) sum += red[first + i];
  }
  if (live && tid == first * 64) p.dgate[row] = sum;
}

// A wave takes 512 columns at a time; a row gets the waves that it fills with
// one vector a thread, up to the workgroup's four.  At 2048 columns and 32768 rows
// one, two and four waves a row take 150, 144 and 142 us (at 9 rows 7.6, 6.8 and
// 7.0), at 512 columns 31.3, 33.4 and 45.5.
int waves_of_row(int I) { return I > 1024 ? 4 : (I > 512 ? 2 : 1); }

}  // namespace

extern "C" moe_status_t moe_swiglu(const void* a, moe_dtype_t dt, int R, int I, long long lda,
                                   void* h, long long ldh, hipStream_t stream) {
  if (R < 0 || I < 0 || I > (1 << 24) || lda < 2LL * I || ldh < I) return MOE_ERR_SHAPE;
  if (!valid_dtype(dt)) return MOE_ERR_UNSUPPORTED;
  if (R == 0 || I == 0) return MOE_OK;
  if (!a || !h) return MOE_ERR_NULL;
  if (!element_aligned(a, dt) || !element_aligned(h, dt)) return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const int vecs = (I + 7) / 8;
  const int slab = (1 << 30) / vecs;      // rows whose vectors count below 2^30
  for (long long r0 = 0; r0 < R; r0 += slab) {
    const uint32_t items = (uint32_t)(R - r0 < slab ? R - r0 : slab) * (uint32_t)vecs;
    if (dt == MOE_BF16)
      hipLaunchKernelGGL(swiglu_kernel<bf16_t>, dim3((items + 255) / 256), dim3(256), 0, stream,
                         static_cast<const bf16_t*>(a) + r0 * lda, lda, items, vecs, I,
                         static_cast<bf16_t*>(h) + r0 * ldh, ldh);
    else
      hipLaunchKernelGGL(swiglu_kernel<float>, dim3((items + 255) / 256), dim3(256), 0, stream,
                         static_cast<const float*>(a) + r0 * lda, lda, items, vecs, I,
                         static_cast<float*>(h) + r0 * ldh, ldh);
    if (moe_status_t s = launch_status()) return s;
  }
  return MOE_OK;
}

extern "C" moe_status_t moe_swiglu_backward(const void* a, const void* dh, moe_dtype_t dt, int R,
                                            int I, long long lda, long long lddh,
                                            const float* row_gate, void* da, long long ldda,
                                            float* dgate, void* hg, long long ldhg,
                                            hipStream_t stream) {
  if (R < 0 || I < 0 || I > (1 << 24) || lda < 2LL * I || lddh < I || ldda < 2LL * I ||
      (hg && ldhg < I))
    return MOE_ERR_SHAPE;
  if (!valid_dtype(dt)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (I > 0 && (!a || !dh || !da)) return MOE_ERR_NULL;
  if (!element_aligned(a, dt) || !element_aligned(dh, dt) || !element_aligned(da, dt) ||
      !element_aligned(hg, dt) || !element_aligned(row_gate, MOE_F32) ||
      !element_aligned(dgate, MOE_F32))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const int wpr = waves_of_row(I), rows = 4 / wpr;
  const long long esize = dt == MOE_BF16 ? 2 : 4;
  auto at = [](const void* p, long long bytes) -> const void* { return p ? static_cast<const char*>(p) + bytes : p; };
  const int slab = rows << 22;            // a launch holds less than 2^32 threads
  for (long long r0 = 0; r0 < R; r0 += slab) {
    const int n = (int)(R - r0 < slab ? R - r0 : slab);
    const BwdParams p{at(a, r0 * lda * esize), at(dh, r0 * lddh * esize), row_gate ? row_gate + r0 : nullptr,
                      const_cast<void*>(at(da, r0 * ldda * esize)), const_cast<void*>(at(hg, r0 * ldhg * esize)),
                      dgate ? dgate + r0 : nullptr, lda, lddh, ldda, ldhg, n, I, wpr};
    const dim3 grid((unsigned)((n - 1) / rows + 1));
    if (dt == MOE_BF16)
      hipLaunchKernelGGL(swiglu_bwd_kernel<bf16_t>, grid, dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL(swiglu_bwd_kernel<float>, grid, dim3(256), 0, stream, p);
    if (moe_status_t s = launch_status()) return s;
  }
  return MOE_OK;
}
