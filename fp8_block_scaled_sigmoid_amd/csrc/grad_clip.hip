// The global norm of many gradient tensors, and clipping by it.
//
//   sumsq = sum over all tensors and elements of x^2   (in double)
//   norm  = sqrt(sumsq),  coef = min(1, max_norm / (norm + 1e-6)), 1 where the
//   norm is not finite;  dst = coef * src  (rounded once to dst's type)
//
// The tensors are cut into chunks of 16384 elements, numbered through in list
// order; a workgroup takes a contiguous range of chunk numbers, so the split
// is even whatever the tensors' sizes.  Squares are summed in double: no
// gradient overflows or vanishes in the sum, and the partial sums are added
// in a fixed order, so the norm is the same on every run.
#include <algorithm>
#include <cmath>
#include <vector>

#include "rows.h"

namespace {

using namespace moe;

constexpr int kChunk = 16384;
constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;
constexpr float kEps = 1e-6f;

struct Entry {                 // one tensor of the list, as the table holds it
  const void* src;
  void* dst;
  long long numel;
  long long first_chunk;       // chunks of the tensors before it
  int src_f32, dst_f32;
};
static_assert(sizeof(Entry) == 40, "table layout");

struct ListParams {
  const Entry* table;
  int n;
  long long chunks;
};

// the last tensor whose first chunk is <= c (empty tensors own no chunk)
__device__ __forceinline__ int find_tensor(const ListParams& p, long long c) {
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.table[mid].first_chunk <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// calls f(entry, first element, elements) for this workgroup's chunks
template <typename F>
__device__ __forceinline__ void for_chunks(const ListParams& p, F f) {
  const long long lo = p.chunks * blockIdx.x / gridDim.x, hi = p.chunks * (blockIdx.x + 1) / gridDim.x;
  if (lo >= hi) return;
  int t = find_tensor(p, lo);
  for (long long c = lo; c < hi; ++c) {
    while (t + 1 < p.n && p.table[t + 1].first_chunk <= c) ++t;
    const Entry e = p.table[t];
    const long long at = (c - e.first_chunk) * kChunk;
    const long long left = e.numel - at;
    f(e, at, (int)(left < kChunk ? left : kChunk));
  }
}

// Sum of v over the workgroup, the same in every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <typename E>
__device__ __forceinline__ double chunk_squares(const E* p, int n) {
  double t = 0.0;
  for (int c = threadIdx.x * 8; c < n; c += kThreads * 8) {
    Vec8<E> x;
    x.load(p + c, n - c);
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) t = __builtin_fma((double)v[j], (double)v[j], t);
  }
  return t;
}

__global__ __launch_bounds__(kThreads) void square_sum_kernel(ListParams p, double* part) {
  double t = 0.0;
  for_chunks(p, [&](const Entry& e, long long at, int n) {
    t += e.src_f32 ? chunk_squares(static_cast<const float*>(e.src) + at, n)
                   : chunk_squares(static_cast<const bf16_t*>(e.src) + at, n);
  });
  t = block_sum(t);
  if (threadIdx.x == 0) part[blockIdx.x] = t;
}

__device__ __forceinline__ double total(const double* part, int parts) {
  double t = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) t += part[i];
  return block_sum(t);
}

__global__ __launch_bounds__(kThreads) void finish_kernel(const double* part, int parts,
                                                           double* sumsq, float* norm) {
  const double t = total(part, parts);
  if (threadIdx.x == 0) {
    if (sumsq) *sumsq = t;
    if (norm) *norm = (float)sqrt(t);
  }
}

template <typename S, typename D>
__device__ __forceinline__ void scale_chunk(const S* s, D* d, int n, float coef) {
  for (int c = threadIdx.x * 8; c < n; c += kThreads * 8) {
    Vec8<S> x;
    x.load(s + c, n - c);
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= coef;
    Vec8<D>::store(d + c, v, n - c);
  }
}

// Scales every tensor.  `part` holds `parts` partial sums of squares (one:
// the sum itself); each workgroup adds them up for itself, in the same order.
__global__ __launch_bounds__(kThreads) void scale_kernel(ListParams p, const double* part, int parts,
                                                          float max_norm, float* result) {
  const float norm = (float)sqrt(total(part, parts));
  const float c = max_norm / (norm + kEps);
  const bool finite = __builtin_isfinite(norm);
  const float coef = finite && c < 1.0f ? c : 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0 && result) {
    result[0] = norm;
    result[1] = coef;
  }
  for_chunks(p, [&](const Entry& e, long long at, int n) {
    if (coef == 1.0f && e.src == e.dst) return;      // nothing to change in place
    if (e.src_f32) {
      const float* s = static_cast<const float*>(e.src) + at;
      if (e.dst_f32) scale_chunk(s, static_cast<float*>(e.dst) + at, n, coef);
      else scale_chunk(s, static_cast<bf16_t*>(e.dst) + at, n, coef);
    } else {
      const bf16_t* s = static_cast<const bf16_t*>(e.src) + at;
      if (e.dst_f32) scale_chunk(s, static_cast<float*>(e.dst) + at, n, coef);
      else scale_chunk(s, static_cast<bf16_t*>(e.dst) + at, n, coef);
    }
  });
}

unsigned grid_of(long long chunks) {
  return (unsigned)(chunks < kMaxBlocks ? (chunks > 0 ? chunks : 1) : kMaxBlocks);
}

moe_status_t check_list(const void* table, int n, long long chunks) {
  if (n < 0 || chunks < 0) return MOE_ERR_SHAPE;
  if (chunks > 0 && (n == 0 || !table)) return MOE_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(table) & 7) return MOE_ERR_ALIGN;
  return MOE_OK;
}

}  // namespace

extern "C" size_t moe_grad_table_bytes(int n) { return n > 0 ? (size_t)n * sizeof(Entry) : 0; }

extern "C" moe_status_t moe_grad_table(const moe_grad_tensor* tensors, int n, void* table,
                                       size_t table_bytes, long long* total_chunks) {
  if (n < 0) return MOE_ERR_SHAPE;
  if (!total_chunks || (n > 0 && (!tensors || !table))) return MOE_ERR_NULL;
  if (table_bytes < moe_grad_table_bytes(n)) return MOE_ERR_WORKSPACE;
  auto bytes = [](moe_dtype_t d) { return d == MOE_F32 ? 4LL : 2LL; };
  long long chunks = 0;
  struct Span {
    uintptr_t lo, hi;
    int tensor;
    bool written;
  };
  std::vector<Span> spans;
  try {
    spans.reserve(2 * (size_t)n);
    for (int i = 0; i < n; ++i) {
      const moe_grad_tensor& t = tensors[i];
      if (t.numel < 0 || t.numel > (1LL << 48)) return MOE_ERR_SHAPE;
      if (!valid_dtype(t.src_dtype) || !valid_dtype(t.dst_dtype)) return MOE_ERR_UNSUPPORTED;
      if (t.numel > 0) {
        if (!t.src || !t.dst) return MOE_ERR_NULL;
        if (!element_aligned(t.src, t.src_dtype) || !element_aligned(t.dst, t.dst_dtype))
          return MOE_ERR_ALIGN;
        if (t.src == t.dst && t.src_dtype != t.dst_dtype) return MOE_ERR_UNSUPPORTED;
        const uintptr_t s = reinterpret_cast<uintptr_t>(t.src), d = reinterpret_cast<uintptr_t>(t.dst);
        if (t.src != t.dst) spans.push_back({s, s + (uintptr_t)(t.numel * bytes(t.src_dtype)), i, false});
        spans.push_back({d, d + (uintptr_t)(t.numel * bytes(t.dst_dtype)), i, true});
      }
      Entry e{t.src, t.dst, t.numel, chunks, t.src_dtype == MOE_F32, t.dst_dtype == MOE_F32};
      static_cast<Entry*>(table)[i] = e;
      chunks += (t.numel + kChunk - 1) / kChunk;
    }
    // memory that is written belongs to one tensor alone
    std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
  } catch (...) {
    return MOE_ERR_WORKSPACE;
  }
  uintptr_t end_any = 0, end_written = 0;
  for (const Span& s : spans) {
    if (s.lo < end_written || (s.written && s.lo < end_any)) return MOE_ERR_UNSUPPORTED;
    end_any = std::max(end_any, s.hi);
    if (s.written) end_written = std::max(end_written, s.hi);
  }
  *total_chunks = chunks;
  return MOE_OK;
}

extern "C" size_t moe_grad_norm_workspace_bytes(long long total_chunks) {
  return (size_t)grid_of(total_chunks) * sizeof(double);
}

extern "C" moe_status_t moe_grad_norm(const void* table, int n, long long total_chunks, void* ws,
                                      size_t ws_bytes, double* sumsq, float* norm,
                                      hipStream_t stream) {
  if (moe_status_t s = check_list(table, n, total_chunks)) return s;
  if (!sumsq && !norm) return MOE_ERR_NULL;
  if (!ws || ws_bytes < moe_grad_norm_workspace_bytes(total_chunks)) return MOE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 7) || (reinterpret_cast<uintptr_t>(sumsq) & 7) ||
      (reinterpret_cast<uintptr_t>(norm) & 3))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const ListParams p{static_cast<const Entry*>(table), n, total_chunks};
  const unsigned grid = grid_of(total_chunks);
  hipLaunchKernelGGL(square_sum_kernel, dim3(grid), dim3(kThreads), 0, stream, p,
                     static_cast<double*>(ws));
  if (moe_status_t s = launch_status()) return s;
  hipLaunchKernelGGL(finish_kernel, dim3(1), dim3(kThreads), 0, stream,
                     static_cast<const double*>(ws), (int)grid, sumsq, norm);
  return launch_status();
}

extern "C" moe_status_t moe_grad_scale(const void* table, int n, long long total_chunks,
                                       const double* sumsq, float max_norm, float* result,
                                       hipStream_t stream) {
  if (moe_status_t s = check_list(table, n, total_chunks)) return s;
  if (!(max_norm >= 0.0f)) return MOE_ERR_SHAPE;
  if (!sumsq) return MOE_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(sumsq) & 7) || (reinterpret_cast<uintptr_t>(result) & 3))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const ListParams p{static_cast<const Entry*>(table), n, total_chunks};
  hipLaunchKernelGGL(scale_kernel, dim3(grid_of(total_chunks)), dim3(kThreads), 0, stream, p, sumsq,
                     1, max_norm, result);
  return launch_status();
}

extern "C" moe_status_t moe_grad_clip(const void* table, int n, long long total_chunks, void* ws,
                                      size_t ws_bytes, float max_norm, float* result,
                                      hipStream_t stream) {
  if (moe_status_t s = check_list(table, n, total_chunks)) return s;
  if (!(max_norm >= 0.0f)) return MOE_ERR_SHAPE;
  if (!ws || ws_bytes < moe_grad_norm_workspace_bytes(total_chunks)) return MOE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 7) || (reinterpret_cast<uintptr_t>(result) & 3))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const ListParams p{static_cast<const Entry*>(table), n, total_chunks};
  const unsigned grid = grid_of(total_chunks);
  hipLaunchKernelGGL(square_sum_kernel, dim3(grid), dim3(kThreads), 0, stream, p,
                     static_cast<double*>(ws));
  if (moe_status_t s = launch_status()) return s;
  hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(kThreads), 0, stream, p,
                     static_cast<const double*>(ws), (int)grid, max_norm, result);
  return launch_status();
}
