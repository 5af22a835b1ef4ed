// The global norm of many gradient tensors, and clipping by it.
//
//   sumsq = sum over all tensors and elements of x^2   (in double)
//   norm  = sqrt(sumsq),  coef = min(1, max_norm / (norm + 1e-6)), 1 where the
//   norm is not finite;  dst = coef * src  (rounded once to dst's type)
//
// The tensors are cut into chunks of 4096 elements, numbered through in list
// order; a workgroup takes a contiguous range of chunk numbers, so the split
// is even whatever the tensors' sizes, and walks its range one stretch (the
// chunks of one tensor) after the other.  Squares are summed in double: no
// gradient overflows or vanishes in the sum, and the partial sums are added
// in a fixed order, so the norm is the same on every run.
//
// Memory bounds it: 1.46 G floats are read for the norm in 1.01 ms (5.75 TB/s),
// then read and written in 2.31 ms (5.05; a large copy reaches 4.78).  Small lists are
// latency: 1.7 M elements in two launches of 3.9 and 6.2 us; the second
// adds the partial sums for itself, which saves a launch between them.
// Chunks of 4096 elements are two vectors a thread, small enough that such a
// list still spreads over every compute unit (2048 and 8192 measure the same).
#include <algorithm>
#include <cmath>
#include <vector>

#include "rows.h"

namespace {

using namespace moe;

constexpr int kChunk = 4096;
constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;         // 3282 us for 1.46 G elements; 1024: 3279, 4096: 3262
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

// The last tensor whose first chunk is <= c (empty tensors own no chunk),
// searched 64 at a time by the lanes of each wave.
__device__ __forceinline__ int find_tensor(const ListParams& p, long long c) {
  int lo = 0, n = p.n;                  // it is one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = (threadIdx.x & 63) * step;
    const bool before = at < n && p.table[lo + at].first_chunk <= c;
    const int last = (int)__builtin_popcountll(__ballot(before)) - 1;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// calls f(entry, first element, elements) for the stretches of this
// workgroup's range (which ends with the table's last tensor, if the caller's
// count of chunks says more)
template <typename F>
__device__ __forceinline__ void for_stretches(const ListParams& p, F f) {
  const long long lo = p.chunks * blockIdx.x / gridDim.x, hi = p.chunks * (blockIdx.x + 1) / gridDim.x;
  if (lo >= hi) return;
  long long c = lo;
  for (int t = find_tensor(p, lo); c < hi && t < p.n; ++t) {
    const Entry e = p.table[t];
    const long long own = (e.numel + kChunk - 1) / kChunk;
    const long long end = min(hi, e.first_chunk + own);
    if (end <= c) continue;
    const long long at = (c - e.first_chunk) * kChunk;
    f(e, at, min(e.numel, (end - e.first_chunk) * kChunk) - at);
    c = end;
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

// Walks the n elements at p, eight a thread and kUnroll vectors at a time so
// that their loads are in flight together; g(element index, value vector).
constexpr int kUnroll = 4;
template <typename E, typename G>
__device__ __forceinline__ void walk(const E* p, long long n, G g) {
  constexpr int kSpan = kThreads * 8;
  long long c = threadIdx.x * 8;
  const long long whole = n - (long long)(kUnroll - 1) * kSpan - 8;
  for (; c <= whole; c += kUnroll * kSpan) {
    Vec8<E> x[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) x[k].load(p + c + k * kSpan, 8);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) g(c + k * kSpan, x[k], 8);
  }
  for (; c < n; c += kSpan) {
    const int valid = (int)min(n - c, 8LL);
    Vec8<E> x;
    x.load(p + c, valid);
    g(c, x, valid);
  }
}

template <typename E>
__device__ __forceinline__ double squares(const E* p, long long n) {
  double t = 0.0;
  walk(p, n, [&](long long, const Vec8<E>& x, int) {
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) t = __builtin_fma((double)v[j], (double)v[j], t);
  });
  return t;
}

__global__ __launch_bounds__(kThreads) void square_sum_kernel(ListParams p, double* part) {
  double t = 0.0;
  for_stretches(p, [&](const Entry& e, long long at, long long n) {
    t += e.src_f32 ? squares(static_cast<const float*>(e.src) + at, n)
                   : squares(static_cast<const bf16_t*>(e.src) + at, n);
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
__device__ __forceinline__ void scale(const S* s, D* d, long long n, float coef) {
  walk(s, n, [&](long long c, const Vec8<S>& x, int valid) {
    float v[8];
    x.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= coef;
    Vec8<D>::store(d + c, v, valid);
  });
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
  for_stretches(p, [&](const Entry& e, long long at, long long n) {
    if (coef == 1.0f && e.src == e.dst) return;      // nothing to change in place
    if (e.src_f32) {
      const float* s = static_cast<const float*>(e.src) + at;
      if (e.dst_f32) scale(s, static_cast<float*>(e.dst) + at, n, coef);
      else scale(s, static_cast<bf16_t*>(e.dst) + at, n, coef);
    } else {
      const bf16_t* s = static_cast<const bf16_t*>(e.src) + at;
      if (e.dst_f32) scale(s, static_cast<float*>(e.dst) + at, n, coef);
      else scale(s, static_cast<bf16_t*>(e.dst) + at, n, coef);
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
