// The router's balance loss with its statistics, and the gradient of the router's
// logits from the gates and from that loss (include/moe_fp8.h gives the formulas).
//
// Both read the scores [T, N] once; a wave takes a token, its lanes the experts.
//
// Loss: a workgroup sums the normalised scores and counts the picks of a tile of
// consecutive tokens, apart for each sequence that the tile meets (and forms the
// results itself where there is one tile).  A tile and a
// sequence that meet own the slot tile + sequence of the workspace: walking
// along the tokens each next pair has a larger tile or a larger sequence, so the
// slots are distinct and tiles + sequences of them are enough.  A second
// kernel adds each sequence's slots in order.
//
// Measured at 16384 x 256, 8 picks: loss 8.1 + 7.2 us over 12 ragged sequences (7.7 + 12.3
// over one: one workgroup reads all slots), gradient 8.8 us (26.7 MB, 3.0 TB/s); at 64 x
// 16 5.0 and 3.3 us.  The 17 and 27 MB that they move would take 4 and 6 us at a copy's
// rate.
#include <type_traits>

#include "rows.h"

namespace {

using namespace moe;

constexpr int kMaxExperts = 1024;
constexpr int kLossThreads = 512, kLossWaves = kLossThreads / 64;
// Tiles: one a compute unit, of at least 16 tokens.  Captured, tiles of 8, 16, 32 and 64 tokens
// at least take 9.4, 9.1, 9.6 and 10.5 us at 256 x 256, 10.6, 9.7, 9.5 and 10.9 at 512 x 256,
// and, with fewer slots to add, 16.6, 16.5, 13.0 and 12.4 at 4096 x 256.
constexpr int kTokens = 16, kMostTokens = 1024;
constexpr int kTiles = 256;
constexpr int kAtOnce = 4;              // tokens whose scores a wave has in flight
// What one workgroup does by itself, in one launch.  Captured, it and the two launches take 5.5
// and 8.5 us at 64 x 64, 7.4 and 8.7 at 128 x 64, 10.8 and 8.8 at 256 x 64; 9.7 and 12.5 at 64 x
// 1024, 17.0 and 15.0 at 192 x 1024; two sequences, which it takes one after the other, 6.8 and 7.7
// at 64 x 64 and 12.1 and 12.1 at 64 x 1024, four 9.9 and 7.5.  (Alone the border could be at 128.)
constexpr int kOneTokens = 64, kOneSequences = 2;

constexpr int kMostSequences = 1 << 23;                // a workgroup of 256 threads each fits a launch

// Sequence i's first token and, at i + 1, the one behind its last.
struct Sequences {
  const int32_t* offsets;       // NULL: one sequence of all tokens
  int n, T;
  __device__ __forceinline__ int at(int i) const {
    if (!offsets) return i == 0 ? 0 : T;
    const int v = offsets[i];
    return v < 0 ? 0 : (v > T ? T : v);
  }
  // Sequences that end at or before token t.
  __device__ __forceinline__ int ended(int t) const {
    int lo = 0, hi = n;         // at(i + 1) <= t below lo, > t from hi on
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid + 1) <= t) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  }
};

// A lane's PER consecutive experts of a row; 0 past the last.
template <int PER>
__device__ __forceinline__ void load_row(const float* row, int N, int lane, float (&v)[PER]) {
  typedef float vec_t __attribute__((ext_vector_type(PER), aligned(4)));
  const int first = lane * PER, have = N - first;
  if (have >= PER) {
    const vec_t x = *reinterpret_cast<const vec_t*>(row + first);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = ((const float*)&x)[i];
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < have ? row[first + i] : 0.0f;
  }
}
template <int PER>
__device__ __forceinline__ float row_sum(const float (&v)[PER]) {
  float sum = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) sum += v[i];
  return wave_sum(sum);
}
// v[i] / sum by the reciprocal, both scaled where it would overflow; 1 / N where the
// sum is zero.
template <int PER>
__device__ __forceinline__ void shares(const float (&v)[PER], float sum, int N, float (&out)[PER]) {
  const float up = sum < 0x1p-60f ? 0x1p64f : 1.0f, inv = 1.0f / (sum * up);
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = sum == 0.0f ? 1.0f / N : v[i] * up * inv;
}

struct LossParams {
  moe_balance_args a;
  int tile;             // tokens of a tile
  float* mass;          // [slots][N]
  int32_t* picks;       // [slots][N]
  int32_t* live;        // [slots]
};

// Statistics of a sequence at expert e, and its term of the loss.
__device__ __forceinline__ double finish(const moe_balance_args& a, int s, int e, double mass, int picks, int n) {
  const double load = n ? (double)a.N * picks / ((double)a.k * n) : 0.0, prob = n ? mass / n : 0.0;
  const long long at = (long long)s * a.N + e;
  if (a.load) a.load[at] = (float)load;
  if (a.prob) a.prob[at] = (float)prob;
  if (a.counts) a.counts[at] = picks;
  return load * prob;
}
// Sum over the workgroup in a fixed order, in thread 0.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < (int)blockDim.x / 64; ++w) v += part[w];
  return v;
}

// ONE: the tile holds every token, and the results are formed here.
template <int PER, bool ONE>
__global__ __launch_bounds__(kLossThreads) void balance_partial_kernel(LossParams p) {
  __shared__ float mass[kLossWaves][PER * 64];
  __shared__ int picks[PER * 64];
  __shared__ int live[kLossWaves];
  __shared__ double part[kLossWaves];
  const moe_balance_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Sequences seq{a.seq_offsets, a.n_seq, a.T};
  const int first = ONE ? 0 : (int)blockIdx.x * p.tile, last = ONE ? a.T : min(first + p.tile, a.T);
  for (int s = ONE ? 0 : seq.ended(first); s < a.n_seq; ++s) {
    const int lo = max(seq.at(s), first), hi = min(seq.at(s + 1), last);
    if (!ONE && lo >= last) break;
    if (!ONE && lo >= hi) {             // and every other empty one at this token
      s = max(s, seq.ended(lo) - 1);
      continue;
    }
    for (int i = tid; i < PER * 64; i += kLossThreads) picks[i] = 0;
    __syncthreads();
    for (int i = tid; i < (hi - lo) * a.k; i += kLossThreads) {
      const int e = a.topk_idx[(long long)lo * a.k + i];
      if (e >= 0 && e < a.N && !(a.token_mask && !a.token_mask[lo + i / a.k])) atomicAdd(&picks[e], 1);
    }
    float sum[PER] = {};
    int n = 0;
    for (int t = lo + wave; t < hi; t += kLossWaves * kAtOnce) {
      float v[kAtOnce][PER];
      bool there[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int at = t + u * kLossWaves;
        there[u] = at < hi && !(a.token_mask && !a.token_mask[at]);
        if (there[u]) load_row<PER>(a.scores + at * a.lds, a.N, lane, v[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (!there[u]) continue;
        ++n;
        float share[PER];
        shares<PER>(v[u], row_sum<PER>(v[u]), a.N, share);
#pragma unroll
        for (int i = 0; i < PER; ++i) sum[i] += share[i];
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) mass[wave][lane * PER + i] = sum[i];
    if (lane == 0) live[wave] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kLossWaves; ++w) n += live[w];
    const long long slot = (long long)blockIdx.x + s;
    double term = 0.0;
    for (int e = tid; e < a.N; e += kLossThreads) {
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < kLossWaves; ++w) m += mass[w][e];
      if constexpr (ONE) {
        term += finish(a, s, e, m, picks[e], n);
      } else {
        p.mass[slot * a.N + e] = m;
        p.picks[slot * a.N + e] = picks[e];
      }
    }
    if constexpr (ONE) {
      term = block_sum(term, part);
      if (tid == 0) {
        if (a.tokens) a.tokens[s] = n;
        if (a.loss) a.loss[s] = (float)(a.alpha * term);
      }
    } else if (tid == 0) {
      p.live[slot] = n;
    }
    __syncthreads();
  }
}

// One workgroup per sequence; its threads are blockDim / W parts of the slots times W
// experts.
template <int W>
__global__ __launch_bounds__(1024) void balance_finish_kernel(LossParams p) {
  __shared__ double mass[1024];
  __shared__ int picks[1024], live[1024];
  __shared__ double part[16];
  const moe_balance_args& a = p.a;
  const Sequences seq{a.seq_offsets, a.n_seq, a.T};
  const int tid = threadIdx.x, parts = blockDim.x / W, mine = tid / W, col = tid % W;
  const int s = blockIdx.x, lo = seq.at(s), hi = seq.at(s + 1);
  const int tile0 = lo / p.tile, tile1 = hi > lo ? (hi - 1) / p.tile + 1 : tile0;
  int n = 0;
  for (int t = tile0 + tid; t < tile1; t += blockDim.x) n += p.live[t + s];
  live[tid] = n;
  __syncthreads();
  for (int half = blockDim.x / 2; half > 0; half >>= 1) {
    if (tid < half) live[tid] += live[tid + half];
    __syncthreads();
  }
  n = live[0];
  double term = 0.0;
  for (int e0 = 0; e0 < a.N; e0 += W) {
    const int e = e0 + col;
    double m = 0.0;
    int c = 0;
    if (e < a.N) {
#pragma unroll 4
      for (int t = tile0 + mine; t < tile1; t += parts) {
        const long long at = (long long)(t + s) * a.N + e;
        m += p.mass[at];
        c += p.picks[at];
      }
    }
    mass[tid] = m;
    picks[tid] = c;
    __syncthreads();
    if (mine == 0 && e < a.N) {
      for (int q = 1; q < parts; ++q) m += mass[q * W + col], c += picks[q * W + col];
      term += finish(a, s, e, m, c, n);
    }
    __syncthreads();
  }
  term = block_sum(term, part);
  if (tid == 0) {
    if (a.tokens) a.tokens[s] = n;
    if (a.loss) a.loss[s] = (float)(a.alpha * term);
  }
}

constexpr int kBwdThreads = 256, kBwdWaves = kBwdThreads / 64;

template <int PER, typename E>
__device__ __forceinline__ void store_row(E* row, int N, int lane, const float (&v)[PER]) {
  typedef E vec_t __attribute__((ext_vector_type(PER), aligned(sizeof(E))));
  const int first = lane * PER, have = N - first;
  if (have >= PER) {
    vec_t x;
#pragma unroll
    for (int i = 0; i < PER; ++i) ((E*)&x)[i] = (E)v[i];
    *reinterpret_cast<vec_t*>(row + first) = x;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < have) row[first + i] = (E)v[i];
  }
}

// What lanes of a wave wrote to LDS is there for the others, without a wait between waves.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One wave per token (2 or 4 tokens a wave, their loads in flight together: 8.8 and
// 10.0 us against 8.6 at 16384 x 256, and a small batch takes longer).
template <int PER, typename E>
__global__ __launch_bounds__(kBwdThreads) void router_backward_kernel(moe_router_bwd_args a) {
  // the picks' parts by expert, and which pick wrote them
  __shared__ __align__(16) float part_of[kBwdWaves][PER * 64];
  __shared__ int pick_of[kBwdWaves][PER * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int t = (int)blockIdx.x * kBwdWaves + wave;
  if (t >= a.T) return;
  const Sequences seq{a.seq_offsets, a.n_seq, a.T};
  const bool few = a.n_seq <= 64;       // a lane a sequence
  int end = 0;
  if (a.load && few && lane < a.n_seq) end = seq.at(lane + 1);
  float s[PER], dz[PER] = {};
  load_row<PER>(a.scores + t * a.lds, a.N, lane, s);
  if (a.dgate) {
    float* const part = part_of[wave];
    int* const pick = pick_of[wave];
    float g = 0.0f, d = 0.0f;
    int e = -1;
    if (lane < a.k) {
      const long long at = (long long)t * a.k + lane;
      g = a.topk_gate[at];
      d = a.dgate[at];
      e = a.topk_idx[at];
      if (e >= a.N) e = -1;
    }
    const bool picks = e >= 0;
    // the picks' scores, and then their parts, meet their experts through LDS (comparing
    // every pick with a lane's experts instead makes the kernel bound by its arithmetic,
    // 12.2 us)
#pragma unroll
    for (int i = 0; i < PER; ++i) part[lane * PER + i] = s[i];
    if (picks) pick[e] = lane;
    wave_sync();
    const float picked = picks ? part[e] : 0.0f;
    const bool twice = picks && pick[e] != lane;
    wave_sync();
#pragma unroll
    for (int i = 0; i < PER; ++i) part[lane * PER + i] = 0.0f;
    const float mean = wave_sum(d * g), any = wave_sum(picked);
    const float mine = any == 0.0f ? 0.0f : g * (1.0f - picked) * (d - mean);
    wave_sync();
    if (__builtin_amdgcn_ballot_w64(twice) == 0) {
      if (picks) part[e] = mine;
    } else {                            // an expert picked twice: one pick after the other
      for (int j = 0; j < a.k; ++j) {
        if (lane == j && picks) part[e] += mine;
        wave_sync();
      }
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < PER; ++i) dz[i] = part[lane * PER + i];
  }
  if (a.load && !(a.token_mask && !a.token_mask[t])) {
    const int q = few ? __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < a.n_seq && end <= t)) : seq.ended(t);
    if (q < a.n_seq && seq.at(q) <= t) {
      const int n = a.tokens[q];
      const float all = row_sum<PER>(s);
      if (all != 0.0f && n > 0) {
        const float c = a.alpha * (a.dloss ? a.dloss[q] : 1.0f) / n;
        float load[PER], share[PER], dot = 0.0f;
        load_row<PER>(a.load + (long long)q * a.N, a.N, lane, load);
        shares<PER>(s, all, a.N, share);
#pragma unroll
        for (int i = 0; i < PER; ++i) dot += load[i] * share[i];
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < PER; ++i) dz[i] += c * share[i] * (1.0f - s[i]) * (load[i] - dot);
      }
    }
  }
  store_row<PER, E>(static_cast<E*>(a.dz) + t * a.ldz, a.N, lane, dz);
}

bool sizes_ok(int T, int N, int k, int n_seq, long long lds) {
  return T >= 0 && N >= 1 && N <= kMaxExperts && k >= 1 && k <= 32 && n_seq >= 0 && lds >= N;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Tokens of a tile: kTiles tiles, between kTokens and kMostTokens (so that few shares are
// added in float).
int tile_of(int T) {
  const int even = (T + kTiles - 1) / kTiles;
  return even < kTokens ? kTokens : even > kMostTokens ? kMostTokens : even;
}
bool one_tile(int T, int n_seq) { return T <= kOneTokens && n_seq <= kOneSequences; }
long long slots_of(int T, int n_seq) { return (long long)(T + tile_of(T) - 1) / tile_of(T) + n_seq; }

// f with the experts of a lane as a constant.
template <typename F>
void with_experts(int N, F f) {
  if (N <= 64) f(std::integral_constant<int, 1>{});
  else if (N <= 128) f(std::integral_constant<int, 2>{});
  else if (N <= 256) f(std::integral_constant<int, 4>{});
  else if (N <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace

extern "C" size_t moe_balance_loss_workspace_bytes(int T, int N, int n_seq) {
  if (T < 1 || N < 1 || n_seq < 1 || one_tile(T, n_seq)) return 0;
  return (size_t)slots_of(T, n_seq) * (2 * (size_t)N + 1) * 4;
}

extern "C" moe_status_t moe_balance_loss(const moe_balance_args* args, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_balance_args& a = *args;
  if (!sizes_ok(a.T, a.N, a.k, a.n_seq, a.lds) || (!a.seq_offsets && a.n_seq > 1)) return MOE_ERR_SHAPE;
  if (a.T > (1 << 24) || a.n_seq > kMostSequences) return MOE_ERR_UNSUPPORTED;
  if (a.n_seq == 0) return MOE_OK;
  if (a.T > 0 && (!a.scores || !a.topk_idx)) return MOE_ERR_NULL;
  const void* words[] = {a.scores, a.topk_idx, a.seq_offsets, a.loss, a.load, a.prob, a.counts, a.tokens};
  for (const void* w : words)
    if (!aligned4(w)) return MOE_ERR_ALIGN;
  const size_t need = moe_balance_loss_workspace_bytes(a.T, a.N, a.n_seq);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const long long slots = slots_of(a.T, a.n_seq);
  LossParams p{a, tile_of(a.T), static_cast<float*>(ws), nullptr, nullptr};
  if (one_tile(a.T, a.n_seq)) {
    with_experts(a.N, [&](auto per) {
      hipLaunchKernelGGL((balance_partial_kernel<decltype(per)::value, true>), dim3(1), dim3(kLossThreads), 0, stream, p);
    });
    return launch_status();
  }
  p.picks = reinterpret_cast<int32_t*>(p.mass + slots * a.N);
  p.live = p.picks + slots * a.N;
  if (a.T > 0) {
    const unsigned tiles = (unsigned)((a.T + p.tile - 1) / p.tile);
    with_experts(a.N, [&](auto per) {
      hipLaunchKernelGGL((balance_partial_kernel<decltype(per)::value, false>), dim3(tiles), dim3(kLossThreads), 0,
                         stream, p);
    });
    if (moe_status_t s = launch_status()) return s;
  }
  // a few slots a sequence leave most of a large workgroup idle
  const int threads = slots > 4LL * a.n_seq ? 1024 : 256;
  if (a.N <= 64)
    hipLaunchKernelGGL(balance_finish_kernel<64>, dim3((unsigned)a.n_seq), dim3(threads), 0, stream, p);
  else
    hipLaunchKernelGGL(balance_finish_kernel<256>, dim3((unsigned)a.n_seq), dim3(threads), 0, stream, p);
  return launch_status();
}

extern "C" moe_status_t moe_router_backward(const moe_router_bwd_args* args, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_router_bwd_args& a = *args;
  if (!sizes_ok(a.T, a.N, a.k, a.n_seq, a.lds) || a.ldz < a.N || (!a.seq_offsets && a.n_seq > 1)) return MOE_ERR_SHAPE;
  if (a.T > (1 << 24) || a.n_seq > kMostSequences || !valid_dtype(a.out_dtype)) return MOE_ERR_UNSUPPORTED;
  if (a.T == 0) return MOE_OK;
  if (!a.scores || !a.dz || (a.dgate && (!a.topk_gate || !a.topk_idx)) || (a.load && !a.tokens)) return MOE_ERR_NULL;
  const void* words[] = {a.scores, a.topk_idx, a.topk_gate, a.dgate, a.load, a.tokens, a.seq_offsets, a.dloss};
  for (const void* w : words)
    if (!aligned4(w)) return MOE_ERR_ALIGN;
  if (!element_aligned(a.dz, a.out_dtype)) return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const dim3 grid((unsigned)((a.T + kBwdWaves - 1) / kBwdWaves)), block(kBwdThreads);
  with_experts(a.N, [&](auto per) {
    constexpr int P = decltype(per)::value;
    if (a.out_dtype == MOE_F32)
      hipLaunchKernelGGL((router_backward_kernel<P, float>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((router_backward_kernel<P, __bf16>), grid, block, 0, stream, a);
  });
  return launch_status();
}
