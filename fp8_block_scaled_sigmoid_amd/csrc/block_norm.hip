// The norms around a block, fused with the block's gate and the residual
// scale, and their backward pass.
//
// Forward, per token t (all sums and statistics in float):
//   n = b / sqrt(mean(b^2) + eps) * w_post      (n = b without w_post)
//   r = alpha x + beta gate n                   (r = x without a block output)
//   h = r / sqrt(mean(r^2) + eps) * w_pre
// Backward, with r^ = r / rms(r), b^ = b / rms(b) and d the gradient that
// reaches r from both of its uses:
//   v  = dh w_pre,   d  = dr + (v - r^ mean(v r^)) / rms(r),   dx = alpha d
//   dn = beta gate d, u = dn w_post, db = (u - b^ mean(u b^)) / rms(b)
//   dw_pre = sum_t dh r^,  dw_post = sum_t dn b^,  dgate = beta d n (summed
//   over what the gate is shared by)
// Both statistics come from the rows themselves, so nothing but r and b has to
// be kept between the passes.
//
// Memory bounds both passes (forward x, b, r, h; backward r, dr, b, dh, dx, db).
// At 8192 x 7168 in bf16: forward 470 MB in 93 us, 5.05 TB/s; backward 705 MB in
// 152 us + 5 us for the sums over tokens, 4.5 TB/s (a large copy: 4.78).  At one
// token the forward kernel takes 4.4 us: launch, the row's latency, two sums.
#include <type_traits>

#include "rows.h"

namespace {

using namespace moe;

constexpr int kMaxWaves = 16;
constexpr int kMaxWidth = 16384;
constexpr int kFwdWaves = 8, kBwdWaves = 16;      // waves of a workgroup
constexpr int kMaxBlocks = 1 << 20, kMaxRows = 1 << 30;

// How rows are laid over threads: `wpr` waves share a row, a workgroup holds
// `groups` rows at a time, and a thread owns vectors t, t + 64 wpr, ... of its
// row, `items` of them.  Forward workgroups have 8 waves, the backward ones 16: a
// forward row has one reduction after another and more, smaller workgroups on a
// compute unit hide it (93 us at 8192 x 7168, against 97 with 16 waves
// and 100 with 4); a
// backward workgroup keeps two float sums for each channel, and the more
// waves share a row the more registers are left for the next row's loads.
// Widths up to 512 run one wave per row, without barriers.
struct RowShape {
  int wpr, groups, items;
};

RowShape row_shape(int H, int waves) {
  RowShape s;
  const int vecs = (H + 7) / 8;
  s.items = 1;
  while (vecs > waves * 64 * s.items) s.items *= 2;
  s.wpr = (vecs + 64 * s.items - 1) / (64 * s.items);
  s.groups = waves / s.wpr;
  return s;
}

// Sums N values over the waves of a row; every thread of the row gets them.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[kMaxWaves], int wave, int lane,
                                         int first_wave, int wpr) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (wpr == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][wave] = v[i];
  }
  __syncthreads();
  const int w = lane & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = row16_sum(w < wpr ? red[i][first_wave + w] : 0.0f);
}

struct FwdParams {
  moe_block_norm_args a;
  int wpr, groups;
};

template <typename X, typename B, int ITEMS>
__global__ __launch_bounds__(kFwdWaves * 64) void block_norm_kernel(FwdParams p) {
  // one buffer per reduction and row parity: a row's sums are read behind its
  // own barrier, and the buffer is written again two barriers later
  __shared__ float red_b[2][1][kMaxWaves], red_r[2][1][kMaxWaves];
  int par = 0;
  const moe_block_norm_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave / p.wpr, first_wave = grp * p.wpr;
  const int gt = tid - first_wave * 64, stride = p.wpr * 64;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool has_b = a.b != nullptr;

  for (int row0 = blockIdx.x * p.groups; row0 < a.T; row0 += gridDim.x * p.groups, par ^= 1) {
    const int row = row0 + grp;
    const bool live = row < a.T;
    Vec8<X> xv[ITEMS];
    Vec8<B> bv[ITEMS];
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      xv[i].zero();
      bv[i].zero();
      if (live && c < H) {
        xv[i].load(static_cast<const X*>(a.x) + (long long)row * a.ldx + c, H - c);
        if (has_b) bv[i].load(static_cast<const B*>(a.b) + (long long)row * a.ldb + c, H - c);
      }
    }
    float inv_b = 1.0f;
    if (has_b && a.w_post) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float b[8];
        bv[i].get(b);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(b[j], b[j], sum[0]);
      }
      row_sums(sum, red_b[par], wave, lane, first_wave, p.wpr);
      inv_b = 1.0f / __builtin_sqrtf(sum[0] * inv_h + a.eps);
    }
    float r[ITEMS][8];
    sum[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      xv[i].get(r[i]);
      if (has_b && live && c < H) {
        float b[8], s[8];
        bv[i].get(b);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = a.beta * inv_b;
        if (a.w_post) {
          Vec8<float> w;
          float f[8];
          w.load(a.w_post + c, H - c);
          w.get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] *= f[j];
        }
        if (a.gate_mode == MOE_GATE_TOKEN) {
          const float g = static_cast<const float*>(a.gate)[row];
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] *= g;
        } else if (a.gate_mode == MOE_GATE_CHANNEL) {
          Vec8<float> w;
          float f[8];
          w.load(static_cast<const float*>(a.gate) + c, H - c);
          w.get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] *= f[j];
        } else if (a.gate_mode == MOE_GATE_FULL) {
          Vec8<B> w;
          float f[8];
          w.load(static_cast<const B*>(a.gate) + (long long)row * a.ldg + c, H - c);
          w.get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] *= f[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = __builtin_fmaf(b[j], s[j], a.alpha * r[i][j]);
        Vec8<X>::store(static_cast<X*>(a.r) + (long long)row * a.ldr + c, r[i], H - c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(r[i][j], r[i][j], sum[0]);
    }
    if (!a.h) continue;
    // h comes from r before its rounding: one rounding between x, b and h
    row_sums(sum, red_r[par], wave, lane, first_wave, p.wpr);
    const float inv_r = 1.0f / __builtin_sqrtf(sum[0] * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      if (live && c < H) {
        Vec8<float> w;
        float f[8];
        w.load(a.w_pre + c, H - c);
        w.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= r[i][j] * inv_r;
        Vec8<B>::store(static_cast<B*>(a.h) + (long long)row * a.ldh + c, f, H - c);
      }
    }
  }
}

// ---- backward

// Rows are handed out block by block (a persistent grid), so that each
// thread keeps the running sums of its channels in registers over all its
// rows; a second kernel adds the workgroups' partial sums in workgroup order.
// Two sums serve all three gradients: dw_pre, and S = sum_t d b^ times a
// per-row gate, from which dw_post = beta gate_c S and, for a gate per channel,
// dgate = beta w_post S.  A row's four inputs are read once, the next row's
// while one is worked on (202 -> 159 us at 8192 x 7168, with the sums by DPP);
// a gate for each element has no registers left for that (1021 x 2049 in
// float: 18 us; 257 vectors make five waves a row, the fifth with one lane, so a
// workgroup holds three rows, 85 of the 256 go round a second time, and nothing is in
// flight for that round).  Rows wider than 8192 do not fit the registers, and read
// theirs again after the first reduction instead (from L2; 4096 x 16384 in bf16: forward
// 119 us, 4.5 TB/s, backward 238 us, 3.4).  One workgroup per compute unit: 256 partial sums of each channel,
// 15 MB at 7168, which the second kernel adds in 5 us.
struct BwdParams {
  moe_block_norm_bwd_args a;
  int wpr, groups;
  float* part;      // [3][blocks][H]: dw_pre, dw_post, dgate
};

template <typename X, typename B, int ITEMS, bool FULL>
__global__ __launch_bounds__(kBwdWaves * 64) void block_norm_bwd_kernel(BwdParams p) {
  __shared__ float red_a[2][3][kMaxWaves], red_c[2][1][kMaxWaves];   // by row parity, as above
  int par = 0;
  const moe_block_norm_bwd_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave / p.wpr, first_wave = grp * p.wpr;
  const int gt = tid - first_wave * 64, stride = p.wpr * 64;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool has_b = a.b != nullptr, post = has_b && a.w_post;
  const bool channel = a.gate_mode == MOE_GATE_CHANNEL, token = a.gate_mode == MOE_GATE_TOKEN;
  constexpr bool kHold = ITEMS == 1, kAhead = kHold && !FULL;      // as registers allow

  // w_pre, and w_n = beta w_post (gate per channel): u = w_n (gate of the row) d
  float w_pre[ITEMS][8] = {}, w_n[ITEMS][8] = {}, acc_pre[ITEMS][8] = {}, acc_b[ITEMS][8] = {};
  auto load_w = [&](const void* w, int c, float (&f)[8]) {
    Vec8<float> v;
    v.load(static_cast<const float*>(w) + c, H - c);
    v.get(f);
  };
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = (gt + i * stride) * 8;
    if (c < H) {
      float f[8];
      if (a.dh) load_w(a.w_pre, c, w_pre[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) w_n[i][j] = a.beta;
      if (post) {
        load_w(a.w_post, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) w_n[i][j] *= f[j];
      }
      if (channel) {
        load_w(a.gate, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) w_n[i][j] *= f[j];
      }
    }
  }

  struct Row {
    Vec8<X> r, dr;
    Vec8<B> b, dh, g;
  };
  auto load_b = [&](int row, int c, Row& v) {
    v.b.zero();
    if (has_b && row < a.T && c < H)
      v.b.load(static_cast<const B*>(a.b) + (long long)row * a.ldb + c, H - c);
  };
  auto load = [&](int row, int i, Row& v) {
    const int c = (gt + i * stride) * 8;
    v.r.zero(), v.dr.zero(), v.dh.zero(), v.g.zero();
    if (row < a.T && c < H) {
      if (a.dh) {
        v.r.load(static_cast<const X*>(a.r) + (long long)row * a.ldr + c, H - c);
        v.dh.load(static_cast<const B*>(a.dh) + (long long)row * a.lddh + c, H - c);
      }
      if (a.dr) v.dr.load(static_cast<const X*>(a.dr) + (long long)row * a.lddr + c, H - c);
      if (FULL) v.g.load(static_cast<const B*>(a.gate) + (long long)row * a.ldg + c, H - c);
    }
    load_b(row, c, v);
  };

  Row cur, next;
  if (kAhead) load(blockIdx.x * p.groups + grp, 0, next);
  for (int row0 = blockIdx.x * p.groups; row0 < a.T; row0 += gridDim.x * p.groups, par ^= 1) {
    const int row = row0 + grp;
    const bool live = row < a.T;
    if (kAhead) {
      cur = next;
      load(row + gridDim.x * p.groups, 0, next);
    } else if (kHold) {
      load(row, 0, cur);
    }
    const float gate_t = live && token ? static_cast<const float*>(a.gate)[row] : 1.0f;
    float s[3] = {0.0f, 0.0f, 0.0f};       // r^2, dh w_pre r, b^2
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!kHold) load(row, i, cur);
      float r[8], dh[8], b[8];
      cur.r.get(r), cur.dh.get(dh), cur.b.get(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = __builtin_fmaf(r[j], r[j], s[0]);
        s[1] = __builtin_fmaf(dh[j] * w_pre[i][j], r[j], s[1]);
        s[2] = __builtin_fmaf(b[j], b[j], s[2]);
      }
    }
    row_sums(s, red_a[par], wave, lane, first_wave, p.wpr);
    const float inv_r = 1.0f / __builtin_sqrtf(s[0] * inv_h + a.eps);
    const float inv_b = post ? 1.0f / __builtin_sqrtf(s[2] * inv_h + a.eps) : 1.0f;
    const float m_r = s[1] * inv_r * inv_h;      // mean(v r^)
    float u[ITEMS][8], t[1] = {0.0f};            // t: sum of u b^ (before a token's gate)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      if (!kHold) load(row, i, cur);
      float r[8], dh[8], d[8];
      cur.r.get(r), cur.dh.get(dh), cur.dr.get(d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float rh = r[j] * inv_r;
        acc_pre[i][j] = __builtin_fmaf(dh[j], rh, acc_pre[i][j]);
        d[j] += inv_r * (dh[j] * w_pre[i][j] - rh * m_r);
      }
      if (a.dx && live && c < H) {
        float dx[8];
        const float al = has_b ? a.alpha : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] = al * d[j];
        Vec8<X>::store(static_cast<X*>(a.dx) + (long long)row * a.lddx + c, dx, H - c);
      }
      if (has_b) {
        float b[8], g[8], dg[8];
        cur.b.get(b), cur.g.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float db = d[j] * (b[j] * inv_b), gj = FULL ? g[j] : gate_t;
          dg[j] = db * w_n[i][j];
          acc_b[i][j] = __builtin_fmaf(db, gj, acc_b[i][j]);
          t[0] = FULL ? __builtin_fmaf(dg[j], gj, t[0]) : t[0] + dg[j];
          u[i][j] = d[j] * w_n[i][j] * gj;
        }
        if (FULL && a.dgate && live && c < H)
          Vec8<B>::store(static_cast<B*>(a.dgate) + (long long)row * a.lddg + c, dg, H - c);
      }
    }
    if (!has_b) continue;
    if (post || token) row_sums(t, red_c[par], wave, lane, first_wave, p.wpr);
    if (token && a.dgate && live && gt == 0) static_cast<float*>(a.dgate)[row] = t[0];
    const float m_b = post ? t[0] * gate_t * inv_h : 0.0f;     // mean(u b^)
    if (a.db && live) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (gt + i * stride) * 8;
        if (c < H) {
          if (!kHold) load_b(row, c, cur);
          float b[8];
          cur.b.get(b);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] = inv_b * (u[i][j] - b[j] * inv_b * m_b);
          Vec8<B>::store(static_cast<B*>(a.db) + (long long)row * a.lddb + c, u[i], H - c);
        }
      }
    }
  }

  // The groups' sums are joined in LDS, one plane at a time, then written.
  extern __shared__ float join[];      // [groups - 1][H] when there are several groups
  auto finish = [&](float (&acc)[ITEMS][8], int plane, const float* w, float k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      if (grp > 0 && c < H) Vec8<float>::store(join + (grp - 1) * H + c, acc[i], H - c);
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (gt + i * stride) * 8;
      if (c >= H) continue;
      float f[8], o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = acc[i][j];
      for (int q = 0; q < p.groups - 1; ++q) {
        load_w(join + q * H, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += f[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= k;
      if (w) {
        load_w(w, c, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= f[j];
      }
      Vec8<float>::store(p.part + ((long long)plane * gridDim.x + blockIdx.x) * H + c, o, H - c);
    }
  };
  if (a.dw_pre) finish(acc_pre, 0, nullptr, 1.0f);
  if (a.dw_post) finish(acc_b, 1, channel ? static_cast<const float*>(a.gate) : nullptr, a.beta);
  if (a.dgate && channel) finish(acc_b, 2, a.w_post, a.beta);
}

// out[c] = sum over the slots of part[slot][c]: 64 channels a workgroup, its 16
// waves taking a sixteenth of the slots each, added in wave order (blockIdx.y
// picks the plane).
__global__ __launch_bounds__(1024) void channel_sum_kernel(const float* part, int slots, int H,
                                                            float* o0, float* o1, float* o2) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
  if (!out) return;
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* src = part + (long long)blockIdx.y * slots * H;
  float t = 0.0f;
  if (c < H) {
    const int lo = slots * q / 16, hi = slots * (q + 1) / 16;
#pragma unroll 16
    for (int i = lo; i < hi; ++i) t += src[(long long)i * H + c];
  }
  s[q][lane] = t;
  __syncthreads();
  if (q == 0 && c < H) {
    t = s[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) t += s[i][lane];
    out[c] = t;
  }
}

int bwd_blocks(int T, int H, int cus) {
  const int groups = row_shape(H, kBwdWaves).groups;
  const int need = (T + groups - 1) / groups;
  return need < cus ? need : cus;
}

constexpr int kMaxCus = 256;    // workspace bound: blocks never exceed this

template <typename E>
struct Type {
  using type = E;
};

// f(X, B, items) with the row types and the vectors a thread owns as types
template <typename F>
void with_types(moe_dtype_t x, moe_dtype_t b, int items, F f) {
  auto with_items = [&](auto xt, auto bt) {
    if (items == 1) f(xt, bt, std::integral_constant<int, 1>{});
    else if (items == 2) f(xt, bt, std::integral_constant<int, 2>{});
    else f(xt, bt, std::integral_constant<int, 4>{});
  };
  if (x == MOE_BF16) {
    if (b == MOE_BF16) with_items(Type<bf16_t>{}, Type<bf16_t>{});
    else with_items(Type<bf16_t>{}, Type<float>{});
  } else {
    if (b == MOE_BF16) with_items(Type<float>{}, Type<bf16_t>{});
    else with_items(Type<float>{}, Type<float>{});
  }
}

bool bad_ld(const void* p, long long ld, int H) { return p && ld < H; }

}  // namespace

extern "C" moe_status_t moe_block_norm(const moe_block_norm_args* args, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_block_norm_args& a = *args;
  if (a.T < 0 || a.H < 1 || a.H > kMaxWidth || !(a.eps > 0.0f)) return MOE_ERR_SHAPE;
  if (a.T > kMaxRows || !valid_dtype(a.x_dtype) || !valid_dtype(a.b_dtype) ||
      a.gate_mode < MOE_GATE_NONE || a.gate_mode > MOE_GATE_FULL)
    return MOE_ERR_UNSUPPORTED;
  if (bad_ld(a.x, a.ldx, a.H) || bad_ld(a.b, a.ldb, a.H) || bad_ld(a.h, a.ldh, a.H) ||
      (a.b && bad_ld(a.r, a.ldr, a.H)) ||
      (a.gate_mode == MOE_GATE_FULL && bad_ld(a.gate, a.ldg, a.H)))
    return MOE_ERR_SHAPE;
  if (a.T == 0) return MOE_OK;
  if (!a.x || (a.b && !a.r) || (!a.b && !a.h) || (a.h && !a.w_pre) ||
      (a.b && a.gate_mode != MOE_GATE_NONE && !a.gate))
    return MOE_ERR_NULL;
  if (!element_aligned(a.x, a.x_dtype) || !element_aligned(a.r, a.x_dtype) ||
      !element_aligned(a.b, a.b_dtype) || !element_aligned(a.h, a.b_dtype) ||
      !element_aligned(a.w_pre, MOE_F32) || !element_aligned(a.w_post, MOE_F32) ||
      !element_aligned(a.gate, a.gate_mode == MOE_GATE_FULL ? a.b_dtype : MOE_F32))
    return MOE_ERR_ALIGN;
  if (moe_status_t s = check_device()) return s;
  const RowShape s = row_shape(a.H, kFwdWaves);
  FwdParams p{a, s.wpr, s.groups};
  if (!a.b) p.a.gate_mode = MOE_GATE_NONE;
  // a launch holds less than 2^32 threads; longer batches go round the kernel's loop
  const int need = (a.T - 1) / s.groups + 1, blocks = need < kMaxBlocks ? need : kMaxBlocks;
  with_types(a.x_dtype, a.b_dtype, s.items, [&](auto x, auto b, auto items) {
    using X = typename decltype(x)::type;
    using B = typename decltype(b)::type;
    hipLaunchKernelGGL((block_norm_kernel<X, B, decltype(items)::value>), dim3(blocks),
                       dim3(s.wpr * s.groups * 64), 0, stream, p);
  });
  return launch_status();
}

extern "C" size_t moe_block_norm_backward_workspace_bytes(int T, int H) {
  if (T <= 0 || H <= 0 || H > kMaxWidth) return 0;
  return (size_t)bwd_blocks(T, H, kMaxCus) * 3 * H * sizeof(float);
}

extern "C" moe_status_t moe_block_norm_backward(const moe_block_norm_bwd_args* args, void* ws,
                                                size_t ws_bytes, hipStream_t stream) {
  if (!args) return MOE_ERR_NULL;
  const moe_block_norm_bwd_args& a = *args;
  if (a.T < 0 || a.H < 1 || a.H > kMaxWidth || !(a.eps > 0.0f)) return MOE_ERR_SHAPE;
  if (a.T > kMaxRows || !valid_dtype(a.x_dtype) || !valid_dtype(a.b_dtype) ||
      a.gate_mode < MOE_GATE_NONE || a.gate_mode > MOE_GATE_FULL)
    return MOE_ERR_UNSUPPORTED;
  const bool full = a.gate_mode == MOE_GATE_FULL;
  if (bad_ld(a.r, a.ldr, a.H) || bad_ld(a.dr, a.lddr, a.H) || bad_ld(a.dh, a.lddh, a.H) ||
      bad_ld(a.b, a.ldb, a.H) || bad_ld(a.dx, a.lddx, a.H) || bad_ld(a.db, a.lddb, a.H) ||
      (full && (bad_ld(a.gate, a.ldg, a.H) || bad_ld(a.dgate, a.lddg, a.H))))
    return MOE_ERR_SHAPE;
  const bool sums = a.dw_pre || a.dw_post || (a.dgate && a.gate_mode == MOE_GATE_CHANNEL);
  if (a.T > 0) {
    if ((!a.dr && !a.dh) || (a.dh && (!a.r || !a.w_pre)) || (a.dw_pre && !a.dh) ||
        (!a.b && (a.db || a.dgate || a.dw_post)) || (a.dw_post && !a.w_post) ||
        (a.b && a.gate_mode != MOE_GATE_NONE && !a.gate) ||
        (a.dgate && a.gate_mode == MOE_GATE_NONE))
      return MOE_ERR_NULL;
    const moe_dtype_t gd = full ? a.b_dtype : MOE_F32;
    if (!element_aligned(a.r, a.x_dtype) || !element_aligned(a.dr, a.x_dtype) ||
        !element_aligned(a.dx, a.x_dtype) || !element_aligned(a.dh, a.b_dtype) ||
        !element_aligned(a.b, a.b_dtype) || !element_aligned(a.db, a.b_dtype) ||
        !element_aligned(a.w_pre, MOE_F32) || !element_aligned(a.w_post, MOE_F32) ||
        !element_aligned(a.gate, gd) || !element_aligned(a.dgate, gd) ||
        !element_aligned(a.dw_pre, MOE_F32) || !element_aligned(a.dw_post, MOE_F32))
      return MOE_ERR_ALIGN;
    if (sums) {
      if (!ws || ws_bytes < moe_block_norm_backward_workspace_bytes(a.T, a.H))
        return MOE_ERR_WORKSPACE;
      if (!aligned16(ws)) return MOE_ERR_ALIGN;
    }
  } else if (!sums) {
    return MOE_OK;
  }
  if (moe_status_t s = check_device()) return s;
  const RowShape s = row_shape(a.H, kBwdWaves);
  int slots = 0;
  if (a.T > 0) {
    int cus = cu_count();
    if (cus < 1 || cus > kMaxCus) cus = kMaxCus;
    slots = bwd_blocks(a.T, a.H, cus);
    BwdParams p{a, s.wpr, s.groups, static_cast<float*>(ws)};
    if (!a.b) p.a.gate_mode = MOE_GATE_NONE;
    const size_t lds = sums ? (size_t)(s.groups - 1) * a.H * sizeof(float) : 0;
    with_types(a.x_dtype, a.b_dtype, s.items, [&](auto x, auto b, auto items) {
      using X = typename decltype(x)::type;
      using B = typename decltype(b)::type;
      constexpr int ITEMS = decltype(items)::value < 2 ? 1 : 2;      // 16 waves never need 4
      if (p.a.gate_mode == MOE_GATE_FULL)
        hipLaunchKernelGGL((block_norm_bwd_kernel<X, B, ITEMS, true>), dim3(slots),
                           dim3(s.wpr * s.groups * 64), lds, stream, p);
      else
        hipLaunchKernelGGL((block_norm_bwd_kernel<X, B, ITEMS, false>), dim3(slots),
                           dim3(s.wpr * s.groups * 64), lds, stream, p);
    });
    if (moe_status_t st = launch_status()) return st;
  }
  if (sums)
    hipLaunchKernelGGL(channel_sum_kernel, dim3((a.H + 63) / 64, 3), dim3(1024), 0, stream,
                       static_cast<const float*>(ws), slots, a.H, a.dw_pre, a.dw_post,
                       a.gate_mode == MOE_GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr);
  return launch_status();
}
