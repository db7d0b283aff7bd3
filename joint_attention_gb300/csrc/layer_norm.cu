// layer_norm.cu — LayerNorm of whole token rows with the residual's addition, a
// gain and a bias of the model's or of each batch item's own (the modulated norms
// of an MM-DiT block), and its backward with the gradients of gain and bias.
//
// Forward, per row of C values of item i (h and y one bf16 rounding each, the rest
// fp32):
//     h = bf16(x + res)                               (without res: h = x)
//     mu = mean_c h_c,  r = (mean_c (h_c - mu)^2 + eps)^(-1/2)
//     y = bf16(g_i (h - mu) r + b_i)                  (without b: 0)
// Backward, with n = (h - mu) r and u = g_i dy:
//     dx = bf16(dh + r (u - mean_c(u) - n mean_c(u n)))
//     dg_i = sum over the item's rows of dy n,  db_i = sum of dy
//
// The mean is taken twice: m0 from the row as it is, then delta = mean(h - m0)
// beside the sum of squares, var = mean((h - m0)^2) - delta^2.  m0 is off by a few
// fp32 roundings of the row's magnitude, which for a row of large equal values would
// be all that n is made of; delta takes them out at one instruction a value.  Both
// means add terms that are divided by C first, so that finite rows have finite means.
//
// Row layout as in token_norm.cu: a row stays in the registers of 1 to 16 warps
// between the sums and the output, every array is read and written once, arithmetic
// in packed fp32 pairs.
#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"
#include "token_rows.cuh"

namespace jattn {
namespace {

constexpr int kLnBwdBlocks = 304;  // blocks of the backward at least, where there are rows: two for each of 152 SMs

// Two sums over the G warps that share a row, joined as row_reduce joins one.
template <int G>
__device__ __forceinline__ float2 row_sums(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (G > 1) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, group = warp / G;
    if (lane == 0) red[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * G) : "memory");
    const float2 v = red[group * G + (lane & (G - 1))];
    a = v.x;
    b = v.y;
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
  }
  return make_float2(a, b);
}

struct LnArgs {
  const uint4* x;
  const uint4* res;  // or null
  const float* g;    // [items, C]
  const float* b;    // likewise, or null
  int64_t T;
  uint32_t item_rows;
  int chunks;  // C / 8
  float inv_c, eps;
  uint4* h;  // null without res
  uint4* y;
  float *mean, *r;  // or null
};

template <int V, int G>
__global__ void __launch_bounds__(32 * block_warps(G)) layer_norm_kernel(const LnArgs a) {
  __shared__ float red[kMaxWarps];
  __shared__ float2 red2[kMaxWarps];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kLanes = 32 * G, kRows = block_warps(G) / G;
  const int lane = threadIdx.x % kLanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kLanes;
  if (row >= a.T) return;  // all warps of a row
  const int64_t base = row * a.chunks;
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * kLanes + lane;
    w[i] = c < a.chunks ? a.x[base + c] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (a.res) {
    uint4 e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      e[i] = c < a.chunks ? a.res[base + c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      F8 u = unpack8(w[i]), v = unpack8(e[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) u.p[j] = f2_add(u.p[j], v.p[j]);
      w[i] = pack8(u);
      if (c < a.chunks) a.h[base + c] = w[i];
    }
  }
  const uint64_t inv2 = f2_make(a.inv_c, a.inv_c);
  uint64_t s2 = 0;  // (0, 0)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const F8 u = unpack8(w[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = f2_fma(u.p[j], inv2, s2);
  }
  float s0, s1;
  f2_split(s2, s0, s1);
  const float m0 = row_reduce<G, false>(s0 + s1, red);
  const uint64_t neg_m = f2_make(-m0, -m0);
  F8 d[V];
  uint64_t d2 = 0, q2 = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * kLanes + lane;
    d[i] = unpack8(w[i]);
    const uint64_t off = c < a.chunks ? neg_m : 0;  // chunks past the row stay zeros
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[i].p[j] = f2_add(d[i].p[j], off);
      d2 = f2_fma(d[i].p[j], inv2, d2);
      q2 = f2_fma(d[i].p[j], d[i].p[j], q2);
    }
  }
  float d0, d1, q0, q1;
  f2_split(d2, d0, d1);
  f2_split(q2, q0, q1);
  const float2 sums = row_sums<G>(d0 + d1, q0 + q1, red2);
  const float delta = sums.x;
  float var = fmaf(sums.y, a.inv_c, -delta * delta);
  if (var < 0.f) var = 0.f;               // (NaN stays NaN)
  if (sums.y > 0x1.fffffep127f) var = sums.y;  // squares beyond the fp32 range: r = 0
  const float r = __frsqrt_rn(var + a.eps);
  if (lane == 0) {
    if (a.mean) a.mean[row] = m0 + delta;
    if (a.r) a.r[row] = r;
  }
  const uint32_t item = static_cast<uint32_t>(row) / a.item_rows;
  const float* g = a.g + static_cast<int64_t>(item) * a.chunks * 8;
  const float* b = a.b ? a.b + static_cast<int64_t>(item) * a.chunks * 8 : nullptr;
  const uint64_t r2 = f2_make(r, r), shift = f2_make(-delta * r, -delta * r);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * kLanes + lane;
    if (c < a.chunks) {
      const F8 gv = load8f(g, c);
      F8 y;
      if (b) {
        const F8 bv = load8f(b, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y.p[j] = f2_fma(f2_fma(d[i].p[j], r2, shift), gv.p[j], bv.p[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y.p[j] = f2_mul(f2_fma(d[i].p[j], r2, shift), gv.p[j]);
      }
      a.y[base + c] = pack8(y);
    }
  }
}

struct LnBwdArgs {
  const uint4* dy;
  const uint4* dh;  // or null; may be dx
  const uint4* h;
  const float *mean, *r;
  const float* g;  // [items, C]
  int item_rows, parts;  // rows and blocks of an item
  int chunks;
  float inv_c;
  uint4* dx;
  float* part;  // [items * parts, kSums, C] partial sums of dg (and of db)
};

// Blocks p of an item take its rows in a fixed stride; each lane sums dy n (and dy)
// of its columns over the rows it meets, then the block's rows are added in order.
template <int V, int G, bool kBias>
__global__ void __launch_bounds__(32 * block_warps(G)) layer_norm_bwd_kernel(const LnBwdArgs a) {
  constexpr int kLanes = 32 * G, kRows = block_warps(G) / G, kSums = kBias ? 2 : 1;
  extern __shared__ __align__(16) float sums[];  // [rows of a block][C], where it has several
  __shared__ float2 red[2][32];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const int item = blockIdx.x / a.parts, p = blockIdx.x - item * a.parts;
  const int64_t first = static_cast<int64_t>(item) * a.item_rows, end = first + a.item_rows;
  const int64_t step = static_cast<int64_t>(a.parts) * kRows;
  const int C = a.chunks * 8;
  F8 g[V];
  uint64_t acc[kSums][V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * kLanes + lane;
    g[i] = load8f(a.g + static_cast<int64_t>(item) * C, c < a.chunks ? c : 0);
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[k][i][j] = 0;
  }
  int it = 0;
  for (int64_t row = first + static_cast<int64_t>(p) * kRows + slot; row < end; row += step, ++it) {
    const int64_t base = row * a.chunks;
    const float mean = a.mean[row], r = a.r[row];
    uint4 wy[V], wh[V], wd[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      const bool in = c < a.chunks;
      wy[i] = in ? a.dy[base + c] : make_uint4(0u, 0u, 0u, 0u);
      wh[i] = in ? a.h[base + c] : make_uint4(0u, 0u, 0u, 0u);
      wd[i] = in && a.dh ? a.dh[base + c] : make_uint4(0u, 0u, 0u, 0u);
    }
    const uint64_t r2 = f2_make(r, r), neg_mean = f2_make(-mean, -mean);
    F8 n[V], u[V];
    uint64_t u2 = 0, un2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const F8 y = unpack8(wy[i]);
      n[i] = unpack8(wh[i]);
      u[i] = y;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[i].p[j] = f2_mul(f2_add(n[i].p[j], neg_mean), r2);
        u[i].p[j] = f2_mul(y.p[j], g[i].p[j]);
        acc[0][i][j] = f2_fma(y.p[j], n[i].p[j], acc[0][i][j]);
        if constexpr (kBias) acc[1][i][j] = f2_add(acc[1][i][j], y.p[j]);
        u2 = f2_add(u2, u[i].p[j]);
        un2 = f2_fma(u[i].p[j], n[i].p[j], un2);  // chunks past the row: u is zero
      }
    }
    float u0, u1, un0, un1;
    f2_split(u2, u0, u1);
    f2_split(un2, un0, un1);
    const float2 s = row_sums<G>(u0 + u1, un0 + un1, red[it & 1]);
    const float mu = -s.x * a.inv_c, mn = -s.y * a.inv_c;
    const uint64_t mu2 = f2_make(mu, mu), mn2 = f2_make(mn, mn);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      F8 o = unpack8(wd[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) o.p[j] = f2_fma(r2, f2_fma(n[i].p[j], mn2, f2_add(u[i].p[j], mu2)), o.p[j]);
      if (c < a.chunks) a.dx[base + c] = pack8(o);
    }
  }
  float* out = a.part + static_cast<size_t>(blockIdx.x) * kSums * C;
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    ulonglong2* mine = reinterpret_cast<ulonglong2*>(kRows > 1 ? sums + static_cast<size_t>(slot) * C : out + k * C);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      if (c < a.chunks) {
        mine[2 * c] = make_ulonglong2(acc[k][i][0], acc[k][i][1]);
        mine[2 * c + 1] = make_ulonglong2(acc[k][i][2], acc[k][i][3]);
      }
    }
    if constexpr (kRows > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < C; c += 32 * block_warps(G)) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) s += sums[i * C + c];
        out[k * C + c] = s;
      }
      if (k + 1 < kSums) __syncthreads();
    }
  }
}

// dg and db of an item: its blocks' partial sums, 8 columns a block.
__global__ void __launch_bounds__(256) ln_sum_kernel(const float* part, int parts, int C, int n_sums, float* dg,
                                                     float* db) {
  griddep_launch_dependents();
  griddep_wait();
  const int blocks_c = C / 8;
  const int job = blockIdx.x / blocks_c, at = (blockIdx.x - job * blocks_c) * 8;
  const int item = job / n_sums, k = job - item * n_sums;
  const float s = column_sum(part + (static_cast<size_t>(item) * parts * n_sums + k) * C + at, parts,
                             static_cast<size_t>(n_sums) * C);
  if (threadIdx.x < 8) (k == 0 ? dg : db)[static_cast<size_t>(item) * C + at + threadIdx.x] = s;
}

// The backward's row layout: at most two chunks a lane, because it keeps n, u and
// the sums of both gradients in registers.
template <typename F>
cudaError_t with_bwd_layout(int chunks, F f) {
  if (chunks <= 32) return f(Layout<1, 1>());
  if (chunks <= 64) return f(Layout<2, 1>());
  if (chunks <= 128) return f(Layout<2, 2>());
  if (chunks <= 256) return f(Layout<2, 4>());
  if (chunks <= 512) return f(Layout<2, 8>());
  if (chunks <= 1024) return f(Layout<2, 16>());
  return f(Layout<2, 32>());
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNorm& t, cudaStream_t st) {
  LnArgs a;
  a.x = reinterpret_cast<const uint4*>(t.x);
  a.res = reinterpret_cast<const uint4*>(t.res);
  a.g = t.g;
  a.b = t.b;
  a.T = t.T;
  a.item_rows = static_cast<uint32_t>(t.T / t.items);
  a.chunks = t.C / 8;
  a.inv_c = 1.f / static_cast<float>(t.C);
  a.eps = t.eps;
  a.h = reinterpret_cast<uint4*>(t.h);
  a.y = reinterpret_cast<uint4*>(t.y);
  a.mean = t.mean;
  a.r = t.r;
  return with_layout(a.chunks, [&](auto l) {
    using L = decltype(l);
    constexpr int kWarps = block_warps(L::G), kRows = kWarps / L::G;
    return launch_pdl(layer_norm_kernel<L::V, L::G>, dim3(static_cast<unsigned>((a.T + kRows - 1) / kRows)),
                      dim3(32 * kWarps), 0, st, a);
  });
}

int layer_norm_bwd_parts(int items, int T, int C) {
  int rows = 1;
  with_bwd_layout(C / 8, [&](auto l) {
    rows = block_warps(decltype(l)::G) / decltype(l)::G;
    return cudaSuccess;
  });
  const int most = (T / items + rows - 1) / rows, want = (kLnBwdBlocks + items - 1) / items;
  return most < want ? most : want;
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwd& t, float* part, int parts, cudaStream_t st) {
  LnBwdArgs a;
  a.dy = reinterpret_cast<const uint4*>(t.dy);
  a.dh = reinterpret_cast<const uint4*>(t.dh);
  a.h = reinterpret_cast<const uint4*>(t.h);
  a.mean = t.mean;
  a.r = t.r;
  a.g = t.g;
  a.item_rows = t.T / t.items;
  a.parts = parts;
  a.chunks = t.C / 8;
  a.inv_c = 1.f / static_cast<float>(t.C);
  a.dx = reinterpret_cast<uint4*>(t.dx);
  a.part = part;
  return with_bwd_layout(a.chunks, [&](auto l) {
    using L = decltype(l);
    constexpr int kWarps = block_warps(L::G), kRows = kWarps / L::G;
    const size_t smem = kRows > 1 ? static_cast<size_t>(kRows) * t.C * sizeof(float) : 0;  // at most 16 KB
    auto kernel = t.db ? layer_norm_bwd_kernel<L::V, L::G, true> : layer_norm_bwd_kernel<L::V, L::G, false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(t.items * parts)), dim3(32 * kWarps), smem, st, a);
  });
}

cudaError_t launch_layer_norm_sums(const float* part, int parts, const LayerNormBwd& t, cudaStream_t st) {
  const int n_sums = t.db ? 2 : 1;
  return launch_pdl(ln_sum_kernel, dim3(static_cast<unsigned>(t.C / 8 * n_sums * t.items)), dim3(256), 0, st, part,
                    parts, t.C, n_sums, t.dg, t.db);
}

}  // namespace jattn
