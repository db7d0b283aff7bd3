// token_norm.cu — RMSNorm of whole token rows with the residual's addition,
// bf16 or 8-bit output, its backward, and 8-bit rows with scales: the
// HBM-bound steps between an MM-DiT block's residual stream and its QKV
// projection.
//
// Forward, per row of C values (h and y one bf16 rounding each, everything
// else fp32):
//     h = bf16(x + res)                      (without res: h = x)
//     r = (mean_c h_c^2 + eps)^(-1/2)
//     z = g * h * r,   y = bf16(z)
//     8-bit output: m = max(max_c |z_c|, 2^-80),  s = m / 448,  y8 = e4m3(448 z / m)
// (the fp32 sum of two bf16 values rounded again to bf16 is their exact sum
// rounded once: 24 bits are more than 2 * 8 + 2).
// Backward, with n = h r and u = g * dy:
//     dx = bf16(dh + r (u - n mean_c(u n))),   dg_c = sum_t dy n
//
// Row layout: a row's 16-byte chunks (8 values) are dealt round-robin to the
// lanes that share it, one warp (C <= 1024) or one block, V chunks a lane,
// kept in registers between the reduction and the output: every array is
// read and written once.
#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"

namespace jattn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-80f;  // smallest row maximum a scale is made from
constexpr int kRowThreads = 256;        // warp rows: 8 rows per block
constexpr int kWarpRowMaxC = 1024;      // wider rows take a block each
constexpr int kMaxBlockRow = 512;       // threads of a block row: 4 chunks a lane cover JATTN_MAX_WIDTH
constexpr int kBwdParts = 304;          // blocks of the backward at most: two for each of 152 SMs

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
// Four fp32 values as e4m3 bytes, lowest first (nearest even; beyond 448: 448; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void load8f(const float* g, int chunk, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g) + 2 * chunk);
  const float4 b = __ldg(reinterpret_cast<const float4*>(g) + 2 * chunk + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Reduction over the lanes that share a row: the warp, or the whole block
// (red: one float per warp; the buffer is free again after the next call's
// first barrier, so two buffers used in turn need no third barrier).
template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? fmaxf(a, b) : a + b;
}
template <bool kBlock, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kBlock) {
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.f;  // maxima are of magnitudes
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
    v = __shfl_sync(0xffffffffu, v, 0);
  }
  return v;
}

struct NormArgs {
  const uint4* x;
  const uint4* res;  // or null
  const float* g;
  int64_t T;
  int chunks;  // C / 8
  float inv_c, eps;
  uint4* h;     // null without res
  uint4* y;     // bf16 output
  uint2* y8;    // 8-bit output
  float* s;     // its scales
  float* r;     // or null
};

enum class RowOp { kNorm, kNormE4m3, kQuant };

template <int V, bool kBlock, RowOp kOp>
__global__ void __launch_bounds__(kBlock ? kMaxBlockRow : kRowThreads) token_rows_kernel(const NormArgs a) {
  __shared__ float red[2][16];
  griddep_launch_dependents();
  griddep_wait();
  const int lanes = kBlock ? blockDim.x : 32;
  const int lane = kBlock ? threadIdx.x : threadIdx.x % 32;
  const int64_t row = kBlock ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32;
  if (row >= a.T) return;  // a whole warp (kBlock: never)
  const int64_t base = row * a.chunks;
  uint4 w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * lanes + lane;
    w[i] = c < a.chunks ? a.x[base + c] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (kOp != RowOp::kQuant && a.res) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float u[8], v[8];
        unpack8(w[i], u);
        unpack8(a.res[base + c], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = __fadd_rn(u[j], v[j]);
        w[i] = pack8(u);
        a.h[base + c] = w[i];
      }
    }
  }
  float r = 1.f;
  if constexpr (kOp != RowOp::kQuant) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float u[8];
      unpack8(w[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(u[j], u[j], ss);
    }
    ss = row_reduce<kBlock, false>(ss, red[0]);
    r = __frsqrt_rn(fmaf(ss, a.inv_c, a.eps));
    if (lane == 0 && a.r) a.r[row] = r;
  }
  auto z8 = [&](int i, int c, float (&z)[8]) {
    unpack8(w[i], z);
    if constexpr (kOp != RowOp::kQuant) {
      float g[8];
      load8f(a.g, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = __fmul_rn(__fmul_rn(z[j], r), g[j]);
    }
  };
  if constexpr (kOp == RowOp::kNorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float z[8];
        z8(i, c, z);
        a.y[base + c] = pack8(z);
      }
    }
  } else {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float z[8];
        z8(i, c, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(z[j]));
      }
    }
    m = row_reduce<kBlock, true>(m, red[1]);
    // 448 z / m as 0.875 z over m / 512, which stays in range for every z and is exact for a bf16 z:
    // midpoints of e4m3 (common then) stay midpoints.  The product with the reciprocal and one residual
    // correction (Markstein, 1990) rounds as the quotient does.
    m = fmaxf(m, kAmaxFloor);
    if (lane == 0) a.s[row] = __fdiv_rn(m, kE4m3Max);
    m = __fmul_rn(m, 1.f / 512);
    const float inv = __frcp_rn(m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float z[8];
        z8(i, c, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = __fmul_rn(z[j], kE4m3Max / 512), q = __fmul_rn(v, inv);
          z[j] = fmaf(fmaf(-q, m, v), inv, q);
        }
        a.y8[base + c] = make_uint2(pack_e4m3x4(z[0], z[1], z[2], z[3]), pack_e4m3x4(z[4], z[5], z[6], z[7]));
      }
    }
  }
}

struct NormBwdArgs {
  const uint4* dy;
  const uint4* dh;  // or null; may be dx
  const uint4* h;
  const float* r;
  const float* g;
  int64_t T;
  int chunks;
  float inv_c;
  uint4* dx;
  float* part;  // [gridDim.x, C] partial sums of dg
};

// Rows in a fixed stride per block; each lane sums dy n of its columns over
// the rows it meets, then the block's warps are added in order.
template <int V, bool kBlock>
__global__ void __launch_bounds__(kBlock ? kMaxBlockRow : kRowThreads) token_norm_bwd_kernel(const NormBwdArgs a) {
  extern __shared__ float sums[];  // warp rows: [warps][chunks * 8]
  __shared__ float red[2][16];
  griddep_launch_dependents();
  griddep_wait();
  const int lanes = kBlock ? blockDim.x : 32;
  const int lane = kBlock ? threadIdx.x : threadIdx.x % 32;
  const int rows_per_pass = kBlock ? 1 : kRowThreads / 32;
  float acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int which = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_pass + (kBlock ? 0 : threadIdx.x / 32); row < a.T;
       row += static_cast<int64_t>(gridDim.x) * rows_per_pass) {
    const int64_t base = row * a.chunks;
    uint4 wy[V], wh[V], wd[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      const bool in = c < a.chunks;
      wy[i] = in ? a.dy[base + c] : make_uint4(0u, 0u, 0u, 0u);
      wh[i] = in ? a.h[base + c] : make_uint4(0u, 0u, 0u, 0u);
      wd[i] = in && a.dh ? a.dh[base + c] : make_uint4(0u, 0u, 0u, 0u);
    }
    const float r = a.r[row];
    float un = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float y[8], h[8], g[8];
        unpack8(wy[i], y);
        unpack8(wh[i], h);
        load8f(a.g, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dn = y[j] * (h[j] * r);
          acc[i][j] += dn;
          un = fmaf(dn, g[j], un);
        }
      }
    }
    const float m = row_reduce<kBlock, false>(un, red[which]) * a.inv_c;
    which ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float y[8], h[8], g[8], d[8];
        unpack8(wy[i], y);
        unpack8(wh[i], h);
        unpack8(wd[i], d);
        load8f(a.g, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(r, fmaf(-(h[j] * r), m, y[j] * g[j]), d[j]);
        a.dx[base + c] = pack8(d);
      }
    }
  }
  const int C = a.chunks * 8;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * C;
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        float4* o = reinterpret_cast<float4*>(out) + 2 * c;
        o[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        o[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
  } else {
    float4* mine = reinterpret_cast<float4*>(sums + static_cast<size_t>(threadIdx.x / 32) * C);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * lanes + lane;
      if (c < a.chunks) {
        mine[2 * c] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        mine[2 * c + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kRowThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kRowThreads / 32; ++w) s += sums[w * C + c];
      out[c] = s;
    }
  }
}

// dg = the sum of the blocks' partial sums, in a fixed order: 32 columns a
// block, 8 threads a column.
__global__ void __launch_bounds__(256) dg_sum_kernel(const float* part, int parts, int C, float* dg) {
  __shared__ float sums[8][33];
  griddep_launch_dependents();
  griddep_wait();
  const int col = threadIdx.x % 32, grp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + col;
  float s = 0.f;
  if (c < C)
    for (int p = grp; p < parts; p += 8) s += part[static_cast<size_t>(p) * C + c];
  sums[grp][col] = s;
  __syncthreads();
  if (grp == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][col];
    dg[c] = s;
  }
}

int block_row_threads(int chunks, int per_lane) { return ((chunks + per_lane - 1) / per_lane + 31) / 32 * 32; }

template <RowOp kOp>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t st) {
  if (a.chunks * 8 <= kWarpRowMaxC) {
    constexpr int kRows = kRowThreads / 32;
    const int64_t blocks = (a.T + kRows - 1) / kRows;
    const dim3 grid(static_cast<unsigned>(blocks));
    switch ((a.chunks + 31) / 32) {
      case 1: return launch_pdl(token_rows_kernel<1, false, kOp>, grid, dim3(kRowThreads), 0, st, a);
      case 2: return launch_pdl(token_rows_kernel<2, false, kOp>, grid, dim3(kRowThreads), 0, st, a);
      case 3: return launch_pdl(token_rows_kernel<3, false, kOp>, grid, dim3(kRowThreads), 0, st, a);
      default: return launch_pdl(token_rows_kernel<4, false, kOp>, grid, dim3(kRowThreads), 0, st, a);
    }
  }
  return launch_pdl(token_rows_kernel<4, true, kOp>, dim3(static_cast<unsigned>(a.T)),
                    dim3(block_row_threads(a.chunks, 4)), 0, st, a);
}

}  // namespace

cudaError_t launch_add_norm(const TokenNorm& t, cudaStream_t st) {
  NormArgs a;
  a.x = reinterpret_cast<const uint4*>(t.x);
  a.res = reinterpret_cast<const uint4*>(t.res);
  a.g = t.g;
  a.T = t.T;
  a.chunks = t.C / 8;
  a.inv_c = 1.f / static_cast<float>(t.C);
  a.eps = t.eps;
  a.h = reinterpret_cast<uint4*>(t.h);
  a.y = reinterpret_cast<uint4*>(t.y);
  a.y8 = reinterpret_cast<uint2*>(t.y8);
  a.s = t.s;
  a.r = t.r;
  if (t.y) return launch_rows<RowOp::kNorm>(a, st);
  return t.g ? launch_rows<RowOp::kNormE4m3>(a, st) : launch_rows<RowOp::kQuant>(a, st);
}

int add_norm_bwd_parts(int T, int C) {
  const int64_t rows = C <= kWarpRowMaxC ? kRowThreads / 32 : 1;
  const int64_t blocks = (T + rows - 1) / rows;
  return static_cast<int>(blocks < kBwdParts ? blocks : kBwdParts);
}

cudaError_t launch_add_norm_bwd(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const float* r,
                                const float* g, int T, int C, uint16_t* dx, float* part, int parts,
                                cudaStream_t st) {
  NormBwdArgs a;
  a.dy = reinterpret_cast<const uint4*>(dy);
  a.dh = reinterpret_cast<const uint4*>(dh);
  a.h = reinterpret_cast<const uint4*>(h);
  a.r = r;
  a.g = g;
  a.T = T;
  a.chunks = C / 8;
  a.inv_c = 1.f / static_cast<float>(C);
  a.dx = reinterpret_cast<uint4*>(dx);
  a.part = part;
  const dim3 grid(static_cast<unsigned>(parts));
  if (C <= kWarpRowMaxC) {
    const size_t smem = static_cast<size_t>(kRowThreads / 32) * C * 4;  // at most 32 KB
    switch ((a.chunks + 31) / 32) {
      case 1: return launch_pdl(token_norm_bwd_kernel<1, false>, grid, dim3(kRowThreads), smem, st, a);
      case 2: return launch_pdl(token_norm_bwd_kernel<2, false>, grid, dim3(kRowThreads), smem, st, a);
      case 3: return launch_pdl(token_norm_bwd_kernel<3, false>, grid, dim3(kRowThreads), smem, st, a);
      default: return launch_pdl(token_norm_bwd_kernel<4, false>, grid, dim3(kRowThreads), smem, st, a);
    }
  }
  return launch_pdl(token_norm_bwd_kernel<4, true>, grid, dim3(block_row_threads(a.chunks, 4)), 0, st, a);
}

cudaError_t launch_dg_sum(const float* part, int parts, int C, float* dg, cudaStream_t st) {
  return launch_pdl(dg_sum_kernel, dim3(static_cast<unsigned>((C + 31) / 32)), dim3(256), 0, st, part, parts, C, dg);
}

}  // namespace jattn
