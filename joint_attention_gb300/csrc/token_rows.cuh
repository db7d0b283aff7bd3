// token_rows.cuh — what the kernels over whole token rows share: a row's 16-byte
// chunks in packed fp32 pairs, the reduction over the warps of a row, and the row
// layout of a width.
#pragma once
#include <cuda_bf16.h>

#include "sm103_ptx.cuh"

namespace jattn {
namespace {

constexpr int kMaxWarps = 16;  // sharing a row: 4 chunks a lane cover JATTN_MAX_WIDTH

// Warps of a block: 8 (8 / G rows), or one row's.
constexpr int block_warps(int G) { return G > 8 ? G : 8; }

// 8 bf16 values and packed fp32 pairs.
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ F8 unpack8(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f2_make(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  return f;
}
__device__ __forceinline__ uint32_t pack2(uint64_t p) {
  float a, b;
  f2_split(p, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
  return make_uint4(pack2(f.p[0]), pack2(f.p[1]), pack2(f.p[2]), pack2(f.p[3]));
}
__device__ __forceinline__ F8 load8f(const float* g, int chunk) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(g) + 2 * chunk);
  const float4 b = __ldg(reinterpret_cast<const float4*>(g) + 2 * chunk + 1);
  return F8{{f2_make(a.x, a.y), f2_make(a.z, a.w), f2_make(b.x, b.y), f2_make(b.z, b.w)}};
}
// Reduction over the G warps that share a row (red: a float for each warp of
// the block; free again after the next call's barrier, so two used in turn need
// no second barrier).
template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? fmaxf(a, b) : a + b;
}
template <int G, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (G > 1) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, group = warp / G;
    if (lane == 0) red[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * G) : "memory");
    v = red[group * G + (lane & (G - 1))];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

// The sum of `parts` partial sums, `step` floats apart, of each of kCols neighbouring
// columns (8: a 32-byte sector) by a block of 256 threads, 256 / kCols a column, in a fixed
// order: returned in the first kCols threads.  Columns from `cols` on are not read.
template <int kCols = 8>
__device__ __forceinline__ float column_sum(const float* from, int parts, size_t step, int cols = kCols) {
  constexpr int kGroups = 256 / kCols;
  __shared__ float sums[kGroups][kCols + 1];
  const int col = threadIdx.x % kCols, grp = threadIdx.x / kCols;
  constexpr int kAhead = 10;
  if (kCols > 8 && col >= cols) parts = 0;
  float s = 0.f;
  for (int p0 = grp; p0 < parts; p0 += kGroups * kAhead) {
    float v[kAhead];  // all on their way at once
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i] = p0 + kGroups * i < parts ? from[(p0 + kGroups * i) * step + col] : 0.f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) s += v[i];
  }
  sums[grp][col] = s;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) s += sums[i][col];
  }
  return s;
}

// Calls f(V, G) with the row layout of a width: as few warps as hold it at
// four chunks a lane.
template <int kV, int kG>
struct Layout {
  static constexpr int V = kV, G = kG;
};
template <typename F>
cudaError_t with_layout(int chunks, F f) {
  if (chunks <= 32) return f(Layout<1, 1>());
  if (chunks <= 64) return f(Layout<2, 1>());
  if (chunks <= 96) return f(Layout<3, 1>());
  if (chunks <= 128) return f(Layout<4, 1>());
  if (chunks <= 192) return f(Layout<3, 2>());
  if (chunks <= 256) return f(Layout<4, 2>());
  if (chunks <= 384) return f(Layout<3, 4>());
  if (chunks <= 512) return f(Layout<4, 4>());
  if (chunks <= 768) return f(Layout<3, 8>());
  if (chunks <= 1024) return f(Layout<4, 8>());
  if (chunks <= 1536) return f(Layout<3, 16>());
  return f(Layout<4, 16>());
}

}  // namespace
}  // namespace jattn
