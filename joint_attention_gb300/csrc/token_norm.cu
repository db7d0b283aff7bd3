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
// lanes of the G warps that share it (1 for C <= 1024, 2 up to 2048, ...), at
// most four chunks a lane, kept in registers between the reduction and the
// output: every array is read and written once.  A block of 8 warps holds 8 / G
// rows (16 warps for G = 16); warps of a row join their sums through shared
// memory and a barrier of their own.  The arithmetic is in packed fp32 pairs: the
// kernels are bound by HBM only while they spend some 10 instructions on a
// value.  Four chunks a lane, that is few warps a row and much in flight for
// each, measured best (9524 x 2048 to 8 bits, at an earlier state, 26.3 us with
// 4, 29.0 with 2, 33.6 with 1, 27.9 with 8).
//
// Measured (device time, inputs out of L2; the copy rate is 6.77 TB/s): forward
// 17616 x 768 17.7 us (6.1 TB/s), 32768 x 4096 155 us (6.9 TB/s); to 8 bits 9524
// x 2048 24.8 us (5.5 TB/s: 16 instructions a value; 29.6 us with gains of 1,
// where ties of e4m3 are common); rows to 8 bits 9524 x 2048 10.0 us (5.9 TB/s); backward 17616 x 768 20.3 us with the sum of dg (5.3 TB/s:
// two launches, and 7.2 rows a warp).
#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"

namespace jattn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 0x1p-80f;  // smallest row maximum a scale is made from
constexpr int kMaxWarps = 16;         // sharing a row: 4 chunks a lane cover JATTN_MAX_WIDTH
constexpr int kBwdParts = 304;        // blocks of the backward at most: two for each of 152 SMs

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
// Four fp32 values as e4m3 bytes, lowest first (nearest even; beyond 448: 448; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(uint64_t ab, uint64_t cd) {
  float a, b, c, d;
  f2_split(ab, a, b);
  f2_split(cd, c, d);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The rare path of norm rows to 8 bits: values that the fp32 arithmetic cannot
// place on one side of a midpoint of e4m3 (about one in 110 000).  r cancels in 448
// z / m but for its power of two (rz), with which z = h rz g is exact as the sum of
// two floats, and so is m, the largest of the row's: 2 * 448 |z| and the sum of the
// neighbours times m are compared exactly.  y8 is the quotient of these rounded to
// fp32 and then to e4m3, as a conversion from a wider type does it: up to half an
// fp32 step from the midpoint is a tie.
//
// The second float of the row's largest |z| (m: the first): the largest of those
// of the values that round to m.
__device__ __noinline__ float max_low(const uint4* h, const float* g, int chunks, float rz, float m) {
  const uint64_t r2 = f2_make(rz, rz);
  float low = -m;  // below any
#pragma unroll 4
  for (int c = threadIdx.x % 32; c < chunks; c += 32) {
    const F8 u = unpack8(h[c]), gv = load8f(g, c);
    float z[8];
    bool here = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f2_split(f2_mul(f2_mul(u.p[j], r2), gv.p[j]), z[2 * j], z[2 * j + 1]);
      here |= fabsf(z[2 * j]) == m || fabsf(z[2 * j + 1]) == m;
    }
    if (here) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[2], y[2];
        f2_split(u.p[j / 2], x[0], x[1]);
        f2_split(gv.p[j / 2], y[0], y[1]);
        const float zl = __fmaf_rn(__fmul_rn(x[j % 2], rz), y[j % 2], -z[j]);
        if (fabsf(z[j]) == m) low = fmaxf(low, copysignf(1.f, z[j]) * zl);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, o));
  return low;
}
__device__ __forceinline__ float e4m3_magnitude(uint32_t code) {
  const uint32_t e = code >> 3 & 15, f = code & 7;
  return e ? __uint_as_float((e + 120) << 23 | f << 20) : f * 0x1p-9f;
}
// Whether a value h whose fp32 quotient's range (lo, hi) holds a midpoint rounds
// to the upper of its neighbours, code.  m, low: the row's largest |z|.
__device__ __forceinline__ bool rounds_up(float h, float g, float rz, float lo, float hi, float m, float low,
                                          uint32_t& code) {
  const float x = __fmul_rn(h, rz), z = __fmul_rn(x, g), za = fabsf(z);
  const uint32_t both = pack_e4m3x4(f2_make(__fmul_rn(z, lo), __fmul_rn(z, hi)), 0);
  code = both >> 8 & 255u;
  // Nearly equal products, in two floats each: every difference and sum below is exact.
  const float zl = copysignf(1.f, z) * __fmaf_rn(x, g, -z);
  const float mid = e4m3_magnitude(both & 127u) + e4m3_magnitude(code & 127u);  // twice the midpoint
  const float ah = __fmul_rn(896.f, za), al = __fmaf_rn(896.f, za, -ah);
  const float bh = __fmul_rn(mid, m), bl = __fmaf_rn(mid, m, -bh);
  const float d = (ah - bh) + ((al - bl) + (896.f * zl - mid * low));
  // m times the fp32 step above the midpoint; below it half of that, if it is a power of two.
  const uint32_t bits = __float_as_uint(mid);
  float step = __fmul_rn(m, __uint_as_float(bits & 0x7F800000u) * 0x1p-24f);
  if (d < 0.f && (bits & 0x007FFFFFu) == 0u) step *= 0.5f;
  return fabsf(d) <= step ? both & 1u : d > 0.f;
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

// To 8 bits the blocks an SM holds are kept at four (two of 16 warps) against the rare path's registers: 24.8
// us for 9524 x 2048, 27.6 without.
template <int V, int G, RowOp kOp>
__global__ void __launch_bounds__(32 * block_warps(G), kOp != RowOp::kNormE4m3 ? 0 : G > 8 ? 2 : 4)
    token_rows_kernel(const NormArgs a) {
  __shared__ float red[2][kMaxWarps];
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
  if (kOp != RowOp::kQuant && a.res) {
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
  float r = 1.f;
  if constexpr (kOp != RowOp::kQuant) {
    uint64_t s2 = 0;  // (0, 0)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const F8 u = unpack8(w[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = f2_fma(u.p[j], u.p[j], s2);
    }
    float s0, s1;
    f2_split(s2, s0, s1);
    const float ss = row_reduce<G, false>(s0 + s1, red[0]);
    r = __frsqrt_rn(fmaf(ss, a.inv_c, a.eps));
    if (lane == 0 && a.r) a.r[row] = r;
  }
  // 8 bits: r cancels in 448 z / m, so that z and m need it only to its power of two, whose product with h
  // is exact; s gets the rest of it, rho in [1, 2).
  const float pow2 = __uint_as_float(__float_as_uint(r) & 0x7F800000u);
  const float rho = kOp == RowOp::kNormE4m3 ? __uint_as_float((__float_as_uint(r) & 0x007FFFFFu) | 0x3F800000u) : 1.f;
  const float rz = kOp == RowOp::kNormE4m3 ? pow2 : r;
  const uint64_t r2 = f2_make(rz, rz);
  auto z_of = [&](int i, int c) {  // (h r) g
    F8 z = unpack8(w[i]);
    if constexpr (kOp != RowOp::kQuant) {
      const F8 g = load8f(a.g, c);
#pragma unroll
      for (int j = 0; j < 4; ++j) z.p[j] = f2_mul(f2_mul(z.p[j], r2), g.p[j]);
    }
    return z;
  };
  if constexpr (kOp == RowOp::kNorm) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      if (c < a.chunks) a.y[base + c] = pack8(z_of(i, c));
    }
  } else {
    F8 z[V];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      if (c < a.chunks) {
        z[i] = z_of(i, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u, v;
          f2_split(z[i].p[j], u, v);
          m = fmax3(m, fabsf(u), fabsf(v));
        }
      }
    }
    m = row_reduce<G, true>(m, red[1]);
    const float mz = __fmul_rn(m, rho);
    if (lane == 0) a.s[row] = __fdiv_rn(fmaxf(mz, kAmaxFloor), kE4m3Max);
    if constexpr (kOp == RowOp::kNormE4m3) {
      // z, m, 448 / m, the end of the range and the product round once each, 5 * 2^-24 in all, and a tie reaches
      // 2^-24 far: rounded from both ends of a range (7 * 2^-24 below, 8 above), which nearly always agree.  (A corrected quotient, rounded as it is, took 26.3 us
      // for 9524 x 2048 and gave the other neighbour for one value in a million.)
      const bool low = mz < kAmaxFloor;
      const float most = low ? __fdiv_rn(kAmaxFloor, rho) : m;
      const float by = __fdiv_rn(kE4m3Max, most);
      const float lo = __fmul_rn(by, 1.f - 7 * 0x1p-24f), hi = __fmul_rn(by, 1.f + 8 * 0x1p-24f);
      const uint64_t lo2 = f2_make(lo, lo), hi2 = f2_make(hi, hi);
      unsigned open = 0;  // undecided values: bit 8 b + 2 i + w for byte b of word w of chunk i
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * kLanes + lane;
        if (c < a.chunks) {
          const F8& v = z[i];
          const uint32_t y0 = pack_e4m3x4(f2_mul(v.p[0], lo2), f2_mul(v.p[1], lo2));
          const uint32_t y1 = pack_e4m3x4(f2_mul(v.p[2], lo2), f2_mul(v.p[3], lo2));
          const uint32_t u0 = pack_e4m3x4(f2_mul(v.p[0], hi2), f2_mul(v.p[1], hi2));
          const uint32_t u1 = pack_e4m3x4(f2_mul(v.p[2], hi2), f2_mul(v.p[3], hi2));
          // (Neighbouring codes differ in their last bit.)
          open |= (((y0 ^ u0) & 0x01010101u) | ((y1 ^ u1) & 0x01010101u) << 1) << (2 * i);
          a.y8[base + c] = make_uint2(y0, y1);
        }
      }
      if (__any_sync(0xffffffffu, open != 0)) {
        // The row of h: complete, since its warps have met in row_reduce after their stores.
        const uint4* h = (a.res ? a.h : a.x) + base;
        const float m_low = low ? 0.f : max_low(h, a.g, a.chunks, rz, m);
        for (; open; open &= open - 1) {
          const int bit = __ffs(open) - 1, c = (bit >> 1 & 3) * kLanes + lane, e = 4 * (bit & 1) + (bit >> 3);
          const uint32_t word = reinterpret_cast<const uint16_t*>(h + c)[e];
          uint32_t code;
          if (rounds_up(__uint_as_float(word << 16), __ldg(a.g + c * 8 + e), rz, lo, hi, most, m_low, code))
            reinterpret_cast<uint8_t*>(a.y8 + base + c)[e] = static_cast<uint8_t>(code);
        }
      }
    } else {
      // 448 x / m as 0.875 x over m / 512, which stays in range for every x and is exact: midpoints of e4m3
      // (common here) stay midpoints.  The product with the reciprocal and one residual correction (Markstein,
      // 1990) rounds as the quotient does.
      m = __fmul_rn(fmaxf(m, kAmaxFloor), 1.f / 512);
      const float inv = __frcp_rn(m);
      const uint64_t inv2 = f2_make(inv, inv), neg_m2 = f2_make(-m, -m);
      const uint64_t k2 = f2_make(kE4m3Max / 512, kE4m3Max / 512);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * kLanes + lane;
        if (c < a.chunks) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t v = f2_mul(z[i].p[j], k2), q = f2_mul(v, inv2);
            z[i].p[j] = f2_fma(f2_fma(q, neg_m2, v), inv2, q);
          }
          a.y8[base + c] = make_uint2(pack_e4m3x4(z[i].p[0], z[i].p[1]), pack_e4m3x4(z[i].p[2], z[i].p[3]));
        }
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
// the rows it meets, then the block's rows are added in order.  n and u stay in
// registers between the two uses, 12 instructions a value instead of 20.  (The
// next rows' operands by bulk copies through shared memory, two rows ahead: 22.2
// us for 17616 x 768 instead of 20.3; to registers, one row ahead: slower still.)
template <int V, int G>
__global__ void __launch_bounds__(32 * block_warps(G), G > 8 ? 1 : 2) token_norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kLanes = 32 * G, kRows = block_warps(G) / G;
  extern __shared__ __align__(16) float sums[];  // [rows of a block][C]
  __shared__ float red[2][kMaxWarps];
  const int lane = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  uint64_t acc[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  int it = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + slot; row < a.T; row += step, ++it) {
    const uint4 *dy = a.dy + row * a.chunks, *h = a.h + row * a.chunks;
    const uint4* dh = a.dh ? a.dh + row * a.chunks : nullptr;
    const float r = a.r[row];
    uint4 wy[V], wh[V], wd[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      const bool in = c < a.chunks;
      wy[i] = in ? dy[c] : make_uint4(0u, 0u, 0u, 0u);
      wh[i] = in ? h[c] : make_uint4(0u, 0u, 0u, 0u);
      wd[i] = in && dh ? dh[c] : make_uint4(0u, 0u, 0u, 0u);
    }
    const int64_t base = row * a.chunks;
    const uint64_t r2 = f2_make(r, r);
    F8 n[V], u[V];  // h r and g dy
    uint64_t un2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      const bool in = c < a.chunks;
      const F8 y = unpack8(wy[i]), g = load8f(a.g, in ? c : 0);
      n[i] = unpack8(wh[i]);
      u[i] = y;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[i].p[j] = f2_mul(n[i].p[j], r2);
        u[i].p[j] = f2_mul(y.p[j], g.p[j]);
        acc[i][j] = f2_fma(y.p[j], n[i].p[j], acc[i][j]);
        un2 = f2_fma(u[i].p[j], n[i].p[j], un2);
      }
    }
    float u0, u1;
    f2_split(un2, u0, u1);
    const float m = -row_reduce<G, false>(u0 + u1, red[it & 1]) * a.inv_c;
    const uint64_t m2 = f2_make(m, m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * kLanes + lane;
      F8 d = unpack8(wd[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d.p[j] = f2_fma(r2, f2_fma(n[i].p[j], m2, u[i].p[j]), d.p[j]);
      if (c < a.chunks) a.dx[base + c] = pack8(d);
    }
  }
  const int C = a.chunks * 8;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * C;
  ulonglong2* mine = reinterpret_cast<ulonglong2*>(kRows > 1 ? sums + static_cast<size_t>(slot) * C : out);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = i * kLanes + lane;
    if (c < a.chunks) {
      mine[2 * c] = make_ulonglong2(acc[i][0], acc[i][1]);
      mine[2 * c + 1] = make_ulonglong2(acc[i][2], acc[i][3]);
    }
  }
  if constexpr (kRows > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += 32 * block_warps(G)) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) s += sums[i * C + c];
      out[c] = s;
    }
  }
}

// dg = the sum of the blocks' partial sums, in a fixed order: 8 columns (a
// 32-byte sector of each partial) a block, 32 threads a column.
__global__ void __launch_bounds__(256) dg_sum_kernel(const float* part, int parts, int C, float* dg) {
  __shared__ float sums[32][9];
  griddep_launch_dependents();
  griddep_wait();
  const int col = threadIdx.x % 8, grp = threadIdx.x / 8;
  const float* from = part + blockIdx.x * 8 + col;  // C is a multiple of 8
  float v[(kBwdParts + 31) / 32];  // all on their way at once
#pragma unroll
  for (int i = 0; i < (kBwdParts + 31) / 32; ++i) {
    const int p = grp + 32 * i;
    v[i] = p < parts ? from[static_cast<size_t>(p) * C] : 0.f;
  }
  float s = v[0];
#pragma unroll
  for (int i = 1; i < (kBwdParts + 31) / 32; ++i) s += v[i];
  sums[grp][col] = s;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sums[i][col];
    dg[blockIdx.x * 8 + col] = s;
  }
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

template <RowOp kOp>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t st) {
  return with_layout(a.chunks, [&](auto l) {
    using L = decltype(l);
    constexpr int kWarps = block_warps(L::G), kRows = kWarps / L::G;
    return launch_pdl(token_rows_kernel<L::V, L::G, kOp>, dim3(static_cast<unsigned>((a.T + kRows - 1) / kRows)),
                      dim3(32 * kWarps), 0, st, a);
  });
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
  int rows = 1;
  with_layout(C / 8, [&](auto l) {
    rows = block_warps(decltype(l)::G) / decltype(l)::G;
    return cudaSuccess;
  });
  const int64_t blocks = (static_cast<int64_t>(T) + rows - 1) / rows;
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
  return with_layout(a.chunks, [&](auto l) {
    using L = decltype(l);
    constexpr int kWarps = block_warps(L::G), kRows = kWarps / L::G;
    const size_t smem = kRows > 1 ? static_cast<size_t>(kRows) * C * sizeof(float) : 0;  // at most 32 KB
    return launch_pdl(token_norm_bwd_kernel<L::V, L::G>, dim3(static_cast<unsigned>(parts)), dim3(32 * kWarps), smem,
                      st, a);
  });
}

cudaError_t launch_dg_sum(const float* part, int parts, int C, float* dg, cudaStream_t st) {
  return launch_pdl(dg_sum_kernel, dim3(static_cast<unsigned>(C / 8)), dim3(256), 0, st, part, parts, C, dg);
}

}  // namespace jattn
