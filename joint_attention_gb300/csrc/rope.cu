// rope.cu — rotary positions on several axes (height and width of an image, time of
// a video), with or without the QK-RMSNorm before them, and their backward.
//
// Per row of q (and of k) with d channels and position pos[a] on axis a:
//     z = g x r,  r = (mean_c x_c^2 + eps)^(-1/2)     (without gains: z = x)
//     pair p of the P rotary pairs, on its axis a with angle t = pos[a] freq[p]:
//     (z_i, z_j) -> (z_i cos t - z_j sin t, z_i sin t + z_j cos t)
//     (i, j) = (2 p, 2 p + 1) interleaved, else (p, p + P); channels from 2 P on stay
// and one bf16 rounding.  Backward: the rotation by -t (its transpose), then, with n =
// x r and u = g times that, dx = r (u - n mean_c(u n)) and dg = the sum of (rotated
// gradient) n over all rows and heads.
//
// Angles: pos freq / (2 pi) in turns as the sum of two floats (the product and its
// exact remainder, with 1 / (2 pi) and freq / (2 pi) in two floats as well), whole
// turns taken off exactly, then sincospif of what is left: off by some 2^-24 of a turn
// for angles up to millions, where an fp32 angle would be off by 2^-24 of itself.
//
// Bound by HBM: every value is read and written once.  A thread keeps the cosines and
// sines of one token's 8 pairs and takes 16 channels of that token in a run of heads
// (and batch items, where they share positions), so that sincospif, some 350
// instructions for 8 pairs, is paid once a run.  d / 16 threads a row; a warp covers 4
// or 8 neighbouring tokens of a head, contiguous in memory.
#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"
#include "token_rows.cuh"

namespace jattn {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;       // rows of a thread whose loads are in flight together
constexpr int kMaxRun = 16;     // heads a thread takes at most
constexpr int kBlocks = 152 * 8;     // blocks aimed at
constexpr int kBlocksBwd = 152 * 4;  // with gains' gradients: a partial sum each

struct RopeArgs {
  const uint4* src[2];   // q, k (backward: their rotated gradients)
  const uint4* x[2];     // backward with gains: q, k
  uint4* dst[2];
  const float* gain[2];  // or null
  const float* pos;      // [N, axes], or [B, N, axes]
  const float* freq;     // [P]
  int heads[2];          // heads that share a token's positions: of its batch item, or of all items
  int chunks[2];         // runs of them
  int run;               // heads of a run
  int N, tiles;          // tokens, blocks over them
  int axes, P;
  int pair_end[kMaxAxes];  // pairs before the end of each axis
  bool interleaved;
  float sign;  // of the angles
  float eps;
  float* part;  // backward with gains: [blocks of q, then of k][d]
};

// cos and sin of 2 pi (pos freq / (2 pi)).
__device__ __forceinline__ void rotation(float pos, float freq, float& c, float& s) {
  constexpr float kInv = 0x1.45f306p-3f, kInvLow = 0x1.b9391p-28f;  // 1 / (2 pi)
  const float fh = __fmul_rn(freq, kInv), fl = __fmaf_rn(freq, kInvLow, __fmaf_rn(freq, kInv, -fh));
  const float th = __fmul_rn(pos, fh), tl = __fmaf_rn(pos, fl, __fmaf_rn(pos, fh, -th));
  sincospif(2.f * ((th - rintf(th)) + tl), &s, &c);
}

// Where a block and a thread are, and the thread's cosines and sines.
template <int D>
struct RopeThread {
  static constexpr int kLanes = D / 16, kTokens = kThreads / kLanes;
  int t, item, first, count, token;  // tensor (0: q, 1: k); heads first .. first + count - 1 of the item's
  int chunk[2];                      // the thread's 16-byte chunks of a row
  bool live, rot[2];
  int64_t row0;  // the first head's row
  float c[8], s[8];

  __device__ __forceinline__ explicit RopeThread(const RopeArgs& a) {
    const int per_item = a.chunks[0] + a.chunks[1];
    const int tile = blockIdx.x % a.tiles, job = blockIdx.x / a.tiles;
    item = job / per_item;
    int run = job - item * per_item;
    t = run >= a.chunks[0];
    if (t) run -= a.chunks[0];
    first = run * a.run;
    const int heads = t ? a.heads[1] : a.heads[0];
    count = min(a.run, heads - first);
    token = tile * kTokens + threadIdx.x / kLanes;
    live = token < a.N;
    row0 = (static_cast<int64_t>(item) * heads + first) * a.N + token;
    const int l = threadIdx.x % kLanes;
    if (a.interleaved) {
      chunk[0] = l;
      chunk[1] = l + kLanes;
      rot[0] = chunk[0] < a.P / 4;
      rot[1] = chunk[1] < a.P / 4;
    } else {
      const int lanes = a.P / 8;  // lanes with pairs
      rot[0] = rot[1] = l < lanes;
      chunk[0] = l < lanes ? l : 2 * l;
      chunk[1] = l < lanes ? l + lanes : 2 * l + 1;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = 1.f;
      s[k] = 0.f;
    }
    if (!live) return;
    const float* pos = a.pos + (static_cast<int64_t>(item) * a.N + token) * a.axes;
    float at[kMaxAxes];
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) at[i] = i < a.axes ? __ldg(pos + i) : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!rot[k / 4]) continue;
      const int p = a.interleaved ? 4 * chunk[k / 4] + k % 4 : 8 * l + k;
      float w = at[0];
#pragma unroll
      for (int i = 1; i < kMaxAxes; ++i)
        if (p >= a.pair_end[i - 1]) w = at[i];
      rotation(w, a.sign * __ldg(a.freq + p), c[k], s[k]);
    }
  }
  // The 16 channels, chunk 0 first, rotated.
  __device__ __forceinline__ void rotate(const RopeArgs& a, float (&v)[16]) const {
    auto turn = [&](int i, int j, int k) {
      const float x = v[i], y = v[j];
      v[i] = fmaf(x, c[k], -(y * s[k]));
      v[j] = fmaf(x, s[k], y * c[k]);
    };
    if (a.interleaved) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (rot[h])
#pragma unroll
          for (int k = 0; k < 4; ++k) turn(8 * h + 2 * k, 8 * h + 2 * k + 1, 4 * h + k);
    } else if (rot[0]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) turn(k, 8 + k, k);
    }
  }
};

__device__ __forceinline__ void unpack16(const uint4& lo, const uint4& hi, float (&v)[16]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack_half(const float (&v)[16], int h) {
  return make_uint4(pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                    pack_bf16x2(v[8 * h + 4], v[8 * h + 5]), pack_bf16x2(v[8 * h + 6], v[8 * h + 7]));
}
template <int D>
__device__ __forceinline__ void load_gain(const RopeThread<D>& th, const float* gain, float (&g)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) g[8 * h + i] = __ldg(gain + 8 * th.chunk[h] + i);
}

template <int D, bool kNorm>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const RopeThread<D> th(a);
  const uint4* src = th.t ? a.src[1] : a.src[0];
  uint4* dst = th.t ? a.dst[1] : a.dst[0];
  float g[16];
  if constexpr (kNorm) load_gain(th, th.t ? a.gain[1] : a.gain[0], g);
  constexpr int kRow = D / 8;  // chunks of a row
  const int64_t step = static_cast<int64_t>(a.N) * kRow;
  int64_t at = th.row0 * kRow;
  for (int h0 = 0; h0 < th.count; h0 += kAhead, at += kAhead * step) {
    uint4 w[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[i][h] = th.live && h0 + i < th.count ? src[at + i * step + th.chunk[h]] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h0 + i >= th.count) break;  // the same in the whole block
      float v[16];
      unpack16(w[i][0], w[i][1], v);
      if constexpr (kNorm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
        for (int o = RopeThread<D>::kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = __frsqrt_rn(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = v[e] * r * g[e];
      }
      th.rotate(a, v);
      if (th.live) {
        dst[at + i * step + th.chunk[0]] = pack_half(v, 0);
        dst[at + i * step + th.chunk[1]] = pack_half(v, 1);
      }
    }
  }
}

// With gains: the rotation by -t, the backward of the RMSNorm and the block's part of
// the gain's gradient (each thread its 16 channels over its heads, then the tokens of
// the block in a fixed order).
template <int D>
__global__ void __launch_bounds__(kThreads) rope_norm_bwd_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float sums[kThreads / 32][D];
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kLanes = RopeThread<D>::kLanes;
  const RopeThread<D> th(a);
  const uint4* src = th.t ? a.src[1] : a.src[0];
  const uint4* x = th.t ? a.x[1] : a.x[0];
  uint4* dst = th.t ? a.dst[1] : a.dst[0];
  float g[16], dg[16];
  load_gain(th, th.t ? a.gain[1] : a.gain[0], g);
#pragma unroll
  for (int e = 0; e < 16; ++e) dg[e] = 0.f;
  constexpr int kRow = D / 8, kDeep = 2;
  const int64_t step = static_cast<int64_t>(a.N) * kRow;
  int64_t at = th.row0 * kRow;
  for (int h0 = 0; h0 < th.count; h0 += kDeep, at += kDeep * step) {
    uint4 w[kDeep][2], wx[kDeep][2];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = th.live && h0 + i < th.count;
        w[i][h] = in ? src[at + i * step + th.chunk[h]] : make_uint4(0u, 0u, 0u, 0u);
        wx[i][h] = in ? x[at + i * step + th.chunk[h]] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      if (h0 + i >= th.count) break;  // the same in the whole block
      float v[16], n[16];
      unpack16(w[i][0], w[i][1], v);
      unpack16(wx[i][0], wx[i][1], n);
      th.rotate(a, v);
      float ss = 0.f, ux = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        ss = fmaf(n[e], n[e], ss);
        ux = fmaf(v[e] * g[e], n[e], ux);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        ux += __shfl_xor_sync(0xffffffffu, ux, o);
      }
      const float r = __frsqrt_rn(fmaf(ss, 1.f / D, a.eps));
      const float m = -(ux * r) * (1.f / D);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float nr = n[e] * r;
        dg[e] = fmaf(v[e], nr, dg[e]);
        v[e] = r * fmaf(nr, m, v[e] * g[e]);
      }
      if (th.live) {
        dst[at + i * step + th.chunk[0]] = pack_half(v, 0);
        dst[at + i * step + th.chunk[1]] = pack_half(v, 1);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], o);
  }
  if (threadIdx.x % 32 < kLanes) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[threadIdx.x / 32][8 * th.chunk[h] + i] = dg[8 * h + i];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += sums[i][threadIdx.x];
    // Blocks of q first: an item's runs of q, each over the tiles.
    const int tile = blockIdx.x % a.tiles, job = blockIdx.x / a.tiles;
    const int run = job - th.item * (a.chunks[0] + a.chunks[1]) - (th.t ? a.chunks[0] : 0);
    const int items = gridDim.x / (a.tiles * (a.chunks[0] + a.chunks[1]));
    const int before = th.t ? items * a.chunks[0] : 0;
    const int64_t at_part = static_cast<int64_t>(before + th.item * a.chunks[th.t] + run) * a.tiles + tile;
    a.part[at_part * D + threadIdx.x] = s;
  }
}

// dgq (blockIdx.y = 0) and dgk from the blocks' parts, 8 columns a block.
__global__ void __launch_bounds__(256) rope_gain_kernel(const float* part, int parts_q, int parts_k, int d, float* dgq,
                                                        float* dgk) {
  griddep_launch_dependents();
  griddep_wait();
  const bool k = blockIdx.y != 0;
  const int at = blockIdx.x * 8;
  const float s = column_sum(part + (k ? static_cast<size_t>(parts_q) * d : 0) + at, k ? parts_k : parts_q,
                             static_cast<size_t>(d));
  if (threadIdx.x < 8) (k ? dgk : dgq)[at + threadIdx.x] = s;
}

// How a call is split; all of it a function of the sizes alone.
struct Split {
  int items, heads[2], run, chunks[2], tiles;
  int64_t blocks() const { return static_cast<int64_t>(items) * tiles * (chunks[0] + chunks[1]); }
};
Split split_of(const Rope& t, int aim) {
  Split s;
  const int tokens = kThreads / (t.d / 16);
  s.items = t.per_item ? t.B : 1;
  s.heads[0] = t.per_item ? t.Hq : t.B * t.Hq;
  s.heads[1] = t.per_item ? t.Hk : t.B * t.Hk;
  s.tiles = static_cast<int>((static_cast<int64_t>(t.N) + tokens - 1) / tokens);
  const int64_t each = static_cast<int64_t>(s.items) * s.tiles * (static_cast<int64_t>(s.heads[0]) + s.heads[1]);
  const int64_t run = each / aim;
  // Beyond 2^31 blocks of the longest run aimed at, runs grow instead.
  const int64_t least = each / (int64_t{1} << 30) + 1;
  s.run = static_cast<int>(run < 1 ? 1 : run > kMaxRun ? kMaxRun : run);
  if (s.run < least) s.run = static_cast<int>(least);
  for (int i = 0; i < 2; ++i) s.chunks[i] = (s.heads[i] + s.run - 1) / s.run;
  return s;
}

RopeArgs args_of(const Rope& t, const Split& s, float sign) {
  RopeArgs a = {};
  for (int i = 0; i < 2; ++i) {
    a.heads[i] = s.heads[i];
    a.chunks[i] = s.chunks[i];
  }
  a.run = s.run;
  a.N = t.N;
  a.tiles = s.tiles;
  a.axes = t.axes;
  int end = 0;
  for (int i = 0; i < kMaxAxes; ++i) {
    end += i < t.axes ? t.pairs[i] : 0;
    a.pair_end[i] = i + 1 < t.axes ? end : t.d;  // the last axis' pairs have no axis behind them
  }
  a.P = end;
  a.pos = t.pos;
  a.freq = t.freq;
  a.interleaved = t.interleaved;
  a.sign = sign;
  a.eps = t.eps;
  return a;
}

}  // namespace

cudaError_t launch_rope(const Rope& t, const uint16_t* q, const uint16_t* k, uint16_t* q_out, uint16_t* k_out,
                        bool backward, cudaStream_t st) {
  const Split s = split_of(t, kBlocks);
  RopeArgs a = args_of(t, s, backward ? -1.f : 1.f);
  a.src[0] = reinterpret_cast<const uint4*>(q);
  a.src[1] = reinterpret_cast<const uint4*>(k);
  a.dst[0] = reinterpret_cast<uint4*>(q_out);
  a.dst[1] = reinterpret_cast<uint4*>(k_out);
  const bool norm = !backward && t.gq;
  if (norm) {
    a.gain[0] = t.gq;
    a.gain[1] = t.gk;
  }
  auto kernel = t.d == 64 ? (norm ? rope_kernel<64, true> : rope_kernel<64, false>)
                          : (norm ? rope_kernel<128, true> : rope_kernel<128, false>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(s.blocks())), dim3(kThreads), 0, st, a);
}

int64_t rope_bwd_parts(const Rope& t, int64_t* of_q) {
  const Split s = split_of(t, kBlocksBwd);
  *of_q = static_cast<int64_t>(s.items) * s.tiles * s.chunks[0];
  return s.blocks();
}

cudaError_t launch_rope_norm_bwd(const Rope& t, const uint16_t* dq_rot, const uint16_t* dk_rot, const uint16_t* q,
                                 const uint16_t* k, uint16_t* dq, uint16_t* dk, float* part, cudaStream_t st) {
  const Split s = split_of(t, kBlocksBwd);
  RopeArgs a = args_of(t, s, -1.f);
  a.src[0] = reinterpret_cast<const uint4*>(dq_rot);
  a.src[1] = reinterpret_cast<const uint4*>(dk_rot);
  a.x[0] = reinterpret_cast<const uint4*>(q);
  a.x[1] = reinterpret_cast<const uint4*>(k);
  a.dst[0] = reinterpret_cast<uint4*>(dq);
  a.dst[1] = reinterpret_cast<uint4*>(dk);
  a.gain[0] = t.gq;
  a.gain[1] = t.gk;
  a.part = part;
  return launch_pdl(t.d == 64 ? rope_norm_bwd_kernel<64> : rope_norm_bwd_kernel<128>,
                    dim3(static_cast<unsigned>(s.blocks())), dim3(kThreads), 0, st, a);
}

cudaError_t launch_rope_gains(const Rope& t, const float* part, float* dgq, float* dgk, cudaStream_t st) {
  int64_t of_q;
  const int64_t parts = rope_bwd_parts(t, &of_q);
  return launch_pdl(rope_gain_kernel, dim3(static_cast<unsigned>(t.d / 8), 2), dim3(256), 0, st, part,
                    static_cast<int>(of_q), static_cast<int>(parts - of_q), t.d, dgq, dgk);
}

}  // namespace jattn
