// qkv_proj.cu — the QKV projections of the two token streams with QK-RMSNorm
// in their epilogue, on tcgen05 tensor cores.
//
// The MM-DiT block projects each stream's tokens to Q, K and V with that
// stream's own weights, concatenates the caption and image streams along the
// token axis, normalises Q and K (RMSNorm over the head dim, one learned gain
// vector each) and runs one attention over the joint sequence (re-diffusion
// README, "architecture flowchart"; "design notes" table, row "QK norm").
// One launch covers both streams:
//
//   Y = bf16(X W^T + bias)      X: [B * N_s, C] tokens, W: [3 H d, C] (q heads, k heads, v heads)
//   q, k, v = Y by heads, into the joint [B, H, N, d] layout at the stream's
//             rows row0 .. row0 + N_s - 1 of every batch item
//   q_hat = bf16(gq * q * r(q)), k_hat likewise, r(x) = (mean x^2 + eps)^(-1/2)
//
// with q_hat / k_hat correctly rounded as in the norm kernels (the bf16 value
// nearest the exact real product), and r(q), r(k) kept: exactly what the
// training forward keeps for the backward, so the attention forward starts
// from q_hat / k_hat with no normalisation pass of its own.
//
// Tiles: 128 token rows x 256 output columns per accumulator, K in steps of
// 64; persistent, one CTA per SM, the image stream's tiles then the caption
// stream's.
//   warp 8      TMA producer: the X tile (128 x 64) and the W tile (256 x 64)
//               of each K step, 128-byte swizzle, through a 3-stage ring.
//   warp 9      MMA issuer: 4 MMAs (M 128, N 256, K 16) per K step into one of
//               two TMEM accumulators (256 columns each), so that a tile's
//               epilogue overlaps the next tile's products.
//   warps 0-7   epilogue, one thread per token row (TMEM lane): warps w and
//               w + 4 share the lanes of warp w % 4 and take columns 0-127 and
//               128-255 of the tile (two heads of d = 64, or one of d = 128).
//               Per head: d fp32 values out of TMEM, + bias (the warp's
//               slice, copied to shared memory while the products run),
//               rounded to bf16 (the projection's output) for q / k / v; for
//               q and k the row's RMSNorm from those bf16 values, q_hat /
//               k_hat and r.  Rows are staged in shared memory and written
//               out as whole 128-byte lines, four rows per store instruction.
// Heads past 3 H in the last column tile, and token rows past the stream's
// end in its last row tile, read the TMA's zero fill and are not stored.
//
// The same kernel takes two other forms of the products (template kMode):
//   kE4m3  X and W in e4m3 with fp32 scales of their rows: a K step of 128
//          values in the same 128-byte rows, kind::f8f6f4 products, and
//          Y = bf16(sx sw acc + bias).
//   kLora  low-rank adapters of the batch items' own beside the shared
//          weights: Y = bf16(X W^T + U B^T + bias), U = scale X A^T (one
//          launch of lora_down_kernel before, rounded to bf16), as further K
//          steps of 16 into the same accumulator.  A row tile that holds items
//          with different adapters takes each run of items in turn, with the
//          other rows' lanes disabled in the MMA, so that no row mask or copy of
//          U is needed; a column tile over a q / k / v boundary takes each part
//          with its own columns of U.  Four such (U, B) pairs of 4 + 8 KB fill
//          one ring stage.
//
// Correct rounding: the per-thread sum of the d squares is a balanced tree
// (at most 7 roundings per term, within the 8 that the rounding window of the
// norm kernels allows for), and elements in the bf16-midpoint window are
// re-rounded from a double-float r.
#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"
#include "bf16_round.cuh"

namespace jattn {
namespace {

constexpr int kQkvStages = 3;
constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kATile = kBM * kBK * 2;  // 16 KB
constexpr int kBTile = kBN * kBK * 2;  // 32 KB
constexpr int kStageBytes = kATile + kBTile;
constexpr int kStageRowBytes = 128;                 // 64 bf16 columns of one token row
constexpr int kStagingBytes = 32 * kStageRowBytes;  // per epilogue warp: its 32 rows of 64 columns
constexpr uint32_t kDeadRow = 0xFFFFFFFFu;

// Eight epilogue warps (warps w and w + 4 take the TMEM lanes of warp w % 4
// and columns 0-127 / 128-255 of the tile: two heads of d = 64, or one of
// d = 128), then the TMA producer and the MMA issuer.  Each epilogue warp
// stages its rows in shared memory, in two buffers: at d = 64 raw rows and
// q_hat / k_hat rows, at d = 128 the two 64-column halves, raw, then q_hat /
// k_hat.
template <int D>
struct QkvCfg {
  static constexpr int kEpiWarps = 8;
  static constexpr int kEpiThreads = 32 * kEpiWarps;
  static constexpr int kWarpProd = kEpiWarps, kWarpIssue = kEpiWarps + 1;
  static constexpr int kThreads = 32 * (kEpiWarps + 2);
  static constexpr int kStaging = 2 * kStagingBytes;
  static constexpr int kBiasBytes = 128 * 4;  // per epilogue warp: the bias of its 128 columns
  static constexpr int kOffStaging = kQkvStages * kStageBytes;
  static constexpr int kOffBias = kOffStaging + kEpiWarps * kStaging;
  static constexpr int kSpareBytes = D == 128 ? 256 : 0;  // per epilogue warp: fix_staged_halves' row
  static constexpr int kOffSpare = kOffBias + kEpiWarps * kBiasBytes;
  static constexpr int kOffScale = kOffSpare + kEpiWarps * kSpareBytes;  // kE4m3: their weight scales, likewise
  static constexpr int kDynSmem = kOffScale + 1024;
  static constexpr int kDynSmemE4m3 = kOffScale + kEpiWarps * kBiasBytes + 1024;
};

struct QkvBars {
  uint64_t full[kQkvStages], empty[kQkvStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  __align__(16) float gq[128];
  __align__(16) float gk[128];
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}
__device__ __forceinline__ uint64_t desc_add(uint64_t desc, uint32_t byte_off) { return desc + (byte_off >> 4); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  const uint4 v = ld_shared_v4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// Staging of a warp's 32 token rows of 64 bf16 columns (128 bytes each) in
// shared memory: row i at i * 128, its 16-byte chunk c at slot c ^ (i % 8),
// so that a row written by one lane and a chunk column read across 8 lanes
// both touch every bank once.
__device__ __forceinline__ uint32_t staged(uint32_t buf, int row, int chunk) {
  return buf + row * kStageRowBytes + ((chunk ^ (row & 7)) << 4);
}
// This lane's row: w[0..31] (packed pairs).
__device__ __forceinline__ void stage_row(uint32_t buf, const uint32_t* w, int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c) st_shared_v4(staged(buf, lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
// Writes the 32 staged rows out, four whole rows (four 128-byte lines) per
// store instruction: lanes 8 j' .. 8 j' + 7 take row 4 j + j', one chunk
// each.  rows[j]: the global row index (b H + h) N + n of staged row
// 4 j + lane / 8 for head 0 (kDeadRow: past the stream's end); head_rows =
// h N; col: the first column (0, or 64 within a d = 128 head row).
template <int D>
__device__ __forceinline__ void store_rows(uint32_t buf, uint16_t* base, const uint32_t (&rows)[8],
                                           uint32_t head_rows, int col, int lane) {
  const int ch = lane & 7;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 val = ld_shared_v4(staged(buf, 4 * j + (lane >> 3), ch));
    if (rows[j] != kDeadRow)
      *reinterpret_cast<uint4*>(base + (static_cast<size_t>(rows[j]) + head_rows) * D + col + ch * 8) = val;
  }
}

// The double-float sum of squares of a row spread over the warp, the same
// on every lane: each lane's own error-free sum (s, c), then a butterfly of
// error-free additions (symmetric, so every lane forms the same values).
__device__ __forceinline__ void warp_sum_df(float& s, float& c) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, off), c2 = __shfl_xor_sync(0xffffffffu, c, off);
    float t, e;
    two_sum(s, s2, t, e);
    s = t;
    c = __fadd_rn(__fadd_rn(c, c2), e);
  }
  fast_two_sum(s, c, s, c);
}
__device__ __forceinline__ void add_sq_df(uint32_t w, float& s, float& c) {
  float t, e;
  two_sum(s, __fmul_rn(bf_lo(w), bf_lo(w)), t, e);
  c = __fadd_rn(c, e);
  two_sum(t, __fmul_rn(bf_hi(w), bf_hi(w)), s, e);
  c = __fadd_rn(c, e);
}

// The rare path.  The warp takes each of its rows that has an element near
// a bf16 midpoint (owner: the lane holding the row) together: each lane
// takes D / 32 of the row's values, their squares (exact) are summed by
// error-free additions over the warp, and each lane re-rounds its elements
// that the owner's fp32 path put near a midpoint, from the double-float r.
//
// d = 64 (fix_staged_rows): the row's raw values come from the raw staging
// buffer and each lane writes its word of the row (two elements, re-rounded
// where needed) over the staged q_hat / k_hat row, before that is written
// out.
__device__ __forceinline__ void fix_staged_rows(unsigned todo, uint32_t raw, uint32_t hat, float r, const float* g,
                                                int lane) {
  while (todo) {
    const int o = __ffs(todo) - 1;
    todo &= todo - 1;
    // Word `lane` of row o: elements 2 lane, 2 lane + 1 (chunk lane / 4).
    const uint32_t off = (lane & 3) * 4;
    const uint32_t w = ld_shared_u32(staged(raw, o, lane >> 2) + off);
    const float ro = __shfl_sync(0xffffffffu, r, o);
    float s = 0.f, c = 0.f;
    add_sq_df(w, s, c);
    warp_sum_df(s, c);
    float rh, rl;
    rsqrt_mean_eps_df(s, c, 1.f / 64, rh, rl);
    float f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * lane + j;
      const float x = j ? bf_hi(w) : bf_lo(w);
      const float z = __fmul_rn(__fmul_rn(g[e], x), ro);
      f[j] = near_bf16_midpoint(z) ? round_bf16_df(g[e], x, rh, rl) : z;
    }
    st_shared_u32(staged(hat, o, lane >> 2) + off, pack_bf16x2(f[0], f[1]));
  }
}
// d = 128 (fix_staged_halves): the row's raw values no longer are in a buffer
// (both hold a half of q_hat / k_hat): the owner writes them to its warp's
// spare row, each lane takes four and writes its words (re-rounded where
// needed) over the staged halves.
__device__ __forceinline__ void fix_staged_halves(unsigned todo, const uint32_t (&yb)[64], uint32_t spare,
                                                  uint32_t hat, float r, const float* g, int lane) {
  while (todo) {
    const int o = __ffs(todo) - 1;
    todo &= todo - 1;
    if (lane == o) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        st_shared_v4(spare + c * 16, yb[4 * c], yb[4 * c + 1], yb[4 * c + 2], yb[4 * c + 3]);
    }
    const float ro = __shfl_sync(0xffffffffu, r, o);
    __syncwarp();
    // Words 2 lane, 2 lane + 1 of row o: elements 4 lane .. 4 lane + 3.
    const uint32_t w0 = ld_shared_u32(spare + lane * 8), w1 = ld_shared_u32(spare + lane * 8 + 4);
    float s = 0.f, c = 0.f;
    add_sq_df(w0, s, c);
    add_sq_df(w1, s, c);
    warp_sum_df(s, c);
    float rh, rl;
    rsqrt_mean_eps_df(s, c, 1.f / 128, rh, rl);
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * lane + j;
      const uint32_t w = j < 2 ? w0 : w1;
      const float x = (j & 1) ? bf_hi(w) : bf_lo(w);
      const float z = __fmul_rn(__fmul_rn(g[e], x), ro);
      f[j] = near_bf16_midpoint(z) ? round_bf16_df(g[e], x, rh, rl) : z;
    }
    const uint32_t at = staged(hat + (lane >> 4) * kStagingBytes, o, (lane & 15) >> 1) + (lane & 1) * 8;
    st_shared_u32(at, pack_bf16x2(f[0], f[1]));
    st_shared_u32(at + 4, pack_bf16x2(f[2], f[3]));
    __syncwarp();  // the spare row is free again
  }
}

enum QkvMode { kBf16 = 0, kE4m3 = 1, kLora = 2 };

// One (U, B) pair of a kLora stage: 128 rows and 256 columns, 16 of the rank.
constexpr int kPairA = kBM * 32, kPairB = kBN * 32, kPairBytes = kPairA + kPairB;
constexpr int kStagePairs = kStageBytes / kPairBytes;

struct QkvStream {
  int M;       // token rows (B * N_s)
  int N_s;     // tokens per batch item
  int row0;    // the stream's first row in the joint sequence
  int tile0;   // its first tile
  const float* bias;  // [3 H d] or null
  const float *sx, *sw;  // kE4m3: scales of the token rows and of the weight's rows
};

struct QkvParams {
  QkvStream s[2];     // 0: image stream, 1: caption stream
  int H, C, N;        // heads, model width (K of the product), joint sequence length
  int n_tiles;        // column tiles: ceil(3 H d / 256)
  int tiles;          // all tiles of both streams
  uint16_t* out[3];   // q, k, v: [B, H, N, d]
  uint16_t* hat[2];   // q_hat, k_hat
  float* r[2];        // rq, rk: [B, H, N]
  // kLora: the batch items' adapters (none where outside 0 .. n_adapters - 1),
  // pairs of 16 of the rank, and whether a stream has adapters.
  const int* index;
  int n_adapters, rank_pairs;
  bool lora[2];
};

// kLora: U [M, 3 * 16 rank_pairs] and the adapters' up weights [n, 3 H d, rank], image then caption stream.
struct QkvLoraMaps {
  CUtensorMap u[2], up[2];
};

// The next run of consecutive batch items with one adapter among rows m0 ..
// m1 - 1 of a stream, from item b on: the adapter and the rows lo .. hi - 1
// of the tile.  Items without an adapter are passed over.
__device__ __forceinline__ bool next_run(const QkvParams& p, int N_s, int m0, int m1, int& b, int& adapter, int& lo,
                                         int& hi) {
  while (b * N_s < m1) {
    adapter = __ldg(p.index + b);
    lo = max(b * N_s, m0) - m0;
    do ++b;
    while (b * N_s < m1 && __ldg(p.index + b) == adapter);
    hi = min(b * N_s, m1) - m0;
    if (adapter >= 0 && adapter < p.n_adapters) return true;
  }
  return false;
}
// The q, k, v parts that columns n0 .. n0 + 255 meet.
__device__ __forceinline__ void parts_of(int n0, int hd, int& first, int& last) {
  first = n0 / hd;
  last = min((n0 + kBN - 1) / hd, 2);
}

// TMA maps over the five outputs ([B H, N, d] bf16, box 64 columns x 32 rows,
// 128-byte swizzle: the staging buffers' layout), for warps whose 32 rows lie
// in one batch item.
struct QkvOutMaps {
  CUtensorMap out[3];  // q, k, v
  CUtensorMap hat[2];  // q_hat, k_hat
};
__device__ __forceinline__ void tma_store_3d_s(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Field selection by a runtime index through selects: indexing the kernel's
// parameter arrays with a runtime value would copy them to local memory.
__device__ __forceinline__ uint16_t* out_of(const QkvParams& p, int which) {
  return which == 0 ? p.out[0] : which == 1 ? p.out[1] : p.out[2];
}
__device__ __forceinline__ uint16_t* hat_of(const QkvParams& p, int which) { return which == 0 ? p.hat[0] : p.hat[1]; }
__device__ __forceinline__ float* r_of(const QkvParams& p, int which) { return which == 0 ? p.r[0] : p.r[1]; }
__device__ __forceinline__ const CUtensorMap* out_map(const QkvOutMaps& m, int which) {
  return which == 0 ? &m.out[0] : which == 1 ? &m.out[1] : &m.out[2];
}
__device__ __forceinline__ const CUtensorMap* hat_map(const QkvOutMaps& m, int which) {
  return which == 0 ? &m.hat[0] : &m.hat[1];
}

// Where a warp's 32 staged rows go: one TMA tile store when they are 32
// consecutive rows of one head (contig; n0 and bh0 = b H of the first row),
// else the row-by-row stores of store_rows.
struct RowsOut {
  bool contig;
  int n0, bh0;
};
template <int D>
__device__ __forceinline__ void emit_rows(uint32_t buf, const CUtensorMap* map, uint16_t* base, const RowsOut& ro,
                                          const uint32_t (&rows)[8], uint32_t head_rows, int h, int col, int lane) {
  if (ro.contig) {
    fence_proxy_async_smem();  // this lane's staged writes, to the TMA unit
    __syncwarp();
    if (lane == 0) {
      tma_store_3d_s(map, buf, col, ro.n0, ro.bh0 + h);
      bulk_commit_group();
    }
  } else {
    __syncwarp();
    store_rows<D>(buf, base, rows, head_rows, col, lane);
  }
}
// Before a staging buffer is written again: the TMA stores have read it.
__device__ __forceinline__ void staging_free(int lane) {
  if (lane == 0) bulk_wait_group_read0();
  __syncwarp();
}
__device__ __forceinline__ QkvStream stream_of(const QkvParams& p, int si) {
  QkvStream s;
  s.M = si ? p.s[1].M : p.s[0].M;
  s.N_s = si ? p.s[1].N_s : p.s[0].N_s;
  s.row0 = si ? p.s[1].row0 : p.s[0].row0;
  s.tile0 = si ? p.s[1].tile0 : p.s[0].tile0;
  s.bias = si ? p.s[1].bias : p.s[0].bias;
  s.sx = si ? p.s[1].sx : p.s[0].sx;
  s.sw = si ? p.s[1].sw : p.s[0].sw;
  return s;
}

// r of one row from its bf16 values (packed pairs; exact squares): a
// balanced tree, built block by block (16 values, then across the D / 16
// blocks) so that few partial sums are live at once.  Two neighbouring sums at
// a time in packed fp32 arithmetic; the fma adds two exact squares with one
// rounding, as an addition of them does.
template <int D>
__device__ __forceinline__ float row_rsqrt(const uint32_t (&yb)[D / 2]) {
  float blk[D / 16];
#pragma unroll
  for (int b = 0; b < D / 16; ++b) {
    uint64_t t[4];  // sums of the words (0, 1), (2, 3), (4, 5), (6, 7)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = yb[b * 8 + 2 * i], v = yb[b * 8 + 2 * i + 1];
      const uint64_t lo = f2_make(bf_lo(u), bf_lo(v)), hi = f2_make(bf_hi(u), bf_hi(v));
      t[i] = f2_fma(lo, lo, f2_mul(hi, hi));
    }
    const uint64_t s = f2_add(f2_add(t[0], t[2]), f2_add(t[1], t[3]));
    float s0, s1;
    f2_split(s, s0, s1);
    blk[b] = __fadd_rn(s0, s1);
  }
#pragma unroll
  for (int w = D / 32; w >= 1; w >>= 1)
#pragma unroll
    for (int i = 0; i < w; ++i) blk[i] = __fadd_rn(blk[i], blk[i + w]);
  return rsqrtf(__fadd_rn(__fmul_rn(blk[0], 1.f / D), kEps));
}

// Elements near a bf16 midpoint, two at a time: the smaller of the low halves'
// distances above the window's start, per half of m, starting from kNoneNear
// (the test of near_bf16_midpoint).
constexpr uint32_t kNoneNear = 0xFFFFFFFFu;
__device__ __forceinline__ void near_pair(float z0, float z1, uint32_t& m) {
  constexpr uint32_t kFrom = (0x10000u + kTieWindow / 2 - 0x8000u) & 0xFFFFu;
  m = __viaddmin_u16x2(__byte_perm(__float_as_uint(z0), __float_as_uint(z1), 0x5410), kFrom * 0x10001u, m);
}
__device__ __forceinline__ bool any_near(uint32_t m) {
  return (m & 0xFFFFu) < kTieWindow || (m >> 16) < kTieWindow;
}

// 64 columns of this lane's q_hat / k_hat row, (g x) r per element, staged
// 16 bytes at a time into its row of the staging buffer; `near` collects the
// elements within the midpoint window.
__device__ __forceinline__ void stage_hat_row(uint32_t buf, const uint32_t* y, uint32_t g, float r, uint32_t& near,
                                              int lane) {
  const uint64_t r2 = f2_make(r, r);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    // The gains through ordered shared loads: loaded chunk by chunk, not all
    // at once ahead of the loop.
    const float4 ga = ld_shared_f4(g + c * 32), gb = ld_shared_f4(g + c * 32 + 16);
    const uint64_t gv[4] = {f2_make(ga.x, ga.y), f2_make(ga.z, ga.w), f2_make(gb.x, gb.y), f2_make(gb.z, gb.w)};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t yv = y[4 * c + i];
      float z0, z1;
      f2_split(f2_mul(f2_mul(gv[i], f2_make(bf_lo(yv), bf_hi(yv))), r2), z0, z1);
      near_pair(z0, z1, near);
      w[i] = pack_bf16x2(z0, z1);
    }
    st_shared_v4(staged(buf, lane, c), w[0], w[1], w[2], w[3]);
  }
}

// One head of the warp's 32 token rows: D accumulator columns at taddr
// (this lane's row).  row: head 0's row index (b H N + n) of this lane; the
// head's is row + h N.  bias: this head's D bias values in shared memory.
// kE4m3: sx, the row's scale, and wscale, the D columns' in shared memory.
template <int D, int kMode>
__device__ __forceinline__ void qkv_emit_head(uint32_t taddr, int ocol, bool live, size_t row,
                                              const uint32_t (&rows)[8], const RowsOut& ro, uint32_t stg,
                                              uint32_t bias, float sx, uint32_t wscale, uint32_t spare, const QkvParams& p,
                                              const QkvOutMaps& om, const QkvBars& bars, int lane) {
  const int hd = p.H * D;
  const int which = ocol / hd;  // 0 q, 1 k, 2 v
  const int h = (ocol - which * hd) / D;
  const uint32_t head_rows = static_cast<uint32_t>(h) * static_cast<uint32_t>(p.N);
  const size_t hrow = row + head_rows;
  const uint32_t raw = stg;
  // Y = bf16(acc + bias), 32 columns at a time (packed pairs).
  uint32_t yb[D / 2];
  const uint64_t sx2 = f2_make(sx, sx);
#pragma unroll
  for (int c32 = 0; c32 < D / 32; ++c32) {
    uint32_t acc[32];
    tmem_ld32(taddr + c32 * 32, acc);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      const float4 bv = ld_shared_f4(bias + (c32 * 32 + e) * 4);
      uint64_t y0 = f2_make(__uint_as_float(acc[e]), __uint_as_float(acc[e + 1]));
      uint64_t y1 = f2_make(__uint_as_float(acc[e + 2]), __uint_as_float(acc[e + 3]));
      if constexpr (kMode == kE4m3) {
        const float4 sv = ld_shared_f4(wscale + (c32 * 32 + e) * 4);
        y0 = f2_fma(f2_mul(y0, sx2), f2_make(sv.x, sv.y), f2_make(bv.x, bv.y));
        y1 = f2_fma(f2_mul(y1, sx2), f2_make(sv.z, sv.w), f2_make(bv.z, bv.w));
      } else {
        y0 = f2_add(y0, f2_make(bv.x, bv.y));
        y1 = f2_add(y1, f2_make(bv.z, bv.w));
      }
      float a0, a1, a2, a3;
      f2_split(y0, a0, a1);
      f2_split(y1, a2, a3);
      yb[c32 * 16 + e / 2] = pack_bf16x2(a0, a1);
      yb[c32 * 16 + e / 2 + 1] = pack_bf16x2(a2, a3);
    }
  }
  const float* g = which == 0 ? bars.gq : bars.gk;
  if constexpr (D == 64) {
    const uint32_t hat = raw + kStagingBytes;
    staging_free(lane);
    stage_row(raw, yb, lane);
    if (which == 2) {
      emit_rows<D>(raw, out_map(om, which), out_of(p, which), ro, rows, head_rows, h, 0, lane);
      __syncwarp();
      return;
    }
    const float r = row_rsqrt<D>(yb);
    uint32_t near = kNoneNear;
    stage_hat_row(hat, yb, smem_u32(g), r, near, lane);
    const unsigned todo = __ballot_sync(0xffffffffu, any_near(near) && live);
    __syncwarp();
    if (todo) {
      fix_staged_rows(todo, raw, hat, r, g, lane);
      __syncwarp();
    }
    emit_rows<D>(raw, out_map(om, which), out_of(p, which), ro, rows, head_rows, h, 0, lane);
    emit_rows<D>(hat, hat_map(om, which), hat_of(p, which), ro, rows, head_rows, h, 0, lane);
    if (live) r_of(p, which)[hrow] = r;
    __syncwarp();
  } else {
    // d = 128: a 64-column half in each buffer, raw, then q_hat / k_hat.
    staging_free(lane);
#pragma unroll
    for (int h64 = 0; h64 < 2; ++h64) {
      const uint32_t buf = raw + h64 * kStagingBytes;
      stage_row(buf, yb + h64 * 32, lane);
      emit_rows<D>(buf, out_map(om, which), out_of(p, which), ro, rows, head_rows, h, h64 * 64, lane);
    }
    __syncwarp();
    if (which == 2) return;
    const float r = row_rsqrt<D>(yb);
    uint32_t near = kNoneNear;
    staging_free(lane);
    stage_hat_row(raw, yb, smem_u32(g), r, near, lane);
    stage_hat_row(raw + kStagingBytes, yb + 32, smem_u32(g + 64), r, near, lane);
    const unsigned todo = __ballot_sync(0xffffffffu, any_near(near) && live);
    __syncwarp();
    if (todo)
      fix_staged_halves(todo, *reinterpret_cast<const uint32_t(*)[64]>(yb), spare, raw, r, g, lane);
#pragma unroll
    for (int h64 = 0; h64 < 2; ++h64)
      emit_rows<D>(raw + h64 * kStagingBytes, hat_map(om, which), hat_of(p, which), ro, rows, head_rows, h, h64 * 64,
                   lane);
    if (live) r_of(p, which)[hrow] = r;
    __syncwarp();
  }
}

template <int D, int kMode>
__global__ void __launch_bounds__(QkvCfg<D>::kThreads, 1)
    qkv_norm_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_w0,
                    const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ QkvOutMaps om, const __grid_constant__ QkvLoraMaps lm,
                    const __grid_constant__ QkvParams p, const float* __restrict__ gq,
                    const float* __restrict__ gk, uint32_t* dev_err) {
  using Cfg = QkvCfg<D>;
  constexpr int kStepK = kMode == kE4m3 ? 2 * kBK : kBK;  // values in a K step's 128-byte rows
  constexpr int kWarpProd = Cfg::kWarpProd, kWarpIssue = Cfg::kWarpIssue;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) QkvBars bars;
  uint8_t* sm = align1024(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* ab = &bars.abort;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kQkvStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], Cfg::kEpiThreads);
    }
    mbar_init(&bars.mma_done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpIssue) {
    tmem_alloc(&bars.tmem_base, 2 * kBN);
    tmem_relinquish();
  }
  griddep_wait();  // the previous grid's writes are visible from here on
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    bars.gq[i] = gq[i];
    bars.gk[i] = gk[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int ksteps = (p.C + kStepK - 1) / kStepK;

  if (warp == kWarpProd) {
    if (lane == 0) {
      tma_prefetch_desc(&map_x0);
      tma_prefetch_desc(&map_w0);
      tma_prefetch_desc(&map_x1);
      tma_prefetch_desc(&map_w1);
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
        const int si = t >= p.s[1].tile0 ? 1 : 0;
        const int tl = t - (si ? p.s[1].tile0 : p.s[0].tile0);
        const int mt = tl / p.n_tiles, nt = tl - mt * p.n_tiles;
        const CUtensorMap* mx = si ? &map_x1 : &map_x0;
        const CUtensorMap* mw = si ? &map_w1 : &map_w0;
        for (int kb = 0; kb < ksteps; ++kb) {
          const int s = it % kQkvStages;
          if (it >= kQkvStages && !(ok = mbar_wait(&bars.empty[s], ((it / kQkvStages) - 1) & 1, ab, dev_err)))
            break;
          uint8_t* st = sm + s * kStageBytes;
          mbar_arrive_expect_tx(&bars.full[s], kStageBytes);
          tma_load_2d(st, mx, &bars.full[s], kb * kStepK, mt * kBM);
          tma_load_2d(st + kATile, mw, &bars.full[s], kb * kStepK, nt * kBN);
          ++it;
        }
        if constexpr (kMode == kLora) {
          if (!ok || !(si ? p.lora[1] : p.lora[0])) continue;
          const int N_s = si ? p.s[1].N_s : p.s[0].N_s, M = si ? p.s[1].M : p.s[0].M;
          const int m0 = mt * kBM, m1 = min(m0 + kBM, M);
          const CUtensorMap* mu = si ? &lm.u[1] : &lm.u[0];
          const CUtensorMap* mup = si ? &lm.up[1] : &lm.up[0];
          int p0, p1, b = m0 / N_s, adapter, lo, hi, left = 0;
          parts_of(nt * kBN, p.H * D, p0, p1);
          const int per_run = (p1 - p0 + 1) * p.rank_pairs;
          while (next_run(p, N_s, m0, m1, b, adapter, lo, hi)) left += per_run;
          int in_stage = 0;
          b = m0 / N_s;
          while (ok && left > 0 && next_run(p, N_s, m0, m1, b, adapter, lo, hi)) {
            for (int j = 0; ok && j < per_run; ++j, --left) {
              const int s = it % kQkvStages;
              if (in_stage == 0) {
                if (it >= kQkvStages &&
                    !(ok = mbar_wait(&bars.empty[s], ((it / kQkvStages) - 1) & 1, ab, dev_err)))
                  break;
                mbar_arrive_expect_tx(&bars.full[s], min(left, kStagePairs) * kPairBytes);
              }
              uint8_t* st = sm + s * kStageBytes + in_stage * kPairBytes;
              const int part = p0 + j / p.rank_pairs, kc = j % p.rank_pairs;
              tma_load_2d(st, mu, &bars.full[s], (part * p.rank_pairs + kc) * 16, m0);
              tma_load_3d(st + kPairA, mup, &bars.full[s], kc * 16, nt * kBN, adapter);
              if (++in_stage == kStagePairs || left == 1) {
                in_stage = 0;
                ++it;
              }
            }
          }
        }
      }
      if (*ab) {  // aborted: the copies in flight land before the CTA exits
        for (int i = (it > kQkvStages ? it - kQkvStages : 0); i < it; ++i)
          mbar_wait_drain(&bars.full[i % kQkvStages], (i / kQkvStages) & 1);
      }
    }
  } else if (warp == kWarpIssue) {
    if (lane == 0) {
      constexpr uint32_t idesc =
          kMode == kE4m3 ? idesc_e4m3_f32(kBM, kBN) : idesc_bf16_f32(kBM, kBN, false, false);
      int it = 0, lt = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x, ++lt) {
        const int abuf = lt & 1;
        if (lt >= 2 && !(ok = mbar_wait(&bars.acc_empty[abuf], ((lt >> 1) - 1) & 1, ab, dev_err))) break;
        tc_fence_after();
        const uint32_t acc = tmem + abuf * kBN;
        for (int kb = 0; kb < ksteps; ++kb, ++it) {
          const int s = it % kQkvStages;
          if (!(ok = mbar_wait(&bars.full[s], (it / kQkvStages) & 1, ab, dev_err))) break;
          tc_fence_after();
          const uint32_t st = smem_u32(sm + s * kStageBytes);
          const uint64_t a = sdesc_sw128(st, 16, 1024), b = sdesc_sw128(st + kATile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {  // 32 bytes of each row: 16 bf16 or 32 e4m3 values
            const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
            if constexpr (kMode == kE4m3)
              umma_f8_ss(acc, desc_add(a, kk * 32), desc_add(b, kk * 32), idesc, add);
            else
              umma_bf16_ss(acc, desc_add(a, kk * 32), desc_add(b, kk * 32), idesc, add);
          }
          umma_commit(&bars.empty[s]);
        }
        if constexpr (kMode == kLora) {
          const int si = t >= p.s[1].tile0 ? 1 : 0;
          if (ok && (si ? p.lora[1] : p.lora[0])) {
            const int tl = t - (si ? p.s[1].tile0 : p.s[0].tile0);
            const int mt = tl / p.n_tiles, n0 = (tl - mt * p.n_tiles) * kBN;
            const int N_s = si ? p.s[1].N_s : p.s[0].N_s, M = si ? p.s[1].M : p.s[0].M;
            const int m0 = mt * kBM, m1 = min(m0 + kBM, M), hd = p.H * D;
            int p0, p1, b = m0 / N_s, adapter, lo, hi, in_stage = 0;
            parts_of(n0, hd, p0, p1);
            while (ok && next_run(p, N_s, m0, m1, b, adapter, lo, hi)) {
              uint32_t off[4];  // the lanes (rows) that the run does not hold
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int l = min(max(lo - 32 * w, 0), 32), h = min(max(hi - 32 * w, 0), 32);
                const uint32_t below = l >= 32 ? 0xFFFFFFFFu : (1u << l) - 1u;
                const uint32_t upto = h >= 32 ? 0xFFFFFFFFu : (1u << h) - 1u;
                off[w] = ~(upto & ~below);
              }
              for (int part = p0; ok && part <= p1; ++part) {
                const int c0 = max(part * hd, n0) - n0, c1 = min((part + 1) * hd, n0 + kBN) - n0;
                const uint32_t desc = idesc_bf16_f32(kBM, c1 - c0, false, false);
                for (int kc = 0; kc < p.rank_pairs; ++kc) {
                  const int s = it % kQkvStages;
                  if (in_stage == 0) {
                    if (!(ok = mbar_wait(&bars.full[s], (it / kQkvStages) & 1, ab, dev_err))) break;
                    tc_fence_after();
                  }
                  const uint32_t st = smem_u32(sm + s * kStageBytes + in_stage * kPairBytes);
                  umma_bf16_ss_lanes(acc + c0, sdesc_sw32_kmajor(st, 256),
                                     sdesc_sw32_kmajor(st + kPairA + c0 * 32, 256), desc, off, 1u);
                  if (++in_stage == kStagePairs) {
                    in_stage = 0;
                    umma_commit(&bars.empty[s]);
                    ++it;
                  }
                }
              }
            }
            if (ok && in_stage > 0) {
              umma_commit(&bars.empty[it % kQkvStages]);
              ++it;
            }
          }
        }
        if (ok) umma_commit(&bars.acc_full[abuf]);
      }
      // Every MMA this thread issued has completed once this barrier flips.
      umma_commit(&bars.mma_done);
      mbar_wait_drain(&bars.mma_done, 0);
    }
  } else {
    // Warp w: the TMEM lanes of warp w % 4, and columns 128 (w / 4) .. + 127 of the tile.
    const int lg = warp & 3, wcol = (warp >> 2) * 128;
    const uint32_t stg = smem_u32(sm + Cfg::kOffStaging + warp * Cfg::kStaging);
    const uint32_t bias_w = smem_u32(sm + Cfg::kOffBias + warp * Cfg::kBiasBytes);
    const uint32_t wscale_w = smem_u32(sm + Cfg::kOffScale + warp * Cfg::kBiasBytes);  // kE4m3
    const uint32_t spare_w = smem_u32(sm + Cfg::kOffSpare + warp * Cfg::kSpareBytes);
    const uint32_t lane_base = static_cast<uint32_t>(lg * 32) << 16;
    const int hd3 = 3 * p.H * D;
    int lt = 0;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, ++lt) {
      const int abuf = lt & 1;
      const int si = t >= p.s[1].tile0 ? 1 : 0;
      const QkvStream S = stream_of(p, si);
      const int tl = t - S.tile0;
      const int mt = tl / p.n_tiles, nt = tl - mt * p.n_tiles;
      const int col0 = nt * kBN + wcol;  // the warp's first column in Y
      // The bias of the warp's 128 columns (zero past 3 H d, or without a
      // bias) into its shared slice, while the products are still running.
      float4 bq = make_float4(0.f, 0.f, 0.f, 0.f);
      if (S.bias && col0 + lane * 4 < hd3) bq = __ldg(reinterpret_cast<const float4*>(S.bias + col0) + lane);
      __syncwarp();  // the previous tile's reads of the slice are done
      st_shared_v4(bias_w + lane * 16, __float_as_uint(bq.x), __float_as_uint(bq.y), __float_as_uint(bq.z),
                   __float_as_uint(bq.w));
      if constexpr (kMode == kE4m3) {
        float4 sq = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col0 + lane * 4 < hd3) sq = __ldg(reinterpret_cast<const float4*>(S.sw + col0) + lane);
        st_shared_v4(wscale_w + lane * 16, __float_as_uint(sq.x), __float_as_uint(sq.y), __float_as_uint(sq.z),
                     __float_as_uint(sq.w));
      }
      const bool ok = mbar_wait(&bars.acc_full[abuf], (lt >> 1) & 1, ab, dev_err);
      if (!__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      tc_fence_after();
      const int m = mt * kBM + lg * 32 + lane;
      const bool live = m < S.M;
      float sx = 0.f;
      if constexpr (kMode == kE4m3) {
        if (live) sx = __ldg(S.sx + m);
      }
      const int bi = live ? m / S.N_s : 0;
      const int n = live ? S.row0 + (m - bi * S.N_s) : 0;
      const size_t row = static_cast<size_t>(bi) * p.H * p.N + n;  // < B H N < 2^31 / d
      const uint32_t row32 = live ? static_cast<uint32_t>(row) : kDeadRow;
      uint32_t rows[8];  // the rows this lane writes out in store_rows
#pragma unroll
      for (int j = 0; j < 8; ++j) rows[j] = __shfl_sync(0xffffffffu, row32, 4 * j + (lane >> 3));
      RowsOut ro;
      {
        const uint32_t first = __shfl_sync(0xffffffffu, row32, 0), last = __shfl_sync(0xffffffffu, row32, 31);
        ro.contig = first != kDeadRow && last != kDeadRow && last - first == 31u;
        ro.n0 = __shfl_sync(0xffffffffu, n, 0);
        ro.bh0 = __shfl_sync(0xffffffffu, bi, 0) * p.H;
      }
#pragma unroll
      for (int j = 0; j < 128 / D; ++j) {
        const int ocol = col0 + j * D;  // the head's first column in Y
        if (ocol < hd3)
          qkv_emit_head<D, kMode>(tmem + lane_base + abuf * kBN + wcol + j * D, ocol, live, row, rows, ro, stg,
                                  bias_w + j * D * 4, sx, wscale_w + j * D * 4, spare_w, p, om, bars, lane);
      }
      tc_fence_before();
      mbar_arrive(&bars.acc_empty[abuf]);
    }
    if (lane == 0) bulk_wait_group0();  // this warp's tile stores are complete
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kBN);
  }
}


// --- U = scale X A^T, rounded to bf16 ---------------------------------------
// One CTA per batch item, stream and block of 128 of its token rows: an item
// has one adapter, whose down weights [3 rank, C] are the product's other
// operand, N = 3 * 16 rank_pairs columns (a rank that is not a multiple of 16
// reads the TMA's zero fill).  Items without an adapter write nothing (the
// projection reads nothing of theirs).  The rounding of U to bf16 is that of
// the projection's own operands: U is the left operand of the second product.
// Warps 0-3 read the accumulator out (a row a thread), warp 4 loads, warp 5
// issues.
constexpr int kDownThreads = 192;
constexpr int kDownMaxStages = 6;
constexpr int kDownSmem = 200 * 1024;

struct DownStream {
  int N_s, blocks, cta0;  // rows per item, its 128-row blocks, the stream's first CTA
  uint16_t* u;            // [B N_s, 3 * 16 rank_pairs]
};
struct DownParams {
  DownStream s[2];
  int C, rank_pairs, n_adapters, stages, tmem_cols;
  const int* index;
  const float* scale;
};
struct DownMaps {
  CUtensorMap x[2], down[2];  // [B, N_s, C] with 128-row boxes; [3 n, rank, C] with 16 rank_pairs rows
};
struct DownBars {
  uint64_t full[kDownMaxStages], empty[kDownMaxStages], done;
  uint32_t tmem_base;
  int abort;
};

__global__ void __launch_bounds__(kDownThreads, 1)
    lora_down_kernel(const __grid_constant__ DownMaps maps, const __grid_constant__ DownParams p,
                     uint32_t* dev_err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) DownBars bars;
  uint8_t* sm = align1024(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* ab = &bars.abort;
  griddep_launch_dependents();
  griddep_wait();
  const int si = static_cast<int>(blockIdx.x) >= p.s[1].cta0 ? 1 : 0;
  const int N_s = si ? p.s[1].N_s : p.s[0].N_s, blocks = si ? p.s[1].blocks : p.s[0].blocks;
  const int local = blockIdx.x - (si ? p.s[1].cta0 : p.s[0].cta0);
  const int item = local / blocks, row0 = (local - item * blocks) * kBM;
  const int adapter = __ldg(p.index + item);
  if (adapter < 0 || adapter >= p.n_adapters) return;  // the whole CTA
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&bars.tmem_base, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int ksteps = (p.C + kBK - 1) / kBK;
  const int r16 = 16 * p.rank_pairs;
  const int stage_bytes = kATile + 3 * r16 * 128;
  if (warp == 4) {
    if (lane == 0) {
      const CUtensorMap* mx = si ? &maps.x[1] : &maps.x[0];
      const CUtensorMap* md = si ? &maps.down[1] : &maps.down[0];
      int kb = 0;
      for (; kb < ksteps; ++kb) {
        const int s = kb % p.stages;
        if (kb >= p.stages && !mbar_wait(&bars.empty[s], ((kb / p.stages) - 1) & 1, ab, dev_err)) break;
        uint8_t* st = sm + s * stage_bytes;
        mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
        tma_load_3d(st, mx, &bars.full[s], kb * kBK, row0, item);
        for (int part = 0; part < 3; ++part)
          tma_load_3d(st + kATile + part * r16 * 128, md, &bars.full[s], kb * kBK, 0, 3 * adapter + part);
      }
      if (*ab) {  // aborted: the copies in flight land before the CTA exits
        for (int i = (kb > p.stages ? kb - p.stages : 0); i < kb; ++i)
          mbar_wait_drain(&bars.full[i % p.stages], (i / p.stages) & 1);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const bool one = 3 * r16 <= 256;
      const uint32_t idesc = idesc_bf16_f32(kBM, one ? 3 * r16 : r16, false, false);
      for (int kb = 0; kb < ksteps; ++kb) {
        const int s = kb % p.stages;
        if (!mbar_wait(&bars.full[s], (kb / p.stages) & 1, ab, dev_err)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(sm + s * stage_bytes);
        const uint64_t a = sdesc_sw128(st, 16, 1024), b = sdesc_sw128(st + kATile, 16, 1024);
        for (int kk = 0; kk < kBK / 16; ++kk) {
          const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
          for (int part = 0; part < (one ? 1 : 3); ++part)
            umma_bf16_ss(tmem + part * r16, desc_add(a, kk * 32), desc_add(b, kk * 32 + part * r16 * 128), idesc,
                         add);
        }
        umma_commit(&bars.empty[s]);
      }
      // Every MMA this thread issued has completed once this barrier flips.
      umma_commit(&bars.done);
      mbar_wait_drain(&bars.done, 0);
    }
  } else {
    bool ok = mbar_wait(&bars.done, 0, ab, dev_err);
    ok = __all_sync(0xffffffffu, ok) && !*ab;
    __syncwarp();
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const float scale = __ldg(p.scale + adapter);
      const int n = row0 + warp * 32 + lane;
      uint16_t* u = (si ? p.s[1].u : p.s[0].u) + (static_cast<size_t>(item) * N_s + n) * (3 * r16);
      for (int c = 0; c < 3 * p.rank_pairs; ++c) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c * 16, v);
        tmem_wait_ld();
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = pack_bf16x2(__uint_as_float(v[2 * i]) * scale, __uint_as_float(v[2 * i + 1]) * scale);
        if (n < N_s) {
          uint4* o = reinterpret_cast<uint4*>(u + c * 16);
          o[0] = make_uint4(w[0], w[1], w[2], w[3]);
          o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

}  // namespace

cudaError_t launch_lora_down(const CUtensorMap (&x)[2], const CUtensorMap (&down)[2], const LoraLaunch& l,
                             const QkvLaunch& a, int B, uint32_t* dev_err, cudaStream_t st) {
  DownMaps maps;
  DownParams p;
  const int r16 = (l.rank + 15) / 16 * 16;
  int ctas = 0;
  for (int i = 0; i < 2; ++i) {
    maps.x[i] = x[i];
    maps.down[i] = down[i];
    p.s[i].N_s = a.N_s[i];
    p.s[i].blocks = l.on[i] ? (a.N_s[i] + kBM - 1) / kBM : 0;
    p.s[i].cta0 = ctas;
    p.s[i].u = l.u[i];
    ctas += B * p.s[i].blocks;
  }
  if (ctas == 0) return cudaSuccess;
  p.C = a.C;
  p.rank_pairs = r16 / 16;
  p.n_adapters = l.n_adapters;
  const int stage_bytes = kATile + 3 * r16 * 128;
  p.stages = kDownSmem / stage_bytes < kDownMaxStages ? kDownSmem / stage_bytes : kDownMaxStages;
  p.tmem_cols = 32;
  while (p.tmem_cols < 3 * r16) p.tmem_cols *= 2;
  p.index = l.index;
  p.scale = l.scale;
  const int smem = p.stages * stage_bytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(lora_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_down_kernel, dim3(ctas), dim3(kDownThreads), smem, st, maps, p, dev_err);
}

cudaError_t launch_qkv_norm(const CUtensorMap (&maps)[4], const CUtensorMap (&out_maps)[5], const QkvLaunch& a,
                            uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora,
                            const CUtensorMap* lora_maps) {
  QkvOutMaps om;
  for (int i = 0; i < 3; ++i) om.out[i] = out_maps[i];
  for (int i = 0; i < 2; ++i) om.hat[i] = out_maps[3 + i];
  QkvLoraMaps lm;
  for (int i = 0; i < 2; ++i) {
    lm.u[i] = lora ? lora_maps[i] : maps[0];
    lm.up[i] = lora ? lora_maps[2 + i] : maps[0];
  }
  QkvParams p;
  p.H = a.H;
  p.C = a.C;
  p.N = a.N;
  p.n_tiles = (3 * a.H * a.d + kBN - 1) / kBN;
  int tile0 = 0;
  for (int i = 0; i < 2; ++i) {
    p.s[i].M = a.M[i];
    p.s[i].N_s = a.N_s[i];
    p.s[i].row0 = a.row0[i];
    p.s[i].tile0 = tile0;
    p.s[i].bias = a.bias[i];
    p.s[i].sx = a.sx[i];
    p.s[i].sw = a.sw[i];
    tile0 += ((a.M[i] + kBM - 1) / kBM) * p.n_tiles;
    p.lora[i] = lora && lora->on[i];
  }
  p.tiles = tile0;
  for (int i = 0; i < 3; ++i) p.out[i] = a.out[i];
  for (int i = 0; i < 2; ++i) {
    p.hat[i] = a.hat[i];
    p.r[i] = a.r[i];
  }
  p.index = lora ? lora->index : nullptr;
  p.n_adapters = lora ? lora->n_adapters : 0;
  p.rank_pairs = lora ? (lora->rank + 15) / 16 : 0;
  if (p.tiles == 0) return cudaSuccess;
  const int sms = device_sm_count();
  const int grid = p.tiles < sms ? p.tiles : sms;
  auto go = [&](auto kernel, int threads, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(threads), smem, st, maps[0], maps[1], maps[2], maps[3], om, lm, p,
                      a.gq, a.gk, dev_err);
  };
  auto go_d = [&](auto cfg, auto plain, auto e4m3, auto with_lora) {
    using Cfg = decltype(cfg);
    if (lora) return go(with_lora, Cfg::kThreads, Cfg::kDynSmem);
    if (a.e4m3) return go(e4m3, Cfg::kThreads, Cfg::kDynSmemE4m3);
    return go(plain, Cfg::kThreads, Cfg::kDynSmem);
  };
  if (a.d == 64)
    return go_d(QkvCfg<64>(), qkv_norm_kernel<64, kBf16>, qkv_norm_kernel<64, kE4m3>, qkv_norm_kernel<64, kLora>);
  return go_d(QkvCfg<128>(), qkv_norm_kernel<128, kBf16>, qkv_norm_kernel<128, kE4m3>, qkv_norm_kernel<128, kLora>);
}

}  // namespace jattn
