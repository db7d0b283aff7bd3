// qkv_proj.cuh — the QKV projections of the two token streams with QK-RMSNorm
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
// Tiles (template kPair):
//   kPair   256 token rows x 256 output columns by a pair of CTAs
//           (cta_group::2): each CTA keeps 128 rows, all 256 columns of its
//           accumulator in its TMEM, and half of the weight tile in its shared
//           memory.  One CTA alone with 256 columns would load and read the
//           whole weight tile: 96 KB of shared-memory traffic a K step and 128
//           x 256 products instead of 64 KB (the products alone, 768 px from
//           e4m3 rows: 71.9 us so, 66.2 us by pairs).
//   !kPair  128 token rows x one head's columns by one CTA: for few rows,
//           whose tiles are then four (two) times as many.
// K in steps of 128 bytes a row; persistent, the image stream's tiles then the
// caption stream's.  Warps of each CTA:
//   producer    TMA: the X tile (128 rows) and the CTA's part of the W tile of
//               each K step, 128-byte swizzle, through a ring of stages.  Both
//               CTAs of a pair signal the first one's barriers.
//   issuer      (of a pair: the first CTA's) 4 MMAs per K step into one of two
//               TMEM accumulators, so that a tile's epilogue overlaps the next
//               tile's products.
//   epilogue    one thread per token row (TMEM lane), two heads of d = 64 or
//               one of d = 128 (!kPair: one head).  Per head: d fp32 values out
//               of TMEM, + bias (the warp's slice, copied to shared memory
//               while the products run), rounded to bf16 (the projection's
//               output) for q / k / v; for q and k the row's RMSNorm from those
//               bf16 values, q_hat / k_hat and r.  Rows are staged in shared
//               memory and written out as whole 128-byte lines (a TMA tile
//               store, or four rows per store instruction).
// Heads past 3 H in the last column tile, and token rows past the stream's
// end in its last row tile, read the TMA's zero fill and are not stored.
//
// What bounds it (512 px, C = 768, 12 heads of 64; 57 us from bf16, 39 us from
// e4m3): from bf16 a third of the issuer's time goes to waiting for loads, whose
// latency the ring's 128 KB cover only while nothing is written (with the
// stores left out in a timing copy 48 us; 3 stages 62.5, 2 stages 78 us); from
// e4m3 the epilogue's instructions (issue slots 51 % busy, the products alone
// 22.9 us).  16 epilogue warps of 64 columns at d = 64 took 39.4 us where 8 of
// 128 columns took 42.7 (e4m3); at d = 128 a row is a whole head, 8 warps.
//
// The same kernel takes two other forms of the products (template kMode):
//   kE4m3  X and W in e4m3 with fp32 scales of their rows: a K step of 128
//          values in the same 128-byte rows, kind::f8f6f4 products, and
//          Y = bf16(sx sw acc + bias).
//   kLora  low-rank adapters of the batch items' own beside the shared
//          weights: Y = bf16(X W^T + U B^T + bias), U = scale X A^T (one
//          launch of lora_down_kernel before, kept as two bf16 terms) as
//          further K steps of 16 into the same accumulator.  A row tile that
//          holds items with different adapters takes each run of items in
//          turn, with the other rows' lanes disabled in the MMA, so that no row
//          mask or copy of U is needed; a column tile over a q / k / v boundary
//          takes each part with its own columns of U.  A ring stage holds, for
//          16 of the rank at a time, both terms of U (8 KB) and the B rows of
//          as many runs as fit (2 or 4 KB each): two such groups when there
//          is one run, and U loaded once for 6 to 8 runs when there are many.
//
// Correct rounding: the per-thread sum of the d squares is a balanced tree
// (at most 7 roundings per term, within the 8 that the rounding window of the
// norm kernels allows for), and elements in the bf16-midpoint window are
// re-rounded from a double-float r.
#pragma once
#include <atomic>

#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"
#include "bf16_round.cuh"
#include "fastdiv.cuh"

namespace jattn {
namespace {

enum QkvMode { kBf16 = 0, kE4m3 = 1, kLora = 2 };

constexpr int kBM = 128;                            // token rows of one CTA
constexpr int kStepBytes = 128;                     // of each row in a K step
constexpr int kATile = kBM * kStepBytes;            // 16 KB
constexpr int kStageRowBytes = 128;                 // 64 bf16 columns of one token row
constexpr int kStagingBytes = 32 * kStageRowBytes;  // per epilogue warp: its 32 rows of 64 columns
constexpr uint32_t kDeadRow = 0xFFFFFFFFu;
constexpr int kMaxStages = 6;

// Epilogue warps (warps w and w + 4 take the TMEM lanes of warp w % 4, and
// kWarpCols columns each), then the TMA producer and the MMA issuer.  Each
// epilogue warp stages its rows in shared memory, a buffer for each 64 of its
// columns: raw, then q_hat / k_hat.
// kPair: registers per thread (setmaxnreg).  Each SM sub-partition holds the
// epilogue warps w with one w % 4 and one other warp, and an increase draws only
// on the registers those were launched with, so (epilogue warps / 4) x kEpi +
// kOther must be at most (epilogue warps / 4 + 1) x the launch count (allocated
// by eights).  The launcher refuses any build whose register count differs.
template <int D>
struct QkvRegs {
  static constexpr int kLaunch = D == 64 ? 96 : 168, kEpi = D == 64 ? 104 : 208, kOther = D == 64 ? 64 : 88;
  static constexpr int kEpiWarps = D == 64 ? 16 : 8;
  static_assert(kEpiWarps / 4 * kEpi + kOther == (kEpiWarps / 4 + 1) * kLaunch, "projection register split");
};

template <int D, int kMode, bool kPair>
struct QkvCfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kCols = kQkvCols(D, kPair);       // of a tile
  static constexpr int kBRows = kQkvWRows(D, kPair);     // weight rows that a CTA loads
  static constexpr int kWarpCols = kPair && D == 128 ? 128 : D;
  static constexpr int kEpiWarps = 4 * (kCols / kWarpCols);
  static constexpr int kWarpProd = kEpiWarps, kWarpIssue = kEpiWarps + 1;
  static constexpr int kThreads = 32 * (kEpiWarps + (kPair ? 4 : 2));  // kPair: two warps idle
  static_assert(!kPair || kEpiWarps == QkvRegs<D>::kEpiWarps, "register split");
  static constexpr int kStageBytes = kATile + kBRows * kStepBytes;
  static constexpr int kStages = kPair ? 4 : D == 64 ? 6 : 5;
  static constexpr int kTmemCols = 2 * kCols;
  static constexpr int kStaging = kWarpCols / 64 * kStagingBytes;
  static constexpr int kBiasBytes = kWarpCols * 4;       // per epilogue warp: the bias of its columns
  static constexpr int kSpareBytes = D * 2;              // per epilogue warp: fix_staged_rows' row
  static constexpr int kOffStaging = kStages * kStageBytes;
  static constexpr int kOffBias = kOffStaging + kEpiWarps * kStaging;
  static constexpr int kOffSpare = kOffBias + kEpiWarps * 2 * kBiasBytes;  // two tiles' each
  // kE4m3: the scales of the columns, likewise, and of the rows.
  static constexpr int kOffScale = kOffSpare + kEpiWarps * kSpareBytes;
  static constexpr int kOffXScale = kOffScale + kEpiWarps * 2 * kBiasBytes;
  static constexpr int kDynSmem = (kMode == kE4m3 ? kOffXScale + kEpiWarps * 2 * 128 : kOffScale) + 1024;
  // kLora: a group of operands for 16 of the rank, both terms of U, then the up weights of a run each.
  static constexpr int kUnitA = kBM * 32, kUnitB = kBRows * 32;
  static_assert(kStages <= kMaxStages && kStageBytes % 1024 == 0 && kUnitB % 1024 == 0, "stage layout");
};

struct QkvBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
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
// each.  row: this lane's row's index (b H + n's) for head 0 (kDeadRow: past
// the stream's end); head_rows = h N; col: the first column (0, or 64 within a
// d = 128 head row).
template <int D>
__device__ __forceinline__ void store_rows(uint32_t buf, uint16_t* base, uint32_t row, uint32_t head_rows, int col,
                                           int lane) {
  const int ch = lane & 7;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t to = __shfl_sync(0xffffffffu, row, 4 * j + (lane >> 3));
    const uint4 val = ld_shared_v4(staged(buf, 4 * j + (lane >> 3), ch));
    if (to != kDeadRow)
      *reinterpret_cast<uint4*>(base + (static_cast<size_t>(to) + head_rows) * D + col + ch * 8) = val;
  }
}

// Elements near a bf16 midpoint.  The norm kernels' bound on z = (g x) r with
// one correction of r (corrected_r): the squares' sum takes at most 7
// roundings of nonnegative terms (7 u, u = 2^-24), the mean and eps one, which
// r halves (4 u), the correction and its roundings leave 1 u of its own, the
// two products add 1 u each: 7 u, at most 7 fp32 units in the last place.  The
// window takes 8 on either side of the midpoint.
constexpr uint32_t kNearWindow = 16;
constexpr uint32_t kNearFrom = (0x10000u + kNearWindow / 2 - 0x8000u) & 0xFFFFu;
__device__ __forceinline__ bool near_midpoint(float z) {
  return ((__float_as_uint(z) + kNearFrom) & 0xFFFFu) < kNearWindow;
}
// Two at a time: the smaller of the low halves' distances above the window's
// start, per half of m, starting from kNoneNear.
constexpr uint32_t kNoneNear = 0xFFFFFFFFu;
__device__ __forceinline__ void near_pair(float z0, float z1, uint32_t& m) {
  m = __viaddmin_u16x2(__byte_perm(__float_as_uint(z0), __float_as_uint(z1), 0x5410), kNearFrom * 0x10001u, m);
}
__device__ __forceinline__ bool any_near(uint32_t m) {
  return (m & 0xFFFFu) < kNearWindow || (m >> 16) < kNearWindow;
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

// The rare path.  The warp takes each of its rows that has an element near a
// bf16 midpoint (about one a tile) together: the lane that holds the row writes
// its raw values to the warp's spare row; each lane takes D / 32 of them, their
// squares (exact) are summed by error-free additions over the warp, and each
// lane re-rounds its elements that the fp32 path put near a midpoint, from the
// double-float r, and writes its words over the staged q_hat / k_hat row,
// before that is written out.  (Four rows at a time by 8 lanes each took 2500
// cycles a pass at d = 64 and 3700 at d = 128.)
//   todo: rows by head (bit i: lane i's row); at d = 64 head h's staged rows are
//   in buffer h, at d = 128 the head's halves in both.
template <int D, int kHeads>
__device__ __forceinline__ void fix_staged_rows(const unsigned (&todo)[kHeads], const uint32_t (&yb)[kHeads * D / 2],
                                                uint32_t spare, uint32_t hat, const float (&r)[kHeads],
                                                const float* const (&g)[kHeads], int lane) {
  uint64_t left = todo[0];
  if constexpr (kHeads == 2) left |= static_cast<uint64_t>(todo[1]) << 32;
  while (left) {
    const int bit = __ffsll(static_cast<long long>(left)) - 1;
    left &= left - 1;
    const int o = bit & 31, h = kHeads == 2 ? bit >> 5 : 0;
    if (lane == o) {
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        if (h == i) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint32_t* y = yb + i * (D / 2) + 4 * c;
            st_shared_v4(spare + c * 16, y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
    const float ro = __shfl_sync(0xffffffffu, h ? r[kHeads - 1] : r[0], o);
    const float* gv = h ? g[kHeads - 1] : g[0];
    __syncwarp();
    constexpr int kWords = D / 64;  // of a lane: elements 2 kWords lane ..
    uint32_t w[kWords];
    float s = 0.f, c = 0.f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      w[i] = ld_shared_u32(spare + (kWords * lane + i) * 4);
      add_sq_df(w[i], s, c);
    }
    warp_sum_df(s, c);
    float rh, rl;
    rsqrt_mean_eps_df(s, c, 1.f / D, rh, rl);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int e = 2 * (kWords * lane + i);
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x = j ? bf_hi(w[i]) : bf_lo(w[i]);
        const float z = __fmul_rn(__fmul_rn(gv[e + j], x), ro);
        f[j] = near_midpoint(z) ? round_bf16_df(gv[e + j], x, rh, rl) : z;
      }
      const int chunk = e >> 3;  // at d = 128 chunks 8 .. 15 are in the second buffer
      const uint32_t buf = hat + (D == 64 ? h : chunk >> 3) * kStagingBytes;
      st_shared_u32(staged(buf, o, chunk & 7) + (e & 6) * 2, pack_bf16x2(f[0], f[1]));
    }
    __syncwarp();  // the spare row is free again
  }
}

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
  int n_tiles;        // column tiles
  DivU31 by_tiles;    // division by n_tiles
  int tiles;          // all tiles of both streams
  uint16_t* out[3];   // q, k, v: [B, H, N, d]
  uint16_t* hat[2];   // q_hat, k_hat
  float* r[2];        // rq, rk: [B, H, N]
  // kLora: the batch items' adapters (none where outside 0 .. n_adapters - 1),
  // units of 16 of the rank, and whether a stream has adapters.
  const int* index;
  int n_adapters, rank_units;
  bool lora[2];
  bool after_down;  // the launch before this one is lora_down_kernel's
};

// kLora: U [M, 2 * 3 * 16 rank_units] (the high terms of q, k, v, then the low
// terms) and the adapters' up weights [n, 3 H d, rank], image then caption stream.
struct QkvLoraMaps {
  CUtensorMap u[2], up[2];
};

// The runs of consecutive batch items with one adapter among rows m0 .. m1 - 1
// of a stream: next() gives the next one's adapter and its rows lo .. hi - 1 of
// the tile, passing over items without an adapter.  Two items' indexes are on
// their way ahead of the one that is looked at.
struct Runs {
  const int* index;
  int n_adapters, N_s, m0, m1;
  int b, row;      // the next item, and its first row
  int here, then;  // its index, and the next one's
  int adapter, lo, hi;
  __device__ __forceinline__ Runs(const QkvParams& p, int N_s_, int m0_, int m1_)
      : index(p.index), n_adapters(p.n_adapters), N_s(N_s_), m0(m0_), m1(m1_) {
    b = m0 / N_s;
    row = b * N_s;
    here = __ldg(index + b);
    then = row + N_s < m1 ? __ldg(index + b + 1) : 0;
  }
  __device__ __forceinline__ void step() {
    ++b;
    row += N_s;
    here = then;
    if (row + N_s < m1) then = __ldg(index + b + 1);  // row + N_s < m1 <= B N_s: item b + 1 exists
  }
  __device__ __forceinline__ bool next() {
    while (row < m1) {
      adapter = here;
      lo = max(row, m0) - m0;
      do step();
      while (row < m1 && here == adapter);
      hi = min(row, m1) - m0;
      if (adapter >= 0 && adapter < n_adapters) return true;
    }
    return false;
  }
};
// Rows lo .. hi - 1 of words of 32 rows: the bits of word w.
__device__ __forceinline__ uint32_t rows_of_word(int lo, int hi, int w) {
  const int from = max(lo - 32 * w, 0), to = min(hi - 32 * w, 32);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(from), "r"(max(to - from, 0)));
  return m;
}
// The q, k, v parts that columns n0 .. n0 + cols - 1 meet.
__device__ __forceinline__ void parts_of(int n0, int cols, int hd, int& first, int& last) {
  first = n0 / hd;
  last = min((n0 + cols - 1) / hd, 2);
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
// consecutive rows of one item (contig; n0 and bh0 = b H of the first row),
// else the row-by-row stores of store_rows (row: this lane's, for head 0).
struct RowsOut {
  bool contig;
  int n0, bh0;
  uint32_t row;
};
// Writes out the buffers whose bit in `which` is set, after the lanes have
// staged them: where buffer i goes comes from to(i, map, base, head, column).
template <int D, int kBufs, typename To>
__device__ __forceinline__ void emit_rows(uint32_t buf, unsigned which, const RowsOut& ro, uint32_t N, To to,
                                          int lane) {
  if (ro.contig) fence_proxy_async_smem();  // this lane's staged writes, to the TMA unit
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kBufs; ++i) {
    if ((which >> i) & 1u) {
      const CUtensorMap* map;
      uint16_t* base;
      int h, col;
      to(i, map, base, h, col);
      if (!ro.contig)
        store_rows<D>(buf + i * kStagingBytes, base, ro.row, static_cast<uint32_t>(h) * N, col, lane);
      else if (lane == 0)
        tma_store_3d_s(map, buf + i * kStagingBytes, col, ro.n0, ro.bh0 + h);
    }
  }
  if (ro.contig && lane == 0) bulk_commit_group();
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
//
// r is what is kept; rc, for q_hat / k_hat, takes one Newton step more: r (1 +
// t / 2), t = 1 - m r^2 of order 2^-22, is the root of m to 2^-44 before its
// rounding.
template <int D>
__device__ __forceinline__ void row_rsqrt(const uint32_t* yb, float& r, float& rc) {
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
  const float m = __fadd_rn(__fmul_rn(blk[0], 1.f / D), kEps);
  r = rsqrtf(m);
  const float q = __fmul_rn(m, r);  // 1 - m r^2 = 1 - q r + (q - m r) r
  const float t = __fmaf_rn(__fmaf_rn(-m, r, q), r, __fmaf_rn(-q, r, 1.f));
  rc = __fmaf_rn(__fmul_rn(0.5f, r), t, r);
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
      // Unpacked by other instructions than in row_rsqrt, so that the compiler does not keep the row
      // unpacked in between (128 registers, and spills around the rare path).
      const uint32_t yv = y[4 * c + i];
      const float lo = __uint_as_float(__byte_perm(yv, 0u, 0x1044)), hi = __uint_as_float(__byte_perm(yv, 0u, 0x3244));
      float z0, z1;
      f2_split(f2_mul(f2_mul(gv[i], f2_make(lo, hi)), r2), z0, z1);
      near_pair(z0, z1, near);
      w[i] = pack_bf16x2(z0, z1);
    }
    st_shared_v4(staged(buf, lane, c), w[0], w[1], w[2], w[3]);
  }
}

// The warp's 32 token rows of a tile, 64 kHalves columns from taddr (this
// lane's row) and col0 on.  bias, wscale: those columns' in shared memory; sx:
// the row's scale (kE4m3).  The accumulator is handed back (acc_empty) once
// its values are in registers.
template <int D, int kMode, bool kPair, int kHalves>
__device__ __forceinline__ void qkv_emit(uint32_t taddr, uint64_t* acc_empty, int col0, bool live, size_t row,
                                         const RowsOut& ro, uint32_t stg, uint32_t bias, float sx, uint32_t wscale,
                                         uint32_t spare, const QkvParams& p, const QkvOutMaps& om,
                                         const QkvBars& bars, int lane) {
  constexpr int kHeads = kHalves * 64 / D;
  const int hd = p.H * D;
  const uint64_t sx2 = f2_make(sx, sx);
  // Y = bf16(acc + bias), 16 columns at a time (packed pairs); the next 16 are on their way meanwhile.
  uint32_t yb[kHalves * 32];
  uint32_t acc[2][16];
  tmem_ld16(taddr, acc[0]);
#pragma unroll
  for (int c16 = 0; c16 < 4 * kHalves; ++c16) {
    tmem_wait_ld();
    if (c16 + 1 < 4 * kHalves) {
      tmem_ld16(taddr + (c16 + 1) * 16, acc[(c16 + 1) & 1]);
    } else {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_to<kPair>(acc_empty);
    }
    const uint32_t(&v)[16] = acc[c16 & 1];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const float4 bv = ld_shared_f4(bias + (c16 * 16 + e) * 4);
      uint64_t y0 = f2_make(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
      uint64_t y1 = f2_make(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
      if constexpr (kMode == kE4m3) {
        const float4 sv = ld_shared_f4(wscale + (c16 * 16 + e) * 4);
        y0 = f2_fma(f2_mul(y0, sx2), f2_make(sv.x, sv.y), f2_make(bv.x, bv.y));
        y1 = f2_fma(f2_mul(y1, sx2), f2_make(sv.z, sv.w), f2_make(bv.z, bv.w));
      } else {
        y0 = f2_add(y0, f2_make(bv.x, bv.y));
        y1 = f2_add(y1, f2_make(bv.z, bv.w));
      }
      float a0, a1, a2, a3;
      f2_split(y0, a0, a1);
      f2_split(y1, a2, a3);
      yb[c16 * 8 + e / 2] = pack_bf16x2(a0, a1);
      yb[c16 * 8 + e / 2 + 1] = pack_bf16x2(a2, a3);
    }
  }
  if (col0 >= 3 * hd) return;  // past the last head
  int which[kHeads], head[kHeads];  // 0 q, 1 k, 2 v (3: past the last head)
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    which[i] = (col0 + i * D >= hd) + (col0 + i * D >= 2 * hd) + (col0 + i * D >= 3 * hd);
    head[i] = (col0 + i * D - which[i] * hd) / D;
  }
  auto part = [&](int i) { return D == 64 ? which[i < kHeads ? i : 0] : which[0]; };  // of half i
  auto to_raw = [&](int i, const CUtensorMap*& map, uint16_t*& base, int& h, int& col) {
    map = out_map(om, part(i));
    base = out_of(p, part(i));
    h = head[D == 64 ? i : 0];
    col = D == 64 ? 0 : i * 64;
  };
  auto to_hat = [&](int i, const CUtensorMap*& map, uint16_t*& base, int& h, int& col) {
    map = hat_map(om, part(i));
    base = hat_of(p, part(i));
    h = head[D == 64 ? i : 0];
    col = D == 64 ? 0 : i * 64;
  };
  unsigned raw = 0, normed = 0;  // halves to be written, and those with a norm
#pragma unroll
  for (int i = 0; i < kHalves; ++i) {
    raw |= part(i) < 3 ? 1u << i : 0u;
    normed |= part(i) < 2 ? 1u << i : 0u;
  }
  staging_free(lane);
#pragma unroll
  for (int i = 0; i < kHalves; ++i) stage_row(stg + i * kStagingBytes, yb + i * 32, lane);
  emit_rows<D, kHalves>(stg, raw, ro, p.N, to_raw, lane);
  if (normed == 0) {
    __syncwarp();
    return;
  }
  float r[kHeads], rc[kHeads];
  const float* g[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    row_rsqrt<D>(yb + i * (D / 2), r[i], rc[i]);
    g[i] = which[i] == 0 ? bars.gq : bars.gk;
  }
  staging_free(lane);  // (and, after row-by-row stores, their reads: a barrier)
  unsigned todo[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    uint32_t near = kNoneNear;
    if (which[i] < 2) {
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        stage_hat_row(stg + (i + j) * kStagingBytes, yb + (i * D / 64 + j) * 32, smem_u32(g[i] + j * 64), rc[i], near,
                      lane);
      if (live) r_of(p, which[i])[row + static_cast<size_t>(head[i]) * p.N] = r[i];
    }
    todo[i] = __ballot_sync(0xffffffffu, any_near(near) && live);
  }
  unsigned any = todo[0];
  if constexpr (kHeads == 2) any |= todo[1];
  if (any) {
    __syncwarp();
    fix_staged_rows<D, kHeads>(todo, yb, spare, stg, rc, g, lane);
  }
  emit_rows<D, kHalves>(stg, normed, ro, p.N, to_hat, lane);
  __syncwarp();
}

template <int D, int kMode, bool kPair>
__global__ void __launch_bounds__(QkvCfg<D, kMode, kPair>::kThreads, 1)
    qkv_norm_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_w0,
                    const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ QkvOutMaps om, const __grid_constant__ QkvLoraMaps lm,
                    const __grid_constant__ QkvParams p, const float* __restrict__ gq,
                    const float* __restrict__ gk, uint32_t* dev_err) {
  using Cfg = QkvCfg<D, kMode, kPair>;
  constexpr int kStages = Cfg::kStages, kCtas = Cfg::kCtas, kCols = Cfg::kCols;
  constexpr int kRows = kCtas * kBM;                                  // token rows of a tile
  constexpr int kStepK = kMode == kE4m3 ? kStepBytes : kStepBytes / 2;  // values of a row in a K step
  constexpr int kWarpProd = Cfg::kWarpProd, kWarpIssue = Cfg::kWarpIssue;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) QkvBars bars;
  uint8_t* sm = align1024(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* ab = &bars.abort;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;  // within the pair
  const int first_tile = blockIdx.x / kCtas, tile_step = gridDim.x / kCtas;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], kCtas * Cfg::kEpiWarps);
    }
    mbar_init(&bars.mma_done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpIssue) {
    tmem_alloc<kCtas>(&bars.tmem_base, Cfg::kTmemCols);
    tmem_relinquish<kCtas>();
  }
  // The previous grid's writes are visible from here on.  With adapters the
  // previous grid is lora_down_kernel, which lets this one start once what came
  // before itself is complete: only the loads of U wait for it (the producer).
  if (kMode != kLora || !p.after_down) griddep_wait();
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    bars.gq[i] = gq[i];
    bars.gk[i] = gk[i];
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int ksteps = (p.C + kStepK - 1) / kStepK;

  if (warp >= Cfg::kEpiWarps) {
  if constexpr (kPair) setmaxnreg_dec<QkvRegs<D>::kOther>();
  if (warp == kWarpProd) {
    if (lane == 0) {
      tma_prefetch_desc(&map_x0);
      tma_prefetch_desc(&map_w0);
      tma_prefetch_desc(&map_x1);
      tma_prefetch_desc(&map_w1);
      int it = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < p.tiles; t += tile_step) {
        const int si = t >= p.s[1].tile0 ? 1 : 0;
        const int tl = t - (si ? p.s[1].tile0 : p.s[0].tile0);
        const int mt = tl / p.n_tiles, nt = tl - mt * p.n_tiles;
        const CUtensorMap* mx = si ? &map_x1 : &map_x0;
        const CUtensorMap* mw = si ? &map_w1 : &map_w0;
        for (int kb = 0; kb < ksteps; ++kb) {
          const int s = it % kStages;
          if (it >= kStages && !(ok = mbar_wait(&bars.empty[s], ((it / kStages) - 1) & 1, ab, dev_err))) break;
          uint8_t* st = sm + s * Cfg::kStageBytes;
          const uint32_t full = pair_bar<kPair>(&bars.full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], kCtas * Cfg::kStageBytes);
          tma_load_2d_to<kPair>(st, mx, full, kb * kStepK, mt * kRows + rank * kBM);
          tma_load_2d_to<kPair>(st + kATile, mw, full, kb * kStepK, nt * kCols + rank * Cfg::kBRows);
          ++it;
        }
        if constexpr (kMode == kLora) {
          if (!ok || !(si ? p.lora[1] : p.lora[0])) continue;
          const int N_s = si ? p.s[1].N_s : p.s[0].N_s, M = si ? p.s[1].M : p.s[0].M;
          const int m0 = mt * kRows, m1 = min(m0 + kRows, M), n0 = nt * kCols, hd = p.H * D;
          const CUtensorMap* mu = si ? &lm.u[1] : &lm.u[0];
          const CUtensorMap* mup = si ? &lm.up[1] : &lm.up[0];
          int p0, p1, used = 0;  // bytes of the open stage (0: none open)
          parts_of(n0, kCols, hd, p0, p1);
          bool waited = false;
          // The stage is closed by its one arrival; until then each group's bytes are added to what it expects.
          auto close = [&] {
            if (rank == 0) mbar_arrive(&bars.full[it % kStages]);
            used = 0;
            ++it;
          };
          for (int part = p0; ok && part <= p1; ++part) {
            const int c0 = max(part * hd, n0), width = min((part + 1) * hd, n0 + kCols) - c0;
            for (int kc = 0; ok && kc < p.rank_units; ++kc) {
              Runs runs(p, N_s, m0, m1);
              bool more = runs.next();
              while (ok && more) {
                if (used + 2 * Cfg::kUnitA + Cfg::kUnitB > Cfg::kStageBytes) close();
                const int s = it % kStages;
                if (used == 0) {
                  if (it >= kStages && !(ok = mbar_wait(&bars.empty[s], ((it / kStages) - 1) & 1, ab, dev_err))) break;
                  if (!waited) griddep_wait();  // U is there
                  waited = true;
                }
                const uint32_t full = pair_bar<kPair>(&bars.full[s]);
                uint8_t* st = sm + s * Cfg::kStageBytes;
                const int col = (part * p.rank_units + kc) * 16;
                if (rank == 0) mbar_expect_tx(&bars.full[s], kCtas * 2 * Cfg::kUnitA);
                tma_load_2d_to<kPair>(st + used, mu, full, col, m0 + rank * kBM);
                tma_load_2d_to<kPair>(st + used + Cfg::kUnitA, mu, full, col + 3 * 16 * p.rank_units, m0 + rank * kBM);
                used += 2 * Cfg::kUnitA;
                do {
                  if (rank == 0) mbar_expect_tx(&bars.full[s], kCtas * Cfg::kUnitB);
                  tma_load_3d_to<kPair>(st + used, mup, full, kc * 16, c0 + rank * (width / kCtas), runs.adapter);
                  used += Cfg::kUnitB;
                  more = runs.next();
                } while (more && used + Cfg::kUnitB <= Cfg::kStageBytes);
              }
            }
          }
          if (used > 0) close();
        }
      }
      if constexpr (kMode == kLora) griddep_wait();  // this grid ends after the one before it
      if (*ab) {
        // Aborted: the copies in flight land before the CTA exits.  The second
        // CTA's signal the first one's barriers: it waits out the limit.
        for (int i = (it > kStages ? it - kStages : 0); i < it; ++i)
          mbar_wait_drain(&bars.full[i % kStages], (i / kStages) & 1);
      }
    }
  } else if (warp == kWarpIssue) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc =
          kMode == kE4m3 ? idesc_e4m3_f32(kRows, kCols) : idesc_bf16_f32(kRows, kCols, false, false);
      int it = 0, lt = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < p.tiles; t += tile_step, ++lt) {
        const int abuf = lt & 1;
        if (lt >= 2 && !(ok = mbar_wait(&bars.acc_empty[abuf], ((lt >> 1) - 1) & 1, ab, dev_err))) break;
        tc_fence_after();
        const uint32_t acc = tmem + abuf * kCols;
        for (int kb = 0; kb < ksteps; ++kb, ++it) {
          const int s = it % kStages;
          if (!(ok = mbar_wait(&bars.full[s], (it / kStages) & 1, ab, dev_err))) break;
          tc_fence_after();
          const uint32_t st = smem_u32(sm + s * Cfg::kStageBytes);
          const uint64_t a = sdesc_sw128(st, 16, 1024), b = sdesc_sw128(st + kATile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kStepBytes / 32; ++kk) {  // 32 bytes of each row: 16 bf16 or 32 e4m3 values
            const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
            if constexpr (kMode == kE4m3)
              umma_f8_ss<kCtas>(acc, desc_add(a, kk * 32), desc_add(b, kk * 32), idesc, add);
            else
              umma_bf16_ss<kCtas>(acc, desc_add(a, kk * 32), desc_add(b, kk * 32), idesc, add);
          }
          umma_commit_to<kPair>(&bars.empty[s]);
        }
        if constexpr (kMode == kLora) {
          const int si = t >= p.s[1].tile0 ? 1 : 0;
          if (ok && (si ? p.lora[1] : p.lora[0])) {
            const int tl = t - (si ? p.s[1].tile0 : p.s[0].tile0);
            const int mt = tl / p.n_tiles, n0 = (tl - mt * p.n_tiles) * kCols;
            const int N_s = si ? p.s[1].N_s : p.s[0].N_s, M = si ? p.s[1].M : p.s[0].M;
            const int m0 = mt * kRows, m1 = min(m0 + kRows, M), hd = p.H * D;
            int p0, p1, used = 0;  // as the producer counts
            parts_of(n0, kCols, hd, p0, p1);
            auto close = [&] {
              umma_commit_to<kPair>(&bars.empty[it % kStages]);
              used = 0;
              ++it;
            };
            for (int part = p0; ok && part <= p1; ++part) {
              const int c0 = max(part * hd, n0) - n0, c1 = min((part + 1) * hd, n0 + kCols) - n0;
              const uint32_t desc = idesc_bf16_f32(kRows, c1 - c0, false, false);
              for (int kc = 0; ok && kc < p.rank_units; ++kc) {
                Runs runs(p, N_s, m0, m1);
                bool more = runs.next();
                while (ok && more) {
                  if (used + 2 * Cfg::kUnitA + Cfg::kUnitB > Cfg::kStageBytes) close();
                  const int s = it % kStages;
                  if (used == 0) {
                    if (!(ok = mbar_wait(&bars.full[s], (it / kStages) & 1, ab, dev_err))) break;
                    tc_fence_after();
                  }
                  const uint32_t st = smem_u32(sm + s * Cfg::kStageBytes);
                  const uint64_t u_hi = sdesc_sw32_kmajor(st + used, 256);
                  const uint64_t u_lo = sdesc_sw32_kmajor(st + used + Cfg::kUnitA, 256);
                  used += 2 * Cfg::kUnitA;
                  do {
                    uint32_t off[4 * kCtas];  // the lanes (rows) that the run does not hold
#pragma unroll
                    for (int w = 0; w < 4 * kCtas; ++w) off[w] = ~rows_of_word(runs.lo, runs.hi, w);
                    const uint64_t up = sdesc_sw32_kmajor(st + used, 256);
                    umma_bf16_ss_lanes(acc + c0, u_hi, up, desc, off, 1u);
                    umma_bf16_ss_lanes(acc + c0, u_lo, up, desc, off, 1u);
                    used += Cfg::kUnitB;
                    more = runs.next();
                  } while (more && used + Cfg::kUnitB <= Cfg::kStageBytes);
                }
              }
            }
            if (ok && used > 0) close();
          }
        }
        if (ok) umma_commit_to<kPair>(&bars.acc_full[abuf]);
      }
      // Every MMA this thread issued has completed once this barrier flips.
      umma_commit<kCtas>(&bars.mma_done);
      mbar_wait_drain(&bars.mma_done, 0);
    }
  }
  } else {
    if constexpr (kPair) setmaxnreg_inc<QkvRegs<D>::kEpi>();
    // Warp w: the TMEM lanes of warp w % 4, and kWarpCols columns of the tile from kWarpCols (w / 4) on.
    const int lg = warp & 3, wcol = (warp >> 2) * Cfg::kWarpCols;
    const uint32_t stg = smem_u32(sm + Cfg::kOffStaging + warp * Cfg::kStaging);
    const uint32_t bias_w = smem_u32(sm + Cfg::kOffBias + warp * 2 * Cfg::kBiasBytes);
    const uint32_t wscale_w = smem_u32(sm + Cfg::kOffScale + warp * 2 * Cfg::kBiasBytes);  // kE4m3
    const uint32_t xscale_w = smem_u32(sm + Cfg::kOffXScale + warp * 256);                 // kE4m3
    const uint32_t spare_w = smem_u32(sm + Cfg::kOffSpare + warp * Cfg::kSpareBytes);
    const uint32_t lane_base = static_cast<uint32_t>(lg * 32) << 16;
    const int hd3 = 3 * p.H * D;
    // What the epilogue of a tile reads from global memory, copied to this warp's slices one tile ahead
    // (its latency, some 700 cycles each, is not met): the bias of the warp's columns (zero past 3 H d, or
    // without a bias); kE4m3: their scales, and those of its rows.
    auto fetch = [&](int t, int buf) {
      const QkvStream S = stream_of(p, t >= p.s[1].tile0 ? 1 : 0);
      const int tl = t - S.tile0, mt = static_cast<int>(p.by_tiles.div(tl));
      const int col = (tl - mt * p.n_tiles) * kCols + wcol + lane * 4;
      if (lane * 4 < Cfg::kWarpCols) {
        const uint32_t to = bias_w + buf * Cfg::kBiasBytes + lane * 16;
        if (S.bias && col < hd3)
          cp_async16(to, S.bias + col);
        else
          st_shared_v4(to, 0u, 0u, 0u, 0u);
        if constexpr (kMode == kE4m3) {
          const uint32_t ws = wscale_w + buf * Cfg::kBiasBytes + lane * 16;
          if (col < hd3)
            cp_async16(ws, S.sw + col);
          else
            st_shared_v4(ws, 0u, 0u, 0u, 0u);
        }
      }
      if constexpr (kMode == kE4m3) {
        const int m = mt * kRows + rank * kBM + lg * 32 + lane;
        const uint32_t xs = xscale_w + buf * 128 + lane * 4;
        if (m < S.M)
          cp_async4(xs, S.sx + m);
        else
          st_shared_u32(xs, 0u);
      }
      cp_async_commit();
    };
    int lt = 0;
    if (first_tile < p.tiles) fetch(first_tile, 0);
    for (int t = first_tile; t < p.tiles; t += tile_step, ++lt) {
      const int abuf = lt & 1;
      const QkvStream S = stream_of(p, t >= p.s[1].tile0 ? 1 : 0);
      const int tl = t - S.tile0;
      const int mt = static_cast<int>(p.by_tiles.div(tl)), nt = tl - mt * p.n_tiles;
      const int col0 = nt * kCols + wcol;  // the warp's first column in Y
      const int m = mt * kRows + rank * kBM + lg * 32 + lane;
      const bool live = m < S.M;
      const int bi = live ? m / S.N_s : 0;
      const int n = live ? S.row0 + (m - bi * S.N_s) : 0;
      const size_t row = static_cast<size_t>(bi) * p.H * p.N + n;  // < B H N < 2^31 / d
      const uint32_t row32 = live ? static_cast<uint32_t>(row) : kDeadRow;
      RowsOut ro;
      {
        const uint32_t first = __shfl_sync(0xffffffffu, row32, 0), last = __shfl_sync(0xffffffffu, row32, 31);
        // Of one item: with one head and one stream the next item's rows follow on.
        const int b0 = __shfl_sync(0xffffffffu, bi, 0), b31 = __shfl_sync(0xffffffffu, bi, 31);
        ro.contig = first != kDeadRow && last != kDeadRow && last - first == 31u && b0 == b31;
        ro.n0 = __shfl_sync(0xffffffffu, n, 0);
        ro.bh0 = b0 * p.H;
        ro.row = row32;
      }
      cp_async_wait_all();
      const bool ok = mbar_wait(&bars.acc_full[abuf], (lt >> 1) & 1, ab, dev_err);
      if (!__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      tc_fence_after();
      if (t + tile_step < p.tiles) fetch(t + tile_step, abuf ^ 1);
      float sx = 0.f;
      if constexpr (kMode == kE4m3) sx = __uint_as_float(ld_shared_u32(xscale_w + abuf * 128 + lane * 4));
      qkv_emit<D, kMode, kPair, Cfg::kWarpCols / 64>(tmem + lane_base + abuf * kCols + wcol, &bars.acc_empty[abuf],
                                                     col0, live, row, ro, stg, bias_w + abuf * Cfg::kBiasBytes, sx,
                                                     wscale_w + abuf * Cfg::kBiasBytes, spare_w, p, om, bars, lane);
    }
    if (lane == 0) bulk_wait_group0();  // this warp's tile stores are complete
  }
  tc_fence_before();
  __syncthreads();
  // Neither CTA of a pair leaves, or frees its TMEM, while the other may still use its memory.
  if constexpr (kPair) cluster_sync();
  if (warp == kWarpIssue) {
    tc_fence_after();
    tmem_dealloc<kCtas>(tmem, Cfg::kTmemCols);
  }
}

// How many pairs of a kernel the current device runs at once (a pair beyond
// that number would start when the others have finished), after a check of the
// registers its setmaxnreg split was sized for; asked once per device and
// kernel (`known`: the kernel's own, by device, 0 where not asked yet).
template <typename K>
cudaError_t resident_pairs(K kernel, int threads, int smem, int regs, std::atomic<int>* known, int devices,
                           int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool slot = dev >= 0 && dev < devices;
  *pairs = slot ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*pairs > 0) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if ((fa.numRegs + 7) / 8 * 8 != regs) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*pairs < 1) return cudaErrorInvalidConfiguration;
  if (slot) known[dev].store(*pairs, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int D, int kMode, bool kPair>
cudaError_t launch_qkv_kernel(const CUtensorMap (&maps)[4], const QkvOutMaps& om, const QkvLoraMaps& lm,
                              const QkvParams& p, const float* gq, const float* gk, uint32_t* dev_err,
                              cudaStream_t st) {
  using Cfg = QkvCfg<D, kMode, kPair>;
  auto kernel = qkv_norm_kernel<D, kMode, kPair>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kDynSmem);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  int groups = sms > Cfg::kCtas ? sms / Cfg::kCtas : 1;
  if constexpr (kPair) {
    static std::atomic<int> known[64];
    int fit = 0;
    e = resident_pairs(kernel, Cfg::kThreads, Cfg::kDynSmem, QkvRegs<D>::kLaunch, known, 64, &fit);
    if (e != cudaSuccess) return e;
    if (fit < groups) groups = fit;
  }
  const int grid = (p.tiles < groups ? p.tiles : groups) * Cfg::kCtas;
  return launch_pdl_cluster(kernel, Cfg::kCtas, dim3(grid), dim3(Cfg::kThreads), Cfg::kDynSmem, st, maps[0], maps[1],
                            maps[2], maps[3], om, lm, p, gq, gk, dev_err);
}

}  // namespace

// One form of the projection (each is compiled in a file of its own).
template <int kMode>
cudaError_t launch_qkv_form(const CUtensorMap (&maps)[4], const CUtensorMap (&out_maps)[5], const QkvLaunch& a,
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
  const bool pair = a.pair;
  const int rows = pair ? 2 * kBM : kBM, cols = kQkvCols(a.d, pair);
  QkvParams p;
  p.H = a.H;
  p.C = a.C;
  p.N = a.N;
  p.n_tiles = (3 * a.H * a.d + cols - 1) / cols;
  p.by_tiles = make_div_u31(p.n_tiles);
  int tile0 = 0;
  for (int i = 0; i < 2; ++i) {
    p.s[i].M = a.M[i];
    p.s[i].N_s = a.N_s[i];
    p.s[i].row0 = a.row0[i];
    p.s[i].tile0 = tile0;
    p.s[i].bias = a.bias[i];
    p.s[i].sx = a.sx[i];
    p.s[i].sw = a.sw[i];
    tile0 += ((a.M[i] + rows - 1) / rows) * p.n_tiles;
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
  p.after_down = p.lora[0] || p.lora[1];
  p.rank_units = lora ? (lora->rank + 15) / 16 : 0;
  if (p.tiles == 0) return cudaSuccess;
  if (a.d == 64)
    return pair ? launch_qkv_kernel<64, kMode, true>(maps, om, lm, p, a.gq, a.gk, dev_err, st)
                : launch_qkv_kernel<64, kMode, false>(maps, om, lm, p, a.gq, a.gk, dev_err, st);
  return pair ? launch_qkv_kernel<128, kMode, true>(maps, om, lm, p, a.gq, a.gk, dev_err, st)
              : launch_qkv_kernel<128, kMode, false>(maps, om, lm, p, a.gq, a.gk, dev_err, st);
}

}  // namespace jattn
