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
//   epilogue    a head's columns of 16 or 32 token rows a warp: their values out
//               of TMEM, + bias (the columns', copied to shared memory while the
//               products run), rounded to bf16 (the projection's output) for q /
//               k / v; for q and k the row's RMSNorm from those bf16 values,
//               q_hat / k_hat and r.  Four lanes share a row, 16 neighbouring
//               columns of each 64 a lane, and write it straight from registers
//               as whole 128-byte lines: the weights' rows are loaded in an order
//               that leaves each lane's columns next to each other (qkv_emit).
// Heads past 3 H in the last column tile, and token rows past the stream's
// end in its last row tile, read the TMA's zero fill and are not stored.
//
// What bounds it (512 px, C = 768, 12 heads of 64; 52 us from bf16, 39 us from
// e4m3; 768 px, C = 2048, 16 heads of 128; 141 and 87 us): the epilogue beside
// the products.  The products alone take 38, 24, 120 and 66 us (the rate of
// cuBLAS), the epilogue with one K step 30, 34, 43 and 50, of which 5 to 10 for
// the stores.  From e4m3 at 512 px it is the epilogue's latency, with the issue slots
// 45 % and the tensor pipe 37 % busy: all 16 warps are in one phase of one tile (some
// 930 instructions a warp for 32 rows of 64 columns; of 9.7 cycles between two of
// them 2.6 are spent at the tile's barrier and 1.9 for TMEM and memory).  Else it is
// the loads' latency beside the stores (a ring of 128 KB 56 and 147 us from bf16, of
// 160 KB 52.7 and 141) and shared memory's bandwidth, of which the products take
// most: rows staged there and written out by TMA stores, with 128 KB left for the
// ring, took 57, 39, 151 and 92 us; gains, biases and scales read without a gap every
// 16 columns (two-way bank conflicts), and anew for each row, 5 us more from e4m3 at
// 512 px.
//
// The same kernel takes two other forms of the products (template kMode):
//   kE4m3  X and W in e4m3 with fp32 scales of their rows: a K step of 128
//          values in the same 128-byte rows, kind::f8f6f4 products, and
//          Y = bf16(sx sw acc + bias).
//   kLora  low-rank adapters of the batch items' own beside the shared
//          weights: Y = bf16(X W^T + U B^T + bias), U = scale X A^T (one
//          launch of lora_down_kernel before, kept as three bf16 terms) as
//          further K steps of 16 into the same accumulator.  A row tile that
//          holds items with different adapters takes each adapter in turn, with
//          the other rows' lanes disabled in the MMA, so that no copy of U is
//          needed (a warp of its own lists the next tile's adapters and their
//          rows); a column tile over a q / k / v boundary
//          takes each part with its own columns of U.  A ring stage holds, for
//          16 of the rank at a time, the terms of U (12 KB) and the B rows of
//          as many adapters as fit (2 or 4 KB each): two such groups when there
//          is one, and U loaded once for 5 or 6 when there are many.
//
// Correct rounding: the sum of the d squares is a balanced tree over a lane's
// columns and the four lanes (at most 7 roundings per term, within the 8 that
// the rounding window of the norm kernels allows for), and elements in the
// bf16-midpoint window are re-rounded from a double-float r.
#pragma once
#include <atomic>

#include <cuda_bf16.h>

#include "jattn_internal.h"
#include "sm103_ptx.cuh"
#include "bf16_round.cuh"
#include "fastdiv.cuh"
#include "ring.cuh"

namespace jattn {
namespace {

enum QkvMode { kBf16 = 0, kE4m3 = 1, kLora = 2 };

constexpr int kBM = 128;                            // token rows of one CTA
constexpr int kStepBytes = 128;                     // of each row in a K step
constexpr int kATile = kBM * kStepBytes;            // 16 KB
constexpr uint32_t kDeadRow = 0xFFFFFFFFu;
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 8;

// The adapters that rows m0 .. m1 - 1 of a stream (one row tile) have, and each
// one's rows of the tile (bit i of rows[g][w]: row 32 w + i), wherever its items
// lie among them; in the order of their first rows.
template <int kRows>
struct Groups {
  int count;
  int adapter[kRows];
  uint32_t rows[kRows][kRows / 32];
};

// Epilogue warps, then the TMA producer and the MMA issuer.  Warp w reads the TMEM
// lanes (rows) of warp w % 4, a head's columns of 16 rows or (kHalves = 2) of 32.
// kPair: registers per thread (setmaxnreg).  Each SM sub-partition holds the
// epilogue warps w with one w % 4 and one other warp, and an increase draws only
// on the registers those were launched with, so 4 kEpi + kOther must be at most 5
// times the launch count (allocated by eights).  The launcher refuses any build
// whose register count differs (fits: used registers against the count that a form
// is launched with, 0 for a form without a split).
struct QkvRegs {
  static constexpr int kLaunch = 96, kEpi = 104, kOther = 64;
  static_assert(4 * kEpi + kOther == 5 * kLaunch, "projection register split");
  static constexpr bool fits(int used, int launch) { return launch == 0 || (used + 7) / 8 * 8 == launch; }
};

template <int D, int kMode, bool kPair>
struct QkvCfg {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kCols = kQkvCols(D, kPair);       // of a tile
  static constexpr int kBRows = kQkvWRows(D, kPair);     // weight rows that a CTA loads
  static constexpr int kEpiWarps = kPair ? 16 : 8;
  // Not with adapters, whose producer and issuer have more to keep (512 px 67.0 us without the split, 67.9 with).
  static constexpr bool kSplitRegs = kPair && kMode != kLora;
  static constexpr int kLaunchRegs = kSplitRegs ? QkvRegs::kLaunch : 0;
  static constexpr int kGroupWarps = kEpiWarps * D / kCols;  // that share a head's columns
  static constexpr int kHalves = 8 / kGroupWarps;
  static constexpr int kWarpProd = kEpiWarps, kWarpIssue = kEpiWarps + 1;
  static constexpr int kWarpGroups = kEpiWarps + 2;  // kLora
  static constexpr int kThreads = 32 * (kEpiWarps + (kPair ? 4 : kMode == kLora ? 3 : 2));  // kPair: one or two idle
  static constexpr int kStageBytes = kATile + kBRows * kStepBytes;
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr int kTmemCols = 2 * kCols;
  static constexpr int kColBytes = kCols * 5;            // the bias of a tile's columns, by col_offset
  static constexpr int kOffBias = kStages * kStageBytes;  // two tiles'
  // kE4m3: the scales of the columns, likewise, and of each warp's 32 rows.
  static constexpr int kOffScale = kOffBias + 2 * kColBytes;
  static constexpr int kOffXScale = kOffScale + 2 * kColBytes;
  static constexpr int kOffGroups = kOffScale;  // kLora: two tiles'
  static constexpr int kDynSmem = (kMode == kE4m3   ? kOffXScale + kEpiWarps * 2 * 128
                                   : kMode == kLora ? kOffGroups + 2 * static_cast<int>(sizeof(Groups<kCtas * kBM>))
                                                    : kOffScale) +
                                  1024;
  // kLora: a group of operands for 16 of the rank, the terms of U, then the up weights of an adapter each.
  static constexpr int kTermU = kBM * 32, kUnitU = 3 * kTermU, kUnitB = kBRows * 32;
  static_assert(kStages <= kMaxStages && kStageBytes % 1024 == 0 && kUnitB % 1024 == 0, "stage layout");
};

struct QkvBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done;
  uint64_t groups_full[2], groups_empty[2];  // kLora
  uint32_t tmem_base;
  int abort;
  __align__(16) float gq[160];  // by col_offset
  __align__(16) float gk[160];
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

// 16 consecutive columns of a row, one 32-byte store when the outputs are so
// aligned (wide).  Else two of 16 bytes, with kTurn the upper half first in every other
// lane: the lanes whose halves meet in a 32-byte sector then write them at once.
template <bool kTurn>
__device__ __forceinline__ void store_cols16(uint16_t* to, const uint32_t* w, bool wide, int lane) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* half = reinterpret_cast<uint4*>(to);
    const uint4 lo = make_uint4(w[0], w[1], w[2], w[3]), hi = make_uint4(w[4], w[5], w[6], w[7]);
    const bool turn = kTurn && (lane & 1) == 0;
    half[turn ? 1 : 0] = turn ? hi : lo;
    half[turn ? 0 : 1] = turn ? lo : hi;
  }
}
// All `threads` threads of a named barrier: whether ok holds for every one.
__device__ __forceinline__ bool barrier_all(int id, int threads, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return all != 0;
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

// Floats by column in shared memory: 16 bytes left free after each 16 columns, so
// that four lanes reading 16 columns apart meet different banks.
__device__ __forceinline__ constexpr uint32_t col_offset(uint32_t col) { return col * 4 + col / 16 * 16; }

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
  int whole;          // tiles of both streams that are taken whole
  int parts_log;      // those after them are taken in 1 << parts_log parts of their columns
  int items;          // whole tiles and parts
  uint16_t* out[3];   // q, k, v: [B, H, N, d]
  uint16_t* hat[2];   // q_hat, k_hat
  float* r[2];        // rq, rk: [B, H, N]
  bool wide;          // q, k, v, q_hat, k_hat at 32-byte boundaries
  // kLora: the batch items' adapters (none where outside 0 .. n_adapters - 1),
  // units of 16 of the rank, and whether a stream has adapters.
  const int* index;
  int n_adapters, rank_units;
  bool lora[2];
  bool after_down;  // the launch before this one is lora_down_kernel's
};

// kLora: U [M, 3 rank_units, 3, 16] (for each 16 of the rank of q, k and v the first,
// second and third terms) and the adapters' up weights, image then caption stream.
struct QkvLoraMaps {
  CUtensorMap u[2], up[2];
};

// Rows lo .. hi - 1 of words of 32 rows: the bits of word w.
__device__ __forceinline__ uint32_t rows_of_word(int lo, int hi, int w) {
  const int from = max(lo - 32 * w, 0), to = min(hi - 32 * w, 32);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(from), "r"(max(to - from, 0)));
  return m;
}
// Made by one warp, 32 items at a time.
template <int kRows>
__device__ __forceinline__ void make_groups(Groups<kRows>& out, const QkvParams& p, int si, int mt, int lane) {
  const int N_s = p.s[si].N_s, m0 = mt * kRows, m1 = min(m0 + kRows, p.s[si].M);
  int count = 0;
  for (int first = m0 / N_s; first * N_s < m1; first += 32) {
    const int b = first + lane;
    const bool in = b * N_s < m1;
    const int a = in ? __ldg(p.index + b) : -1;
    const bool has = a >= 0 && a < p.n_adapters;
    int g = -1;  // the item's group
    for (int i = 0; i < count; ++i)
      if (out.adapter[i] == a) g = i;
    const unsigned peers = __match_any_sync(0xffffffffu, has ? a : -1);
    const bool leads = has && g < 0 && lane == __ffs(peers) - 1;
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    if (leads) {
      g = count + __popc(leaders & ((1u << lane) - 1));
      out.adapter[g] = a;
#pragma unroll
      for (int w = 0; w < kRows / 32; ++w) out.rows[g][w] = 0;
    }
    const int of_leader = __shfl_sync(0xffffffffu, g, __ffs(peers) - 1);
    __syncwarp();
    if (has) {
      if (g < 0) g = of_leader;
      const int lo = max(b * N_s, m0) - m0, hi = min(b * N_s + N_s, m1) - m0;
#pragma unroll
      for (int w = 0; w < kRows / 32; ++w) {
        const uint32_t bits = rows_of_word(lo, hi, w);
        if (bits) atomicOr(&out.rows[g][w], bits);
      }
    }
    count += __popc(leaders);
    __syncwarp();
  }
  if (lane == 0) out.count = count;
}
// The pieces of columns n0 .. end - 1 for the adapters: of one of q, k and v, and
// 64, 128 or 256 columns, so that two CTAs' halves of a piece are whole boxes of
// the up weights' rows, or a box's first rows.  next() gives the next one, from
// column c on.
struct Pieces {
  int hd, end, c, cols, part;
  __device__ __forceinline__ Pieces(int H_d, int n0, int end_)
      : hd(H_d), end(min(end_, 3 * H_d)), c(n0), cols(0), part(0) {}
  __device__ __forceinline__ bool next() {
    c += cols;
    if (c >= end) return false;
    part = (c >= hd) + (c >= 2 * hd);
    const int left = min((part + 1) * hd, end) - c;
    cols = left >= 256 ? 256 : left >= 128 ? 128 : 64;
    return true;
  }
};

// An item of work: columns n0 .. n0 + cols - 1 of row tile mt of stream si.
struct QkvItem {
  int si, mt, n0, cols;
};
template <int kCols>
__device__ __forceinline__ QkvItem item_at(const QkvParams& p, int t) {
  QkvItem it;
  int sub = 0;
  it.cols = kCols;
  if (t >= p.whole) {
    sub = (t - p.whole) & ((1 << p.parts_log) - 1);
    t = p.whole + ((t - p.whole) >> p.parts_log);
    it.cols = kCols >> p.parts_log;
  }
  it.si = t >= p.s[1].tile0 ? 1 : 0;
  t -= p.s[it.si].tile0;
  it.mt = static_cast<int>(p.by_tiles.div(t));
  it.n0 = (t - it.mt * p.n_tiles) * kCols + sub * it.cols;
  return it;
}

// This lane's part of a row's sum of squares, from its bf16 values (packed
// pairs; exact squares): a balanced tree over each block of 16 columns, and over
// the lane's two blocks at d = 128.  Two neighbouring sums at a time in packed
// fp32 arithmetic; the fma adds two exact squares with one rounding, as an
// addition of them does.
template <int D>
__device__ __forceinline__ float lane_squares(const uint32_t (&yb)[D / 8]) {
  float blk[D / 64];
#pragma unroll
  for (int b = 0; b < D / 64; ++b) {
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
  return D == 64 ? blk[0] : __fadd_rn(blk[0], blk[D / 64 - 1]);
}

// r of a row of d values from its sum of squares.  r is what is kept; rc, for
// q_hat / k_hat, takes one Newton step more: r (1 + t / 2), t = 1 - m r^2 of
// order 2^-22, is the root of m to 2^-44 before its rounding.  (r = 0, of a row
// whose squares pass the fp32 range, stays: m r is then not a number.)
template <int D>
__device__ __forceinline__ void row_rsqrt(float sum, float& r, float& rc) {
  const float m = __fadd_rn(__fmul_rn(sum, 1.f / D), kEps);
  r = rsqrtf(m);
  const float q = __fmul_rn(m, r);  // 1 - m r^2 = 1 - q r + (q - m r) r
  const float t = __fmaf_rn(__fmaf_rn(-m, r, q), r, __fmaf_rn(-q, r, 1.f));
  rc = r == 0.f ? r : __fmaf_rn(__fmul_rn(0.5f, r), t, r);
}

// The four lanes' sums of their kRows (2 or 4) rows, joined (lanes 2 apart
// first): lane b of the four ends with the whole sum of row b (2 rows: b / 2).
template <int kRows>
__device__ __forceinline__ float quad_row_sum(const float (&s)[kRows], int b) {
  const bool up = b & 2;
  if constexpr (kRows == 2) {
    const float t = __fadd_rn(up ? s[1] : s[0], __shfl_xor_sync(0xffffffffu, up ? s[0] : s[1], 2));
    return __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 1));
  } else {
    const float t0 = __fadd_rn(up ? s[2] : s[0], __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 2));
    const float t1 = __fadd_rn(up ? s[3] : s[1], __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 2));
    const bool odd = b & 1;
    return __fadd_rn(odd ? t1 : t0, __shfl_xor_sync(0xffffffffu, odd ? t0 : t1, 1));
  }
}

// 16 columns of a q_hat / k_hat row, (g x) r per element (y: 8 words of the
// row, g: their gains); `near` collects the elements within the midpoint window.
__device__ __forceinline__ void hat_cols16(const uint32_t* y, const uint64_t (&g)[8], float r, uint32_t (&w)[8],
                                           uint32_t& near) {
  const uint64_t r2 = f2_make(r, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // Unpacked by other instructions than in lane_squares, so that the compiler does not keep the row
    // unpacked in between.
    const float lo = __uint_as_float(__byte_perm(y[i], 0u, 0x1044)), hi = __uint_as_float(__byte_perm(y[i], 0u, 0x3244));
    float z0, z1;
    f2_split(f2_mul(f2_mul(g[i], f2_make(lo, hi)), r2), z0, z1);
    near_pair(z0, z1, near);
    w[i] = pack_bf16x2(z0, z1);
  }
}

// The rare path: a row of four lanes (src the first) that has an element near a
// bf16 midpoint, by the whole warp: each lane takes two columns of each 64 (word
// lane % 8 of lane src + lane / 8), the squares (exact) are summed by error-free
// additions, and elements that the fp32 arithmetic (r) puts near a midpoint are
// rounded from the double-float r.  to: the row.
template <int D>
__device__ __forceinline__ void fix_row(const uint32_t (&yb)[D / 8], int src, float r, const float* g, uint16_t* to,
                                        int lane) {
  uint32_t w[D / 64];
  float s = 0.f, e = 0.f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t v = __shfl_sync(0xffffffffu, yb[c * 8 + k], src + (lane >> 3));
      if ((lane & 7) == k) w[c] = v;
    }
    add_sq_df(w[c], s, e);
  }
  warp_sum_df(s, e);
  float rh, rl;
  rsqrt_mean_eps_df(s, e, 1.f / D, rh, rl);
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const int col = c * 64 + 2 * lane;
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = i ? bf_hi(w[c]) : bf_lo(w[c]);
      const float gv = g[col_offset(col + i) / 4];
      const float z = __fmul_rn(__fmul_rn(gv, x), r);
      f[i] = near_midpoint(z) ? round_bf16_df(gv, x, rh, rl) : z;
    }
    *reinterpret_cast<uint32_t*>(to + col) = pack_bf16x2(f[0], f[1]);
  }
}

// A head's columns (from col0 on) of 16 kHalves token rows, taddr their first
// TMEM lane and column.  rows: lane i's is row i of the warp's 32 (its index
// for head 0, kDeadRow past the stream's end), half0: the first 16 rows to take;
// bias, wscale: the columns' in shared memory; xscale: the 32 rows' (kE4m3).
// The accumulator is handed back (acc_empty) once its values are in registers.
//
// Lane 4 a + b holds rows a and a + 8 of each 16, columns 16 b .. 16 b + 15 of
// each 64: TMEM column 4 j + b is output column 16 b + j, by the order in which
// the weights' rows are loaded.  So four lanes write 128 consecutive bytes of a
// row from registers.
template <int D, int kMode, bool kPair, bool kWide, int kHalves>
__device__ __forceinline__ void qkv_emit(uint32_t taddr, uint64_t* acc_empty, int col0, uint32_t rows, int half0,
                                         uint32_t bias, uint32_t wscale, uint32_t xscale, const QkvParams& p,
                                         const QkvBars& bars, int lane) {
  constexpr int kRows = 2 * kHalves, kUnits = (D / 32) * kHalves;  // of 32 columns x 16 rows
  const bool wide = kPair ? kWide : p.wide;
  // Outputs at 16-byte boundaries, in turn / in one order (512 px at d = 64; 768 px, C = 1024, at d = 128): from bf16
  // 53.3 / 56.6 and 85.2 / 92.5 us, with adapters 69.5 / 75.0 and 103.3 / 110.8, from e4m3 at d = 128 71.8 / 79.9;
  // from e4m3 at d = 64, which has no instructions to spare, 50.0 / 48.3.  (At 32-byte boundaries 52, 83, 66, 99, 58, 38.)
  constexpr bool kTurn = kMode != kE4m3 || D != 64;
  const int a = lane >> 2, b = lane & 3;
  uint32_t row[kRows];
  uint64_t sx2[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    row[i] = __shfl_sync(0xffffffffu, rows, half0 * 16 + a + 8 * i);
    if constexpr (kMode == kE4m3) {
      const float sx = __uint_as_float(ld_shared_u32(xscale + (half0 * 16 + a + 8 * i) * 4));
      sx2[i] = f2_make(sx, sx);
    }
  }
  uint32_t yb[kRows][D / 8];  // packed pairs
  {
    uint32_t acc[2][16];
    tmem_ld_16x128b_x8(taddr, acc[0]);
    float4 bv[2], sv[2];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int c32 = u / kHalves, h = u % kHalves;
      if (h == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = col_offset((c32 / 2) * 64 + b * 16 + (c32 % 2) * 8 + j * 4);
          bv[j] = ld_shared_f4(bias + at);
          if constexpr (kMode == kE4m3) sv[j] = ld_shared_f4(wscale + at);
        }
      }
      tmem_wait_ld();
      if (u + 1 < kUnits) {
        const int c1 = (u + 1) / kHalves, h1 = (u + 1) % kHalves;
        tmem_ld_16x128b_x8(taddr + (static_cast<uint32_t>(16 * h1) << 16) + 32 * c1, acc[(u + 1) & 1]);
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_to<kPair>(acc_empty);
      }
      // Y = bf16(acc + bias), four columns of both rows at a time.
      const uint32_t(&v)[16] = acc[u & 1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint64_t y0 = f2_make(__uint_as_float(v[8 * j + i]), __uint_as_float(v[8 * j + 2 + i]));
          uint64_t y1 = f2_make(__uint_as_float(v[8 * j + 4 + i]), __uint_as_float(v[8 * j + 6 + i]));
          if constexpr (kMode == kE4m3) {
            const uint64_t sx = sx2[2 * h + i];
            y0 = f2_fma(f2_mul(y0, sx), f2_make(sv[j].x, sv[j].y), f2_make(bv[j].x, bv[j].y));
            y1 = f2_fma(f2_mul(y1, sx), f2_make(sv[j].z, sv[j].w), f2_make(bv[j].z, bv[j].w));
          } else {
            y0 = f2_add(y0, f2_make(bv[j].x, bv[j].y));
            y1 = f2_add(y1, f2_make(bv[j].z, bv[j].w));
          }
          float a0, a1, a2, a3;
          f2_split(y0, a0, a1);
          f2_split(y1, a2, a3);
          yb[2 * h + i][c32 * 4 + 2 * j] = pack_bf16x2(a0, a1);
          yb[2 * h + i][c32 * 4 + 2 * j + 1] = pack_bf16x2(a2, a3);
        }
      }
    }
  }
  const int hd = p.H * D;
  if (col0 >= 3 * hd) return;  // past the last head
  const int which = (col0 >= hd) + (col0 >= 2 * hd);  // 0 q, 1 k, 2 v
  const size_t head_rows = static_cast<size_t>((col0 - which * hd) / D) * p.N;
  {
    uint16_t* raw = p.out[which] + head_rows * D + b * 16;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        if (row[i] != kDeadRow)
          store_cols16<kTurn>(raw + static_cast<size_t>(row[i]) * D + c * 64, yb[i] + c * 8, wide, lane);
  }
  if (which == 2) return;
  float rc[kRows];
  {
    float s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = lane_squares<D>(yb[i]);
    float r, mine;
    row_rsqrt<D>(quad_row_sum<kRows>(s, b), r, mine);
    constexpr int kLanesRow = 4 / kRows;  // that hold a row's r
#pragma unroll
    for (int i = 0; i < kRows; ++i) rc[i] = __shfl_sync(0xffffffffu, mine, (lane & 28) + kLanesRow * i);
    const uint32_t own = __shfl_sync(0xffffffffu, rows, half0 * 16 + a + 8 * (b / kLanesRow));
    if (b % kLanesRow == 0 && own != kDeadRow) p.r[which][head_rows + own] = r;
  }
  const float* g = which == 0 ? bars.gq : bars.gk;
  uint16_t* hat = p.hat[which] + head_rows * D;
  uint32_t near[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) near[i] = kNoneNear;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint64_t gv[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = ld_shared_f4(smem_u32(g) + col_offset(c * 64 + b * 16 + j * 4));
      gv[2 * j] = f2_make(f.x, f.y);
      gv[2 * j + 1] = f2_make(f.z, f.w);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t w[8];
      hat_cols16(yb[i] + c * 8, gv, rc[i], w, near[i]);
      if (row[i] != kDeadRow)
        store_cols16<kTurn>(hat + static_cast<size_t>(row[i]) * D + c * 64 + b * 16, w, wide, lane);
    }
  }
  unsigned todo[kRows], any = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    todo[i] = __ballot_sync(0xffffffffu, any_near(near[i]) && row[i] != kDeadRow);
    any |= todo[i];
  }
  if (any) {
    __syncwarp();  // the rows' stores come before those of fix_row
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      while (todo[i]) {
        const int src = (__ffs(todo[i]) - 1) & ~3;
        todo[i] &= ~(15u << src);
        const uint32_t to = __shfl_sync(0xffffffffu, row[i], src);
        fix_row<D>(yb[i], src, __shfl_sync(0xffffffffu, rc[i], src), g, hat + static_cast<size_t>(to) * D, lane);
      }
  }
}

// kWide: of a pair, whether the outputs are at 32-byte boundaries (a kernel of its own for those that are not: with
// both in one 512 px from e4m3 rows took 42.2 us instead of 39.2); single CTAs look at p.wide.
template <int D, int kMode, bool kPair, bool kWide>
__global__ void __launch_bounds__(QkvCfg<D, kMode, kPair>::kThreads, 1)
    qkv_norm_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_w0,
                    const __grid_constant__ CUtensorMap map_x1, const __grid_constant__ CUtensorMap map_w1,
                    const __grid_constant__ QkvLoraMaps lm, const __grid_constant__ QkvParams p, const float* __restrict__ gq,
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
  const int first_item = blockIdx.x / kCtas, item_step = gridDim.x / kCtas;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.acc_full[b], 1);
      mbar_init(&bars.acc_empty[b], kCtas * Cfg::kEpiWarps);
      mbar_init(&bars.groups_full[b], 1);
      mbar_init(&bars.groups_empty[b], rank == 0 ? 2 : 1);  // the producer, and the issuer if it is here
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
    bars.gq[col_offset(i) / 4] = gq[i];
    bars.gk[col_offset(i) / 4] = gk[i];
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int ksteps = (p.C + kStepK - 1) / kStepK;

  if (warp >= Cfg::kEpiWarps) {
  if constexpr (Cfg::kSplitRegs) setmaxnreg_dec<QkvRegs::kOther>();
  if (warp == kWarpProd) {
    if (lane == 0) {
      tma_prefetch_desc(&map_x0);
      tma_prefetch_desc(&map_w0);
      tma_prefetch_desc(&map_x1);
      tma_prefetch_desc(&map_w1);
      int it = 0, lists = 0;
      bool ok = true, waited = false;
      for (int t = first_item; ok && t < p.items; t += item_step) {
        const auto [si, mt, n0, cols] = item_at<kCols>(p, t);
        const int w0 = n0 + rank * (cols / kCtas);  // this CTA's part of the weight rows
        const CUtensorMap* mx = si ? &map_x1 : &map_x0;
        const CUtensorMap* mw = si ? &map_w1 : &map_w0;
        for (int kb = 0; kb < ksteps; ++kb) {
          const int s = it % kStages;
          if (it >= kStages && !(ok = mbar_wait(&bars.empty[s], ((it / kStages) - 1) & 1, ab, dev_err))) break;
          uint8_t* st = sm + s * Cfg::kStageBytes;
          const uint32_t full = pair_bar<kPair>(&bars.full[s]);
          if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], kCtas * Cfg::kStageBytes);
          tma_load_2d_to<kPair>(st, mx, full, kb * kStepK, mt * kRows + rank * kBM);
          tma_load_4d_to<kPair>(st + kATile, mw, full, kb * kStepK, 0, (w0 & 63) >> 2, w0 >> 6);
          ++it;
        }
        if constexpr (kMode == kLora) {
          if (!ok || !p.lora[si]) continue;
          const CUtensorMap* mu = &lm.u[si];
          const int gb = lists & 1;
          if (!(ok = mbar_wait(&bars.groups_full[gb], (lists >> 1) & 1, ab, dev_err))) break;
          const Groups<kRows>& groups = reinterpret_cast<const Groups<kRows>*>(sm + Cfg::kOffGroups)[gb];
          const int count = groups.count;
          int used = 0;  // bytes of the open stage (0: none open)
          // The stage is closed by its one arrival; until then each group's bytes are added to what it expects.
          auto close = [&] {
            if (rank == 0) mbar_arrive(&bars.full[it % kStages]);
            used = 0;
            ++it;
          };
          Pieces pc(p.H * D, n0, n0 + cols);
          while (ok && count > 0 && pc.next()) {
            const int up0 = pc.c + rank * (pc.cols / kCtas);
            for (int kc = 0; ok && kc < p.rank_units; ++kc) {
              int g = 0;
              while (ok && g < count) {
                if (used + Cfg::kUnitU + Cfg::kUnitB > Cfg::kStageBytes) close();
                const int s = it % kStages;
                if (used == 0) {
                  if (it >= kStages && !(ok = mbar_wait(&bars.empty[s], ((it / kStages) - 1) & 1, ab, dev_err))) break;
                  if (!waited) griddep_wait();  // U is there
                  waited = true;
                }
                const uint32_t full = pair_bar<kPair>(&bars.full[s]);
                uint8_t* st = sm + s * Cfg::kStageBytes;
                if (rank == 0) mbar_expect_tx(&bars.full[s], kCtas * Cfg::kUnitU);
                tma_load_3d_to<kPair>(st + used, mu, full, 0, mt * kRows + rank * kBM,
                                      3 * (pc.part * p.rank_units + kc));
                used += Cfg::kUnitU;
                do {
                  if (rank == 0) mbar_expect_tx(&bars.full[s], kCtas * Cfg::kUnitB);
                  tma_load_5d_to<kPair>(st + used, &lm.up[si], full, kc * 16, 0, (up0 & 63) >> 2, up0 >> 6,
                                        groups.adapter[g]);
                  used += Cfg::kUnitB;
                } while (++g < count && used + Cfg::kUnitB <= Cfg::kStageBytes);
              }
            }
          }
          if (used > 0) close();
          mbar_arrive(&bars.groups_empty[gb]);
          ++lists;
        }
      }
      if constexpr (kMode == kLora) griddep_wait();  // this grid ends after the one before it
      // Aborted: the copies in flight land before the CTA, or the pair, exits.  (A role that gives up later has
      // waited a second for the issuer, which has then met every stage, or has itself waited that long for one of
      // them: by then those copies have landed.  The pair's closing barrier keeps both CTAs until then.)
      if (*ab)
        drain_ring(it, kStages, rank == 0, [&](int s, uint32_t parity) { mbar_wait_drain(&bars.full[s], parity); });
    }
  } else if (warp == kWarpIssue) {
    if (lane == 0 && rank == 0) {
      int it = 0, lt = 0, lists = 0;
      bool ok = true;
      for (int t = first_item; ok && t < p.items; t += item_step, ++lt) {
        const auto [si, mt, n0, cols] = item_at<kCols>(p, t);
        const uint32_t idesc =
            kMode == kE4m3 ? idesc_e4m3_f32(kRows, cols) : idesc_bf16_f32(kRows, cols, false, false);
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
          if (ok && p.lora[si]) {
            const int gb = lists & 1;
            if (!(ok = mbar_wait(&bars.groups_full[gb], (lists >> 1) & 1, ab, dev_err))) break;
            const Groups<kRows>& groups = reinterpret_cast<const Groups<kRows>*>(sm + Cfg::kOffGroups)[gb];
            const int count = groups.count;
            int used = 0;  // as the producer counts
            auto close = [&] {
              umma_commit_to<kPair>(&bars.empty[it % kStages]);
              used = 0;
              ++it;
            };
            Pieces pc(p.H * D, n0, n0 + cols);
            while (ok && count > 0 && pc.next()) {
              const uint32_t desc = idesc_bf16_f32(kRows, pc.cols, false, false), at = acc + (pc.c - n0);
              for (int kc = 0; ok && kc < p.rank_units; ++kc) {
                int g = 0;
                while (ok && g < count) {
                  if (used + Cfg::kUnitU + Cfg::kUnitB > Cfg::kStageBytes) close();
                  const int s = it % kStages;
                  if (used == 0) {
                    if (!(ok = mbar_wait(&bars.full[s], (it / kStages) & 1, ab, dev_err))) break;
                    tc_fence_after();
                  }
                  const uint32_t st = smem_u32(sm + s * Cfg::kStageBytes);
                  const uint64_t u = sdesc_sw32_kmajor(st + used, 256);
                  used += Cfg::kUnitU;
                  do {
                    uint32_t off[4 * kCtas];  // the lanes (rows) that are not the group's
#pragma unroll
                    for (int w = 0; w < 4 * kCtas; ++w) off[w] = ~groups.rows[g][w];
                    const uint64_t up = sdesc_sw32_kmajor(st + used, 256);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                      umma_bf16_ss_lanes(at, desc_add(u, k * Cfg::kTermU), up, desc, off, 1u);
                    used += Cfg::kUnitB;
                  } while (++g < count && used + Cfg::kUnitB <= Cfg::kStageBytes);
                }
              }
            }
            if (ok && used > 0) close();
            mbar_arrive(&bars.groups_empty[gb]);
            ++lists;
          }
        }
        if (ok) umma_commit_to<kPair>(&bars.acc_full[abuf]);
      }
      // Every MMA this thread issued has completed once this barrier flips.
      umma_commit<kCtas>(&bars.mma_done);
      mbar_wait_drain(&bars.mma_done, 0);
    }
  } else if (kMode == kLora && warp == Cfg::kWarpGroups) {
    int lists = 0;
    for (int t = first_item; t < p.items; t += item_step) {
      const QkvItem item = item_at<kCols>(p, t);
      if (!p.lora[item.si]) continue;
      const int gb = lists & 1;
      if (lists >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bars.groups_empty[gb], ((lists >> 1) - 1) & 1, ab, dev_err)))
        break;
      make_groups(reinterpret_cast<Groups<kRows>*>(sm + Cfg::kOffGroups)[gb], p, item.si, item.mt, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.groups_full[gb]);
      ++lists;
    }
  }
  } else {
    if constexpr (Cfg::kSplitRegs) setmaxnreg_inc<QkvRegs::kEpi>();
    // Warps of a group share the tile's columns from wcol on: each takes the TMEM lanes of warp w % 4, all 32
    // or one half of them.
    const int lg = warp & 3, group = warp / Cfg::kGroupWarps, wcol = group * D;
    const int half0 = Cfg::kHalves == 2 ? 0 : (warp >> 2) & 1;
    const uint32_t bias_s = smem_u32(sm + Cfg::kOffBias) + wcol * 5;
    const uint32_t wscale_s = smem_u32(sm + Cfg::kOffScale) + wcol * 5;      // kE4m3
    const uint32_t xscale_w = smem_u32(sm + Cfg::kOffXScale + warp * 256);  // kE4m3
    const int hd3 = 3 * p.H * D;
    // What the epilogue of a tile reads from global memory, copied to shared memory one tile ahead (its
    // latency, some 700 cycles each, is not met): the bias of the group's columns (zero past 3 H d, or without
    // a bias) by its first warp; kE4m3: their scales by its second, and by each warp those of its rows.
    auto fetch = [&](int t, int buf) {
      const QkvItem it = item_at<kCols>(p, t);
      const QkvStream& S = p.s[it.si];
      const int col = it.n0 + wcol + lane * 4;
      auto cols = [&](uint32_t to, const float* from) {
        if (lane * 4 >= D) return;
        if (from && col < hd3)
          cp_async16(to + buf * Cfg::kColBytes + col_offset(lane * 4), from + col);
        else
          st_shared_v4(to + buf * Cfg::kColBytes + col_offset(lane * 4), 0u, 0u, 0u, 0u);
      };
      if (warp % Cfg::kGroupWarps == 0) cols(bias_s, S.bias);
      if constexpr (kMode == kE4m3) {
        if (warp % Cfg::kGroupWarps == 1) cols(wscale_s, S.sw);
        const int m = it.mt * kRows + rank * kBM + lg * 32 + lane;
        const uint32_t xs = xscale_w + buf * 128 + lane * 4;
        if (m < S.M)
          cp_async4(xs, S.sx + m);
        else
          st_shared_u32(xs, 0u);
      }
      cp_async_commit();
    };
    int lt = 0;
    if (first_item < p.items) fetch(first_item, 0);
    for (int t = first_item; t < p.items; t += item_step, ++lt) {
      const int abuf = lt & 1;
      const QkvItem it = item_at<kCols>(p, t);
      const QkvStream& S = p.s[it.si];
      const int m = it.mt * kRows + rank * kBM + lg * 32 + lane;
      uint32_t row = kDeadRow;
      if (m < S.M) {
        const int bi = m / S.N_s;
        // < B H N < 2^31 / d
        row = static_cast<uint32_t>(bi) * p.H * p.N + S.row0 + (m - bi * S.N_s);
      }
      cp_async_wait_all();
      bool ok = mbar_wait(&bars.acc_full[abuf], (lt >> 1) & 1, ab, dev_err);
      // The group's copies have landed, it is done with the other buffer, and it goes on as one.
      ok = barrier_all(1 + group, 32 * Cfg::kGroupWarps, ok);
      if (!ok) break;
      tc_fence_after();
      if (t + item_step < p.items) fetch(t + item_step, abuf ^ 1);
      if (wcol >= it.cols) {  // a part without this group's columns
        if (lane == 0) mbar_arrive_to<kPair>(&bars.acc_empty[abuf]);
        continue;
      }
      qkv_emit<D, kMode, kPair, kWide, Cfg::kHalves>(
          tmem + (static_cast<uint32_t>(lg * 32 + half0 * 16) << 16) + abuf * kCols + wcol, &bars.acc_empty[abuf],
          it.n0 + wcol, row, half0, bias_s + abuf * Cfg::kColBytes, wscale_s + abuf * Cfg::kColBytes,
          xscale_w + abuf * 128, p, bars, lane);
    }
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
// registers its setmaxnreg split (if regs is not 0) was sized for; asked once per device and
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
  if (!QkvRegs::fits(fa.numRegs, regs)) return cudaErrorInvalidConfiguration;
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

template <int D, int kMode, bool kPair, bool kWide>
cudaError_t launch_qkv_kernel(const CUtensorMap (&maps)[4], const QkvLoraMaps& lm, QkvParams& p, int tiles,
                              const float* gq, const float* gk, uint32_t* dev_err, cudaStream_t st) {
  using Cfg = QkvCfg<D, kMode, kPair>;
  auto kernel = qkv_norm_kernel<D, kMode, kPair, kWide>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kDynSmem);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count();
  int groups = sms > Cfg::kCtas ? sms / Cfg::kCtas : 1;
  if constexpr (kPair) {
    static std::atomic<int> known[64];
    int fit = 0;
    e = resident_pairs(kernel, Cfg::kThreads, Cfg::kDynSmem, Cfg::kLaunchRegs, known, 64, &fit);
    if (e != cudaSuccess) return e;
    if (fit < groups) groups = fit;
  }
  // The tiles left over once all pairs have taken as many: in parts of a head (d = 64) or of two, when there
  // are enough pairs for each to take a part at most.  In parts / whole (bf16, d = 64, C = 768): 81 tiles on 76
  // pairs 14.5 / 16.6 us, 108 tiles 15.5 / 17.0, 621 tiles 51.3 / 53.0; by one head / by two: 14.5 / 15.1 (81).
  const int left = tiles % groups;
  p.whole = tiles;
  p.parts_log = 0;
  if (kPair && left > 0) {
    for (int l = D == 64 ? 2 : 1; l > 0 && p.parts_log == 0; --l)
      if ((left << l) <= groups) p.parts_log = l;
    if (p.parts_log > 0) p.whole = tiles - left;
  }
  p.items = p.whole + ((tiles - p.whole) << p.parts_log);
  const int grid = (p.items < groups ? p.items : groups) * Cfg::kCtas;
  return launch_pdl_cluster(kernel, Cfg::kCtas, dim3(grid), dim3(Cfg::kThreads), Cfg::kDynSmem, st, maps[0], maps[1],
                            maps[2], maps[3], lm, p, gq, gk, dev_err);
}

template <int D, int kMode>
cudaError_t launch_qkv_tiles(const CUtensorMap (&maps)[4], const QkvLoraMaps& lm, QkvParams& p, int tiles,
                             const QkvLaunch& a, uint32_t* dev_err, cudaStream_t st) {
  if (!a.pair) return launch_qkv_kernel<D, kMode, false, false>(maps, lm, p, tiles, a.gq, a.gk, dev_err, st);
  if (a.wide) return launch_qkv_kernel<D, kMode, true, true>(maps, lm, p, tiles, a.gq, a.gk, dev_err, st);
  return launch_qkv_kernel<D, kMode, true, false>(maps, lm, p, tiles, a.gq, a.gk, dev_err, st);
}

}  // namespace

// One form of the projection (each is compiled in a file of its own).
template <int kMode>
cudaError_t launch_qkv_form(const CUtensorMap (&maps)[4], const QkvLaunch& a, uint32_t* dev_err, cudaStream_t st,
                            const LoraLaunch* lora, const CUtensorMap* lora_maps) {
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
  for (int i = 0; i < 3; ++i) p.out[i] = a.out[i];
  for (int i = 0; i < 2; ++i) {
    p.hat[i] = a.hat[i];
    p.r[i] = a.r[i];
  }
  p.wide = a.wide;
  p.index = lora ? lora->index : nullptr;
  p.n_adapters = lora ? lora->n_adapters : 0;
  p.after_down = p.lora[0] || p.lora[1];
  p.rank_units = lora ? (lora->rank + 15) / 16 : 0;
  if (tile0 == 0) return cudaSuccess;
  if (a.d == 64) return launch_qkv_tiles<64, kMode>(maps, lm, p, tile0, a, dev_err, st);
  return launch_qkv_tiles<128, kMode>(maps, lm, p, tile0, a, dev_err, st);
}

}  // namespace jattn
