// grouped.cuh — the order in which the persistent attention kernels take the blocks
// of packed sequences with grouped heads, causal or not.
#pragma once
#include <algorithm>

#include "fastdiv.cuh"
#include "jattn_internal.h"

namespace jattn {

// The segments' blocks of `block` rows, for each of `heads` heads, as units 0, 1, ...  A
// block's level is its place in its segment, and the work of a causal block grows by one
// with its level (counted from the segment's start for queries, from its end for keys).
// Segments are sorted by length, the longest first.
//
// falling: by levels, the highest first, each with all the segments that have it and all
// heads, so that the work falls from first to last, and the CTAs take each round's units in
// turn from the one and the other end.  Else by segments, heads, levels, and every CTA the
// one gridDim.x further on: CTAs side by side then share a head's keys and values.
// Measured: forward, causal, 16 heads of 128, 16384 rows 924 us falling, 1089 else (8192
// rows 254, 323); not causal, 4 x 2381 rows, 24 heads of 128 315 us falling, 296 else.
// Backward, causal, 8192 rows, 590 and 966 us, not causal, 16 x 1101 rows, 12 heads of 64
// 245 and 265: its units of one head at once would add to the same dQ.
template <bool kCausal, bool kFalling>
struct GroupedOrder {
  static_assert(kFalling || !kCausal, "causal blocks of other work one after the other");
  int n;                    // segments
  int start[kMaxSegments];  // their first rows, and rows
  int len[kMaxSegments];
  int prow[kMaxSegments];  // their first rows in the padded scratch (SegTable)
  // Blocks before those of segment i; causal: before the levels that just segments 0 .. i
  // have.
  int first[kMaxSegments + 1];
  int blocks[kMaxSegments];   // of segment i
  DivU31 div[kMaxSegments];   // causal: by i + 1; else by segment i's blocks
  DivU31 by_heads;
  int heads;

  __device__ __forceinline__ void unit(int u, int* seg, int* head, int* level) const {
    int k = u, each = heads;
    if (kFalling) {
      k = static_cast<int>(by_heads.div(static_cast<uint32_t>(u)));
      each = 1;
      *head = u - k * heads;
    }
    int lo = 0, hi = n;  // first[lo] * each <= k < first[hi] * each
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] * each <= k) lo = mid;
      else hi = mid;
    }
    const int off = k - first[lo] * each;
    *seg = lo;
    *level = off;
    if (kCausal) {
      const int row = static_cast<int>(div[lo].div(static_cast<uint32_t>(off)));
      *seg = off - row * (lo + 1);
      *level = blocks[lo] - 1 - row;
    } else if (!kFalling) {
      *head = static_cast<int>(div[lo].div(static_cast<uint32_t>(off)));
      *level = off - *head * blocks[lo];
    }
  }
  // The unit after u of a CTA, its ui-th.
  __device__ __forceinline__ int next(int u, int ui) const {
    const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return kFalling ? ui * grid + (ui & 1 ? grid - 1 - c : c) : u + grid;
  }
  // From the segments of s, in blocks of that many rows, for each of the heads; returns how many units.
  int make(const GroupedShape& s, int block, int of_heads) {
    n = s.seg.n;
    int by[kMaxSegments];
    for (int i = 0; i < n; ++i) by[i] = i;
    auto rows = [&](int i) { return s.seg.cu[i + 1] - s.seg.cu[i]; };
    std::stable_sort(by, by + n, [&](int a, int b) { return rows(a) > rows(b); });
    for (int i = 0; i < n; ++i) {
      start[i] = s.seg.cu[by[i]];
      len[i] = rows(by[i]);
      prow[i] = s.seg.pcu[by[i]];
      blocks[i] = (len[i] + block - 1) / block;
    }
    first[0] = 0;
    for (int i = 0; i < n; ++i) {
      first[i + 1] = first[i] + (kCausal ? (blocks[i] - (i + 1 < n ? blocks[i + 1] : 0)) * (i + 1) : blocks[i]);
      div[i] = make_div_u31(static_cast<uint32_t>(kCausal ? i + 1 : blocks[i]));
    }
    heads = of_heads;
    by_heads = make_div_u31(static_cast<uint32_t>(heads));
    return first[n] * heads;
  }
};

// The unit after u, a CTA's ui-th, of any work description.
template <class W>
__device__ __forceinline__ int next_unit(const W& w, int u, int ui) {
  if constexpr (W::kGrouped) return w.order.next(u, ui);
  else return u + static_cast<int>(gridDim.x);
}

}  // namespace jattn
