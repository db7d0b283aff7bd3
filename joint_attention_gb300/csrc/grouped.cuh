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
// Segments are sorted by length.  Causal: by levels, the highest first, each with all the
// segments that have it; else, where all blocks of a segment cost the same, by segments; a
// block's heads side by side.  So the work falls from first to last, and the CTAs take each
// round's units in turn from the one and the other end.  (By segments, heads, levels
// instead, so that a head's units run side by side: 16 heads of 128, 16384 rows, causal,
// forward 1089 us instead of 924, backward, 4 kv heads, 3374 instead of 2167; not causal,
// 4 x 2381 rows, 24 heads of 128, forward 307 and 306 us; 16 x 1101 rows, 12 heads of 64,
// backward 265 instead of 245, as units of one head add to the same dQ at once.)
template <bool kCausal>
struct GroupedOrder {
  int n;                    // segments
  int start[kMaxSegments];  // their first rows, and rows
  int len[kMaxSegments];
  int prow[kMaxSegments];  // their first rows in the padded scratch (SegTable)
  // Blocks before those of segment i; causal: before the levels that just segments 0 .. i
  // have.
  int first[kMaxSegments + 1];
  int blocks[kMaxSegments];  // of segment i
  DivU31 by_count[kCausal ? kMaxSegments : 1];  // by i + 1
  DivU31 by_heads;
  int heads;

  __device__ __forceinline__ void unit(int u, int* seg, int* head, int* level) const {
    const int k = static_cast<int>(by_heads.div(static_cast<uint32_t>(u)));
    *head = u - k * heads;
    int lo = 0, hi = n;  // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= k) lo = mid;
      else hi = mid;
    }
    const int off = k - first[lo];
    if constexpr (kCausal) {
      const int row = static_cast<int>(by_count[lo].div(static_cast<uint32_t>(off)));
      *seg = off - row * (lo + 1);
      *level = blocks[lo] - 1 - row;
    } else {
      *seg = lo;
      *level = off;
    }
  }
  // A CTA's ui-th unit.
  __device__ __forceinline__ int of(int ui) const {
    const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return ui * grid + (ui & 1 ? grid - 1 - c : c);
  }
  // From the segments of s, in blocks of that many rows, for each of the heads; returns how many units.
  int make(const GroupedShape& s, int block, int of_heads) {
    n = s.seg.n;
    int by[kMaxSegments];
    for (int i = 0; i < n; ++i) by[i] = i;
    auto rows = [&](int i) { return s.seg.cu[i + 1] - s.seg.cu[i]; };
    std::sort(by, by + n, [&](int a, int b) { return rows(a) != rows(b) ? rows(a) > rows(b) : a < b; });
    for (int i = 0; i < n; ++i) {
      start[i] = s.seg.cu[by[i]];
      len[i] = rows(by[i]);
      prow[i] = s.seg.pcu[by[i]];
      blocks[i] = (len[i] + block - 1) / block;
    }
    first[0] = 0;
    for (int i = 0; i < n; ++i) {
      first[i + 1] = first[i] + (kCausal ? (blocks[i] - (i + 1 < n ? blocks[i + 1] : 0)) * (i + 1) : blocks[i]);
      if constexpr (kCausal) by_count[i] = make_div_u31(static_cast<uint32_t>(i + 1));
    }
    heads = of_heads;
    by_heads = make_div_u31(static_cast<uint32_t>(heads));
    return first[n] * heads;
  }
};

// The unit after u, a CTA's ui-th, of any work description.
template <class W>
__device__ __forceinline__ int next_unit(const W& w, int u, int ui) {
  if constexpr (W::kGrouped) return w.order.of(ui);
  else return u + static_cast<int>(gridDim.x);
}

}  // namespace jattn
