// grouped.cuh — the order in which the persistent attention kernels take the blocks
// of packed sequences with grouped heads, causal or not.
#pragma once
#include <algorithm>

#include "jattn_internal.h"

namespace jattn {

// The segments' blocks of `block` rows.  A block's level is its place in its segment,
// and the work of a causal block grows by one with its level (counted from the
// segment's start for queries, from its end for keys).  Segments are sorted by length,
// the longest first; causal: by levels, the highest first, each with all the segments
// that have it, so that the work falls from first to last; not causal, where all
// blocks of a segment cost the same: by segments.
struct GroupedOrder {
  int n;                    // segments
  int start[kMaxSegments];  // their first rows, and rows
  int len[kMaxSegments];
  int prow[kMaxSegments];  // their first rows in the padded scratch (SegTable)
  int first[kMaxSegments + 1];   // causal: blocks before the levels that just segments 0 .. i have; else before segment i
  int blocks[kMaxSegments];  // of segment i
  int pre[kMaxSegments];

  // Segment and level of block k.
  __host__ __device__ __forceinline__ void at(int k, bool causal, int* seg, int* level) const {
    int lo = 0, hi = n;  // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= k) lo = mid;
      else hi = mid;
    }
    const int off = k - first[lo];
    if (causal) {
      const int row = off / (lo + 1);
      *seg = off - row * (lo + 1);
      *level = blocks[lo] - 1 - row;
    } else {
      *seg = lo;
      *level = off;
    }
  }
#ifndef ORDER
#define ORDER 1
#endif
  __host__ __device__ __forceinline__ void unit(int u, int heads, bool causal, int* seg, int* head, int* level) const {
    if (ORDER == 1) {
      const int k = u / heads;
      *head = u - k * heads;
      at(k, causal, seg, level);
      return;
    }
    // segments, heads, levels
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] * heads <= u) lo = mid;
      else hi = mid;
    }
    const int off = u - pre[lo] * heads;
    *seg = lo;
    *head = off / blocks[lo];
    const int l = off - *head * blocks[lo];
    *level = causal ? blocks[lo] - 1 - l : l;
  }
  // From the segments of s, in blocks of that many rows; returns how many blocks.
  int make(const GroupedShape& s, int block) {
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
    pre[0] = 0;
    for (int i = 1; i < n; ++i) pre[i] = pre[i - 1] + blocks[i - 1];
    first[0] = 0;
    for (int i = 0; i < n; ++i)
      first[i + 1] = first[i] + (s.causal ? (blocks[i] - (i + 1 < n ? blocks[i + 1] : 0)) * (i + 1) : blocks[i]);
    return first[n];
  }
};

// The unit after u, a CTA's ui-th.  Where the work falls from first to last (grouped) the CTAs take
// each round's units in turn from the one and the other end.
template <bool kGrouped>
__device__ __forceinline__ int next_unit(int u, int ui) {
  if constexpr (kGrouped) {
    const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
#ifndef SNAKE
#define SNAKE 1
#endif
    if (SNAKE) return ui * grid + (ui & 1 ? grid - 1 - c : c);
    return u + grid;
  } else {
    return u + static_cast<int>(gridDim.x);
  }
}

}  // namespace jattn
