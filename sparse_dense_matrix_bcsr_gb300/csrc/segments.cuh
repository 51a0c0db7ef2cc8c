// segments.cuh -- rows of a batch grouped into segments, each with an adapter.
#pragma once

#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace spmm {

// A warp's search for the last segment s with seg_ptr[s] <= n, 32 probes a step
// (two dependent loads up to 1024 segments); -1 if there is none.  Whatever
// seg_ptr holds, the answer is -1 or an index below n_seg.
__device__ __forceinline__ int32_t last_segment_from(const int64_t *__restrict__ seg_ptr, int32_t n_seg, int64_t n) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = n_seg;  // the answer lies in [lo, hi) if there is one
  while (lo < hi) {
    const int32_t stride = (hi - lo + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane) * stride;
    const bool below = i < hi && seg_ptr[i] <= n;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    if (c == 0) return -1;
    const int32_t at = lo + (c - 1) * stride;
    if (stride == 1) return at;
    hi = min(hi, at + stride);
    lo = at;
  }
  return -1;
}

// The adapter of segment s: -1 for none; an index outside the pool is recorded
// in the status word and taken as none.
__device__ __forceinline__ int32_t checked_adapter(int32_t a, int32_t n_adapters, uint32_t *status) {
  if (a < -1 || a >= n_adapters) {
    atomicOr(status, kDevIndex);
    return -1;
  }
  return a;
}

// Batches of up to kFewSegments are looked through whole, with every load in
// flight at once: one memory round trip instead of a search's three or four,
// which is what a decoding step waits for.
constexpr int kFewGroups = 4;
constexpr int32_t kFewSegments = 32 * kFewGroups;

// Lane l holds segments first + l, first + l + 32, ...; segments that do not
// exist are empty.
struct FewSegments {
  int64_t begin[kFewGroups], end[kFewGroups];
  int32_t adapter[kFewGroups];
  __device__ __forceinline__ FewSegments(const int64_t *__restrict__ seg_ptr, const int32_t *__restrict__ seg_adapter,
                                         int32_t n_seg, int32_t first = 0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < kFewGroups; ++g) {
      const int32_t s = first + 32 * g + lane;
      const bool in = s < n_seg;
      begin[g] = in ? seg_ptr[s] : 0;
      end[g] = in ? seg_ptr[s + 1] : 0;
      adapter[g] = in ? seg_adapter[s] : -1;
    }
  }
};

// Row tiles of `rows` rows cut at the segments' ends: piece e is the part of tile
// t that lies in segment s, with e = t + s.  From one piece to the next either
// the tile or the segment moves on, so the sum is a number of its own for every
// piece (numbers without one are left over where both move on or a segment is
// empty), pieces number below tiles + n_seg, and one search finds piece e: the
// last segment with s + tile(seg_ptr[s]) <= e.
struct RowPiece {
  int64_t begin, end;  // rows of the batch
  int32_t tile, adapter;
};
__device__ __forceinline__ RowPiece find_piece(const int64_t *__restrict__ seg_ptr, const int32_t *__restrict__ seg_adapter,
                                               int32_t n_seg, int32_t n_adapters, int32_t rows, int64_t N, int32_t e,
                                               uint32_t *status) {
  const int lane = threadIdx.x & 31;
  RowPiece r{0, 0, 0, -1};
  int32_t s = -1, adapter = -1;
  int64_t b = 0, last = 0;
  if (n_seg <= kFewSegments) {
    const FewSegments few(seg_ptr, seg_adapter, n_seg);
#pragma unroll
    for (int g = 0; g < kFewGroups; ++g) {
      const int32_t i = 32 * g + lane;
      const int c = __popc(__ballot_sync(0xffffffffu, i < n_seg && i + few.begin[g] / rows <= e));
      if (c > 0) {
        s = 32 * g + c - 1;
        b = __shfl_sync(0xffffffffu, few.begin[g], c - 1);
        last = __shfl_sync(0xffffffffu, few.end[g], c - 1);
        adapter = __shfl_sync(0xffffffffu, few.adapter[g], c - 1);
      }
    }
    if (s < 0) return r;
  } else {
    int32_t lo = 0, hi = n_seg;
    while (lo < hi) {
      const int32_t stride = (hi - lo + 31) / 32;
      const int64_t i = lo + static_cast<int64_t>(lane) * stride;
      const bool below = i < hi && i + seg_ptr[i] / rows <= e;
      const int c = __popc(__ballot_sync(0xffffffffu, below));
      if (c == 0) break;
      const int32_t at = lo + (c - 1) * stride;
      if (stride == 1) {
        s = at;
        break;
      }
      hi = min(hi, at + stride);
      lo = at;
    }
    if (s < 0) return r;
    b = seg_ptr[s];
    last = seg_ptr[s + 1];
    adapter = seg_adapter[s];
  }
  r.tile = e - s;
  r.begin = max(max(b, int64_t{0}), static_cast<int64_t>(r.tile) * rows);
  r.end = min(min(last, N), static_cast<int64_t>(r.tile + 1) * rows);
  if (r.begin < r.end) r.adapter = checked_adapter(adapter, n_adapters, status);
  return r;
}

// The segment that holds row n, by one warp: its rows and adapter (-1 for none).
struct RowSegment {
  int64_t begin, end;
  int32_t adapter;
};
__device__ __forceinline__ RowSegment find_row(const int64_t *__restrict__ seg_ptr, const int32_t *__restrict__ seg_adapter,
                                               int32_t n_seg, int32_t n_adapters, int64_t n, uint32_t *status) {
  RowSegment r{0, 0, -1};
  if (n_seg <= kFewSegments) {
    const FewSegments few(seg_ptr, seg_adapter, n_seg);
#pragma unroll
    for (int g = 0; g < kFewGroups; ++g) {
      const uint32_t hit = __ballot_sync(0xffffffffu, few.begin[g] <= n && n < few.end[g]);
      if (hit) {
        const int l = __ffs(hit) - 1;
        r.begin = __shfl_sync(0xffffffffu, few.begin[g], l);
        r.end = __shfl_sync(0xffffffffu, few.end[g], l);
        r.adapter = __shfl_sync(0xffffffffu, few.adapter[g], l);
      }
    }
  } else {
    const int32_t s = last_segment_from(seg_ptr, n_seg, n);
    if (s < 0) return r;
    r.begin = seg_ptr[s];
    r.end = seg_ptr[s + 1];
    r.adapter = n < r.end ? seg_adapter[s] : -1;
  }
  r.adapter = checked_adapter(r.adapter, n_adapters, status);
  return r;
}

// The segments with an adapter among rows [row0, row1), in order, by one warp:
// out[i] with rows relative to row0.  Returns how many (at most cap; row1 - row0 is enough, as segments
// share no row).
__device__ __forceinline__ int32_t list_segments(const int64_t *__restrict__ seg_ptr,
                                                 const int32_t *__restrict__ seg_adapter, int32_t n_seg,
                                                 int32_t n_adapters, int64_t row0, int64_t row1, TileSegment *out,
                                                 int32_t cap, uint32_t *status) {
  const int lane = threadIdx.x & 31;
  int32_t count = 0;
  auto group = [&](int64_t begin, int64_t end, int32_t adapter) {
    TileSegment t{-1, 0, 0, 0};
    const int64_t lo = max(begin, row0), hi = min(end, row1);
    if (lo < hi) {
      t.adapter = checked_adapter(adapter, n_adapters, status);
      t.begin = static_cast<int32_t>(lo - row0);
      t.end = static_cast<int32_t>(hi - row0);
    }
    const uint32_t active = __ballot_sync(0xffffffffu, t.adapter >= 0);
    const int32_t at = count + __popc(active & ((1u << lane) - 1u));
    if (t.adapter >= 0 && at < cap) out[at] = t;
    count = min(count + __popc(active), cap);
  };
  if (n_seg <= kFewSegments) {
    const FewSegments few(seg_ptr, seg_adapter, n_seg);
#pragma unroll
    for (int g = 0; g < kFewGroups; ++g) group(few.begin[g], few.end[g], few.adapter[g]);
    return count;
  }
  for (int32_t base = max(last_segment_from(seg_ptr, n_seg, row0), 0); base < n_seg; base += 32) {
    const int32_t s = base + lane;
    const bool in = s < n_seg;
    const int64_t b = in ? seg_ptr[s] : row1, e = in ? seg_ptr[s + 1] : row1;
    group(b, e, in ? seg_adapter[s] : -1);
    if (__any_sync(0xffffffffu, b >= row1)) break;
  }
  return count;
}

}  // namespace spmm
