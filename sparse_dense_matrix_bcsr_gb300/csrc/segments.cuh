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

// The segment that holds row n, or -1.
__device__ __forceinline__ int32_t find_segment(const int64_t *__restrict__ seg_ptr, int32_t n_seg, int64_t n) {
  const int32_t s = last_segment_from(seg_ptr, n_seg, n);
  return s >= 0 && seg_ptr[s + 1] > n ? s : -1;
}

// The adapter of segment s: -1 for none; an index outside the pool is recorded
// in the status word and taken as none.
__device__ __forceinline__ int32_t segment_adapter(const int32_t *__restrict__ seg_adapter, int32_t s, int32_t n_adapters,
                                                   uint32_t *status) {
  const int32_t a = seg_adapter[s];
  if (a < -1 || a >= n_adapters) {
    atomicOr(status, kDevIndex);
    return -1;
  }
  return a;
}

// The segments with an adapter among rows [row0, row1), in order, by one warp:
// their rows relative to row0.  Returns how many (at most cap; row1 - row0 is
// enough, as segments share no row).
__device__ __forceinline__ int32_t list_segments(const int64_t *__restrict__ seg_ptr,
                                                 const int32_t *__restrict__ seg_adapter, int32_t n_seg,
                                                 int32_t n_adapters, int64_t row0, int64_t row1, TileSegment *out,
                                                 int32_t cap, uint32_t *status) {
  const int lane = threadIdx.x & 31;
  int32_t count = 0;
  for (int32_t base = max(last_segment_from(seg_ptr, n_seg, row0), 0); base < n_seg; base += 32) {
    const int32_t s = base + lane;
    bool past = true;
    TileSegment t{-1, 0, 0, 0};
    if (s < n_seg) {
      const int64_t b = seg_ptr[s], e = seg_ptr[s + 1];
      past = b >= row1;
      const int64_t lo = max(b, row0), hi = min(e, row1);
      if (lo < hi) {
        t.adapter = segment_adapter(seg_adapter, s, n_adapters, status);
        t.begin = static_cast<int32_t>(lo - row0);
        t.end = static_cast<int32_t>(hi - row0);
      }
    }
    const uint32_t active = __ballot_sync(0xffffffffu, t.adapter >= 0);
    const int32_t at = count + __popc(active & ((1u << lane) - 1u));
    if (t.adapter >= 0 && at < cap) out[at] = t;
    count = min(count + __popc(active), cap);
    if (__any_sync(0xffffffffu, past)) break;
  }
  return count;
}

}  // namespace spmm
