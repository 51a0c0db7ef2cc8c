// segments.cuh -- rows of a batch grouped into segments, each with an adapter.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace spmm {

// A warp's search for the segment that holds row n: the last s with
// seg_ptr[s] <= n, 32 probes a step (two dependent loads up to 1024 segments).
// Returns -1 when the row lies in no segment; seg_ptr entries that decrease
// give some segment or -1, always an index below n_seg.
__device__ __forceinline__ int32_t find_segment(const int64_t *__restrict__ seg_ptr, int32_t n_seg, int64_t n) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, hi = n_seg;  // the answer lies in [lo, hi) if there is one
  while (lo < hi) {
    const int32_t stride = (hi - lo + 31) / 32;
    const int64_t i = lo + static_cast<int64_t>(lane) * stride;
    const bool below = i < hi && seg_ptr[i] <= n;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    if (c == 0) return -1;
    const int32_t at = lo + (c - 1) * stride;
    if (stride == 1) return seg_ptr[at + 1] > n ? at : -1;
    hi = min(hi, at + stride);
    lo = at;
  }
  return -1;
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

}  // namespace spmm
