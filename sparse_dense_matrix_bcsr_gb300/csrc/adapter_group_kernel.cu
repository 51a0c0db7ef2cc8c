// adapter_group_kernel.cu -- rows of a short batch sorted by their adapter
// (spmm_run_linear_adapters, spmm_adapters_grad).
//
// The tiled kernels work on rows of one segment, and a segment of one row costs them
// as much as one of 64: the gradient of 432 segments of one row, 4 adapters of rank 8,
// through 3880 x 16048 took 1004 us.  A batch with more segments than adapters is
// therefore sorted first where that pays (see the rules at the calls): one CTA gives
// every row its place (rows of adapter 0, of 1, ..., then those without, each in the
// batch's order, so the sums' order is fixed), X and dY are copied to their places,
// the kernels run on one segment per adapter, and Y or dX is copied back: 66 us.  The
// places come from a bitonic sort, 1024 rows one a thread (comparing every row with
// every other took 30 us longer for 1000 rows).
#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kSortThreads = kGroupRows;
static_assert(kGroupRows == 1024, "adapter and row in 32 bits, a thread a row");
constexpr int kCopyThreads = 256;

// The last s with ptr[s] <= n, -1 if there is none; n_seg of them.
__device__ __forceinline__ int32_t last_at(const int64_t *ptr, int32_t n_seg, int32_t n) {
  int32_t lo = -1, hi = n_seg;
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (ptr[mid] <= n)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kSortThreads) adapter_group_kernel(const AdapterGroupParams p) {
  __shared__ uint32_t buf[kGroupRows];
  __shared__ int64_t ptr[kGroupRows];
  __shared__ int32_t heads[kSortThreads / 32], rows[kSortThreads / 32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const bool few = p.n_seg <= kGroupRows;
  if (few && t < p.n_seg) ptr[t] = p.seg_ptr[t];
  __syncthreads();
  // the row's adapter (n_adapters for none) above its number: sorted, both in order
  uint32_t v = 0xffffffffu;
  if (t < p.N) {
    const int32_t s = last_at(few ? ptr : p.seg_ptr, p.n_seg, t);
    int32_t a = -1;
    if (s >= 0 && t < p.seg_ptr[s + 1]) a = checked_adapter(p.seg_adapter[s], p.n_adapters, p.status);
    v = static_cast<uint32_t>(a < 0 ? p.n_adapters : a) * kGroupRows + t;
  }
  // bitonic sort, one value a thread; partners within a warp by shuffles
  for (int size = 2; size <= kGroupRows; size *= 2) {
    for (int d = size / 2; d > 0; d /= 2) {
      uint32_t other;
      if (d >= 32) {
        __syncthreads();
        buf[t] = v;
        __syncthreads();
        other = buf[t ^ d];
      } else {
        other = __shfl_xor_sync(0xffffffffu, v, d);
      }
      const bool low = ((t & size) == 0) == ((t & d) == 0);
      v = low ? min(v, other) : max(v, other);
    }
  }
  __syncthreads();
  buf[t] = v;
  __syncthreads();
  const int32_t key = static_cast<int32_t>(v / kGroupRows);
  if (t < p.N) p.place[v % kGroupRows] = t;
  const bool has = t < p.N && key < p.n_adapters;
  const bool head = has && (t == 0 || static_cast<int32_t>(buf[t - 1] / kGroupRows) != key);
  const uint32_t vote = __ballot_sync(0xffffffffu, head);
  const int32_t mine = __popc(__ballot_sync(0xffffffffu, has));
  if (lane == 0) {
    heads[warp] = __popc(vote);
    rows[warp] = mine;
  }
  __syncthreads();
  int32_t before = 0, groups = 0, with = 0;
  for (int w = 0; w < kSortThreads / 32; ++w) {
    before += w < warp ? heads[w] : 0;
    groups += heads[w];
    with += rows[w];
  }
  if (head) {
    const int32_t g = before + __popc(vote & ((1u << lane) - 1));
    p.group_ptr[g] = t;
    p.group_adapter[g] = key;
  }
  for (int g = groups + t; g <= p.n_groups; g += kSortThreads) {
    p.group_ptr[g] = with;
    if (g < p.n_groups) p.group_adapter[g] = -1;
  }
}

// dst[place[n]] = src[n], or (back) dst[n] = src[place[n]], rows of 16-byte words.
struct MoveRows {
  const uint4 *src[2];
  uint4 *dst[2];
  int64_t words[2];
};
__global__ void __launch_bounds__(kCopyThreads) adapter_move_rows_kernel(const MoveRows m, const int32_t *__restrict__ place,
                                                                         bool back) {
  const int w = blockIdx.y;
  const int64_t n = blockIdx.x, at = place[n], words = m.words[w];
  const uint4 *__restrict__ src = m.src[w] + (back ? at : n) * words;
  uint4 *__restrict__ dst = m.dst[w] + (back ? n : at) * words;
  for (int64_t i = threadIdx.x; i < words; i += 4 * kCopyThreads) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kCopyThreads < words) v[u] = src[i + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kCopyThreads < words) dst[i + u * kCopyThreads] = v[u];
  }
}

}  // namespace

cudaError_t launch_adapter_group(const AdapterGroupParams &p, const void *X, void *xs, int64_t k, const void *dY, void *dys,
                                 int64_t m, cudaStream_t s) {
  adapter_group_kernel<<<1, kSortThreads, 0, s>>>(p);
  const MoveRows rows{{static_cast<const uint4 *>(X), static_cast<const uint4 *>(dY)},
                      {static_cast<uint4 *>(xs), static_cast<uint4 *>(dys)},
                      {k / 8, m / 8}};
  adapter_move_rows_kernel<<<dim3(static_cast<unsigned>(p.N), dY ? 2 : 1), kCopyThreads, 0, s>>>(rows, p.place, false);
  return cudaGetLastError();
}

cudaError_t launch_adapter_ungroup(const int32_t *place, int64_t N, const void *src, void *dst, int64_t row_bytes,
                                   cudaStream_t s) {
  const MoveRows rows{{static_cast<const uint4 *>(src)}, {static_cast<uint4 *>(dst)}, {row_bytes / 16}};
  adapter_move_rows_kernel<<<static_cast<unsigned>(N), kCopyThreads, 0, s>>>(rows, place, true);
  return cudaGetLastError();
}

}  // namespace spmm
