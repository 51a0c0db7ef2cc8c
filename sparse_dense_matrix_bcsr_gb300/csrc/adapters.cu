// adapters.cu -- low-rank adapters of many requests beside the shared
// block-sparse projection (spmm_run_linear_adapters, spmm_adapters_grad):
//   h[n] = scale[a] * D_a x[n],   y[n] = W x[n] + U_a h[n]
// with a the adapter of row n's segment, D_a rank x k and U_a m x rank.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "segments.cuh"

namespace spmm {
namespace {

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 p;
    if constexpr (BF16)
      p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[i]));
    else
      p = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// ---------------------------------------------------------------- down projection, a few rows per segment
// h[n][j] = scale * <D_a[j], x[n]> in fp32.  One block per (row that starts a
// run, group of kShrinkRanks ranks): a run is the rows of one segment within 4
// consecutive rows, so a row of D is read once for up to 4 rows of X and every
// single-row request still has its own block.  The block's warps take 256-column
// pieces of k in turn and add their sums in warp order.
constexpr int kShrinkThreads = 256;
constexpr int kShrinkWarps = kShrinkThreads / 32;
constexpr int kShrinkRanks = 4;
constexpr int kShrinkRows = 4;

template <bool BF16, int ROWS>
__device__ __forceinline__ void shrink_run(const uint4 *__restrict__ D, const uint4 *__restrict__ X, int32_t k8, int rows,
                                           float (&acc)[kShrinkRanks][ROWS]) {
#pragma unroll(ROWS == 1 ? 3 : 1)
  for (int32_t c = threadIdx.x; c < k8; c += kShrinkThreads) {
    uint4 w[kShrinkRanks], x[ROWS];
#pragma unroll
    for (int j = 0; j < kShrinkRanks; ++j) w[j] = D[static_cast<int64_t>(j) * k8 + c];
#pragma unroll
    for (int t = 0; t < ROWS; ++t)
      if (t < rows) x[t] = X[static_cast<int64_t>(t) * k8 + c];
    float wf[kShrinkRanks][8];
#pragma unroll
    for (int j = 0; j < kShrinkRanks; ++j) unpack8<BF16>(w[j], wf[j]);
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
      if (t >= rows) continue;
      float xf[8];
      unpack8<BF16>(x[t], xf);
#pragma unroll
      for (int j = 0; j < kShrinkRanks; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][t] = fmaf(wf[j][i], xf[i], acc[j][t]);
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kShrinkThreads, 3) shrink_rows_kernel(const AdapterParams p) {
  grid_launch_dependents();  // the projection may set up and run its shared product beside this
  const int64_t n = blockIdx.x;
  const RowSegment seg = find_row(p.seg_ptr, p.seg_adapter, p.n_seg, p.n_adapters, n, p.status);
  const int32_t a = seg.adapter;
  const int64_t group = n / kShrinkRows * kShrinkRows;
  if (a < 0 || n != max(seg.begin, group)) return;
  const int rows = static_cast<int>(min(min(seg.end, static_cast<int64_t>(p.N)), group + kShrinkRows) - n);
  const int32_t j0 = blockIdx.y * kShrinkRanks;
  const int32_t k8 = p.K / 8;
  const uint4 *D = static_cast<const uint4 *>(p.down) + (static_cast<int64_t>(a) * p.rank + j0) * k8;
  const uint4 *X = static_cast<const uint4 *>(p.X) + n * k8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float sums[kShrinkWarps][kShrinkRanks][kShrinkRows];
  if (rows == 1) {
    float acc[kShrinkRanks][1] = {};
    shrink_run<BF16, 1>(D, X, k8, 1, acc);
#pragma unroll
    for (int j = 0; j < kShrinkRanks; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j][0] += __shfl_xor_sync(0xffffffffu, acc[j][0], o);
      if (lane == 0) sums[warp][j][0] = acc[j][0];
    }
  } else {
    float acc[kShrinkRanks][kShrinkRows] = {};
    shrink_run<BF16, kShrinkRows>(D, X, k8, rows, acc);
#pragma unroll
    for (int j = 0; j < kShrinkRanks; ++j)
#pragma unroll
      for (int t = 0; t < kShrinkRows; ++t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[j][t] += __shfl_xor_sync(0xffffffffu, acc[j][t], o);
        if (lane == 0) sums[warp][j][t] = acc[j][t];
      }
  }
  __syncthreads();
  const int t = threadIdx.x / kShrinkRanks, j = threadIdx.x % kShrinkRanks;
  if (t < rows) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kShrinkWarps; ++w) v += sums[w][j][t];
    p.H[(n + t) * p.rank + j0 + j] = v * p.scale[a];
  }
}

}  // namespace

cudaError_t launch_shrink(const AdapterParams &p, bool bf16, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.N), static_cast<unsigned>(p.rank / kShrinkRanks));
  if (bf16)
    shrink_rows_kernel<true><<<grid, kShrinkThreads, 0, s>>>(p);
  else
    shrink_rows_kernel<false><<<grid, kShrinkThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace spmm
