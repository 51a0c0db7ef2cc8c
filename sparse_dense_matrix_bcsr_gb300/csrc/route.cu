// route.cu -- tokens sorted by expert and back (spmm_route_* in include/spmm.h).
//
// A routing is T x topk expert ids; entry i = t * topk + j.  The stable counting
// sort gives every kept entry its slot: entries of expert 0 first, each
// expert's in entry order.  Rows then move by the slots alone:
//   gather        out[position[t, j]] = x[t]
//   combine       out[t] = sum_j w[t, j] * y[position[t, j]]
//   combine_grad  dy[position[t, j]] = w[t, j] * dout[t],  dw[t, j] = <dout[t], y[position[t, j]]>
// and the gradient of gather is combine with unit weights.  Everything here
// moves bytes: a row is read once and written once however many experts it
// goes to, so the HBM rate is the bound for prompts and launch plus one memory
// round trip for decoding batches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace spmm {
namespace {

// ---------------------------------------------------------------- sort
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

// Number of each expert's ids in every chunk: counts[chunk][expert].
template <int STEPS>
__global__ void __launch_bounds__(kSortThreads) route_count_kernel(const int32_t *__restrict__ ids, int64_t n, int32_t E,
                                                                   int32_t *__restrict__ counts) {
  extern __shared__ int32_t hist[];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kSortThreads * STEPS);
  int32_t id[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t q = base + i * kSortThreads + threadIdx.x;
    id[i] = q < n ? ids[q] : -1;
  }
  for (int e = threadIdx.x; e < E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (static_cast<uint32_t>(id[i]) < static_cast<uint32_t>(E)) atomicAdd(&hist[id[i]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
  grid_launch_dependents();
}

// Long lists: the counts of each expert summed over the chunks before, in place, and
// over all of them in a row of their own.  A block takes 32 experts, a warp a share
// of the chunks.
constexpr int kScanAtOnce = 8;
__global__ void __launch_bounds__(kSortThreads) route_scan_kernel(int32_t *__restrict__ counts, int32_t n_chunks, int32_t E) {
  __shared__ int32_t part[kSortWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t e = blockIdx.x * 32 + lane;
  const int32_t begin = static_cast<int32_t>(static_cast<int64_t>(n_chunks) * warp / kSortWarps);
  const int32_t end = static_cast<int32_t>(static_cast<int64_t>(n_chunks) * (warp + 1) / kSortWarps);
  grid_dependency_wait();  // the counts
  int32_t sum = 0;
  if (e < E) {
#pragma unroll kScanAtOnce
    for (int32_t c = begin; c < end; ++c) sum += counts[static_cast<int64_t>(c) * E + e];
  }
  part[warp][lane] = sum;
  __syncthreads();
  int32_t before = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) before += w < warp ? part[w][lane] : 0;
  if (e < E) {
    if (warp == kSortWarps - 1) counts[static_cast<int64_t>(n_chunks) * E + e] = before + sum;
    for (int32_t c = begin; c < end; c += kScanAtOnce) {
      int32_t v[kScanAtOnce];
#pragma unroll
      for (int i = 0; i < kScanAtOnce; ++i) v[i] = c + i < end ? counts[static_cast<int64_t>(c + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanAtOnce; ++i) {
        if (c + i < end) counts[static_cast<int64_t>(c + i) * E + e] = before;
        before += v[i];
      }
    }
  }
  grid_launch_dependents();
}

// Slots of one chunk's entries (STEPS * 32 consecutive ids per warp).  An
// entry's slot is its expert's offset (a scan of all counts), plus the expert's
// entries in earlier chunks, in earlier warps' parts of this chunk, and before
// it in its own warp's part; no atomic decides an order, so the sort is stable
// and the same every time.  Up to kRouteScanChunks chunks each block adds up the chunks'
// counts itself (chunks x E words out of L2); above, a kernel between does it once for all
// (64 experts, without / with it: 131072 ids 7.5 / 8.1 us, 262144 10.0 / 7.4, 2^20 43 / 16, 2^24
// 4160 / 184).  A single
// chunk needs no counts from a kernel before it, which is what a decoding batch
// takes: its length sets STEPS, so that 96 ids are one step and not sixteen.
template <int STEPS>
__global__ void __launch_bounds__(kSortThreads)
    route_place_kernel(const int32_t *__restrict__ ids, int64_t n, int32_t E, int32_t n_chunks,
                       const int32_t *__restrict__ counts, int64_t *__restrict__ offsets,
                       int32_t *__restrict__ order, int32_t *__restrict__ position) {
  extern __shared__ int32_t smem[];
  int32_t *part = smem;                    // [kSortWarps][E]: entries of each expert in each warp's part
  int32_t *first = smem + kSortWarps * E;  // [E]: first slot of this chunk's entries of each expert
  __shared__ int64_t warp_sum[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = blockIdx.x;
  const int64_t base = static_cast<int64_t>(chunk) * (kSortThreads * STEPS) + warp * (32 * STEPS);

  int32_t id[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t q = base + i * 32 + lane;
    const int32_t v = q < n ? ids[q] : -1;
    id[i] = static_cast<uint32_t>(v) < static_cast<uint32_t>(E) ? v : -1;
  }
  for (int e = threadIdx.x; e < kSortWarps * E; e += kSortThreads) part[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (id[i] >= 0) atomicAdd(&part[warp * E + id[i]], 1);
  grid_dependency_wait();  // the counts of a kernel before this one
  __syncthreads();
  // scan over experts, kSortThreads at a time
  int64_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    int64_t total = 0, before = 0;
    if (e < E) {
      int32_t mine = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {  // warps' parts -> exclusive prefix
        const int32_t c = part[w * E + e];
        part[w * E + e] = mine;
        mine += c;
      }
      if (n_chunks == 1) {
        total = mine;
      } else if (n_chunks > kRouteScanChunks) {
        total = counts[static_cast<int64_t>(n_chunks) * E + e];
        before = counts[static_cast<int64_t>(chunk) * E + e];
      } else {
#pragma unroll 8
        for (int c = 0; c < n_chunks; ++c) {
          const int32_t v = counts[static_cast<int64_t>(c) * E + e];
          total += v;
          if (c < chunk) before += v;
        }
      }
    }
    int64_t incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t pre = carry;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int64_t s = warp_sum[w];
      if (w < warp) pre += s;
      carry += s;
    }
    if (e < E) {
      first[e] = static_cast<int32_t>(pre + incl - total + before);
      if (chunk == 0) offsets[e] = pre + incl - total;
    }
    __syncthreads();
  }
  const int64_t kept = carry;
  if (chunk == 0 && threadIdx.x == 0) offsets[E] = kept;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t q = base + i * 32 + lane;
    const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int32_t slot = -1;
    if (id[i] >= 0) slot = first[id[i]] + part[warp * E + id[i]] + rank;
    if (i + 1 < STEPS) {
      __syncwarp();
      if (id[i] >= 0 && rank == 0) part[warp * E + id[i]] += __popc(same);
      __syncwarp();
    }
    if (q < n) {
      position[q] = slot;
      if (slot >= 0) order[slot] = static_cast<int32_t>(q);
      if (q >= kept) order[q] = -1;  // slots that no entry takes
    }
  }
}

// ---------------------------------------------------------------- rows
// A row is moved VEC elements of T per lane and step: as 16-byte words where
// rows start on 16 bytes, else as single elements.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
  using type = uint4;
};
template <>
struct Word<4> {
  using type = uint32_t;
};
template <>
struct Word<2> {
  using type = uint16_t;
};
template <typename T, int VEC>
using RowWord = typename Word<sizeof(T) * VEC>::type;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const RowWord<T, VEC> &w, float (&f)[VEC]) {
  const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
  for (int c = 0; c < VEC; ++c) f[c] = to_f32(e[c]);
}
template <typename T, int VEC>
__device__ __forceinline__ RowWord<T, VEC> pack(const float (&f)[VEC]) {
  RowWord<T, VEC> w;
  T *e = reinterpret_cast<T *>(&w);
#pragma unroll
  for (int c = 0; c < VEC; ++c) e[c] = from_f32<T>(f[c]);
  return w;
}

constexpr int kRowThreads = 256;
constexpr int kRowSteps = 4;  // packs per lane and work item: 2 KB of a row in flight per warp

// Work item = (token, 32 * kRowSteps packs of its row), one warp each; the
// blocks past `item_blocks` write zeros to the rows that no entry takes.
template <typename T, int VEC>
__global__ void __launch_bounds__(kRowThreads)
    route_gather_kernel(const T *__restrict__ x, const int32_t *__restrict__ position, const int64_t *__restrict__ kept_ptr,
                        T *__restrict__ out, int64_t T_, int32_t topk, int64_t d, int32_t n_parts, int64_t item_blocks) {
  using P = RowWord<T, VEC>;
  const int64_t packs = d / VEC;
  const int lane = threadIdx.x & 31;
  const int64_t rows = T_ * topk;
  if (blockIdx.x >= item_blocks) {
    const int64_t kept = min(max(*kept_ptr, int64_t{0}), rows);
    const P zero{};
    P *dst = reinterpret_cast<P *>(out) + kept * packs;
    const int64_t total = (rows - kept) * packs;
    for (int64_t i = (blockIdx.x - item_blocks) * kRowThreads + threadIdx.x; i < total;
         i += (gridDim.x - item_blocks) * kRowThreads)
      dst[i] = zero;
    return;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / n_parts;
  if (t >= T_) return;
  const int64_t p0 = (item - t * n_parts) * (32 * kRowSteps) + lane;
  const int32_t my_pos = lane < topk ? position[t * topk + lane] : -1;
  const P *src = reinterpret_cast<const P *>(x) + t * packs;
  P v[kRowSteps];
#pragma unroll
  for (int i = 0; i < kRowSteps; ++i)
    if (p0 + 32 * i < packs) v[i] = src[p0 + 32 * i];
  for (int j = 0; j < topk; ++j) {
    const int32_t pos = __shfl_sync(0xffffffffu, my_pos, j);
    if (pos < 0 || pos >= rows) continue;
    P *dst = reinterpret_cast<P *>(out) + static_cast<int64_t>(pos) * packs;
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i)
      if (p0 + 32 * i < packs) dst[p0 + 32 * i] = v[i];
  }
}

// out[t] = sum over j (in order, fp32, one rounding) of w[t, j] * y[position[t, j]];
// dropped entries are skipped, whatever their weight holds.  A block takes a
// part of one token's row, STEPS packs per thread, and has eight loads of y in
// flight per thread (a warp per part that fetched its positions by lane and
// branched on each entry had 4.9 TB/s for 32K tokens with six entries each).
constexpr int kCombineThreads = 128;
template <typename T, int VEC, int STEPS>
__global__ void __launch_bounds__(kCombineThreads)
    route_combine_kernel(const T *__restrict__ y, const int32_t *__restrict__ position, const float *__restrict__ weights,
                         T *__restrict__ out, int64_t T_, int32_t topk, int64_t d, int32_t n_parts) {
  using P = RowWord<T, VEC>;
  constexpr int kGroup = 8 / STEPS;  // entries at a time
  const int64_t packs = d / VEC;
  const int64_t rows = T_ * topk;
  const int64_t t = blockIdx.x / n_parts;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x - t * n_parts) * (kCombineThreads * STEPS) + threadIdx.x;
  float acc[STEPS][VEC] = {};
  for (int j0 = 0; j0 < topk; j0 += kGroup) {
    int32_t pos[kGroup];
    float w[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const bool in = j0 + j < topk;
      pos[j] = in ? __ldg(position + t * topk + j0 + j) : -1;
      w[j] = !in ? 0.0f : weights ? __ldg(weights + t * topk + j0 + j) : 1.0f;
      if (pos[j] >= rows) pos[j] = -1;
    }
    P v[kGroup][STEPS];
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        if (pos[j] >= 0 && p0 + kCombineThreads * i < packs)
          v[j][i] = reinterpret_cast<const P *>(y)[pos[j] * packs + p0 + kCombineThreads * i];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      if (pos[j] < 0) continue;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        float f[VEC];
        unpack<T, VEC>(v[j][i], f);
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[i][c] = fmaf(w[j], f[c], acc[i][c]);
      }
    }
  }
  P *dst = reinterpret_cast<P *>(out) + t * packs;
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (p0 + kCombineThreads * i < packs) dst[p0 + kCombineThreads * i] = pack<T, VEC>(acc[i]);
}

// One block per token: dout[t] is read once for all of its entries of a group
// of kGradGroup, y's rows once, dy's rows written once; dw by a block sum in a
// fixed order.  The blocks past T_ write zeros to dy's rows that no entry takes.
constexpr int kGradThreads = 128;
constexpr int kGradGroup = 4;
template <typename T, int VEC>
__global__ void __launch_bounds__(kGradThreads)
    route_combine_grad_kernel(const T *__restrict__ dout, const T *__restrict__ y, const int32_t *__restrict__ position,
                              const float *__restrict__ weights, const int64_t *__restrict__ kept_ptr, T *__restrict__ dy,
                              float *__restrict__ dw, int64_t T_, int32_t topk, int64_t d) {
  using P = RowWord<T, VEC>;
  const int64_t packs = d / VEC;
  const int64_t rows = T_ * topk;
  if (blockIdx.x >= T_) {
    const int64_t kept = min(max(*kept_ptr, int64_t{0}), rows);
    const P zero{};
    P *dst = reinterpret_cast<P *>(dy) + kept * packs;
    const int64_t total = (rows - kept) * packs;
    for (int64_t i = (blockIdx.x - T_) * kGradThreads + threadIdx.x; i < total; i += (gridDim.x - T_) * kGradThreads)
      dst[i] = zero;
    return;
  }
  __shared__ float sums[kGradThreads / 32][kGradGroup];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const P *src = reinterpret_cast<const P *>(dout) + t * packs;
  for (int j0 = 0; j0 < topk; j0 += kGradGroup) {
    int32_t pos[kGradGroup];
    float w[kGradGroup], dot[kGradGroup];
#pragma unroll
    for (int j = 0; j < kGradGroup; ++j) {
      pos[j] = j0 + j < topk ? position[t * topk + j0 + j] : -1;
      if (pos[j] >= rows) pos[j] = -1;
      w[j] = j0 + j < topk ? (weights ? weights[t * topk + j0 + j] : 1.0f) : 0.0f;
      dot[j] = 0.0f;
    }
    for (int64_t p = threadIdx.x; p < packs; p += kGradThreads) {
      float g[VEC];
      unpack<T, VEC>(src[p], g);
      P v[kGradGroup];
#pragma unroll
      for (int j = 0; j < kGradGroup; ++j)
        if (pos[j] >= 0) v[j] = reinterpret_cast<const P *>(y)[static_cast<int64_t>(pos[j]) * packs + p];
#pragma unroll
      for (int j = 0; j < kGradGroup; ++j) {
        if (pos[j] < 0) continue;
        float yf[VEC], o[VEC];
        unpack<T, VEC>(v[j], yf);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          dot[j] = fmaf(g[c], yf[c], dot[j]);
          o[c] = w[j] * g[c];
        }
        reinterpret_cast<P *>(dy)[static_cast<int64_t>(pos[j]) * packs + p] = pack<T, VEC>(o);
      }
    }
#pragma unroll
    for (int j = 0; j < kGradGroup; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) sums[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < kGradGroup && j0 + static_cast<int>(threadIdx.x) < topk) {
      float s = 0.0f;
#pragma unroll
      for (int wq = 0; wq < kGradThreads / 32; ++wq) s += sums[wq][threadIdx.x];
      dw[t * topk + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

constexpr int64_t kZeroBlocks = 152;

template <typename T, int VEC>
cudaError_t gather_rows(const RouteRows &r, cudaStream_t s) {
  const int64_t packs = r.d / VEC;
  const int32_t parts = static_cast<int32_t>((packs + 32 * kRowSteps - 1) / (32 * kRowSteps));
  const int64_t blocks = (r.T * parts + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t zero = r.T * r.topk < kZeroBlocks ? r.T * r.topk : kZeroBlocks;
  if (blocks + zero >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  route_gather_kernel<T, VEC><<<static_cast<unsigned>(blocks + zero), kRowThreads, 0, s>>>(
      static_cast<const T *>(r.src), r.position, r.kept, static_cast<T *>(r.dst), r.T, r.topk, r.d, parts, blocks);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t combine_rows(const RouteRows &r, cudaStream_t s) {
  const int64_t packs = r.d / VEC;
  // four packs a thread where tokens alone fill the GPU, one where a few tokens
  // leave latency as the bound
  const int steps = r.T >= 1024 ? 4 : 1;
  const int32_t parts = static_cast<int32_t>((packs + kCombineThreads * steps - 1) / (kCombineThreads * steps));
  if (r.T * parts >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  auto kern = steps == 4 ? route_combine_kernel<T, VEC, 4> : route_combine_kernel<T, VEC, 1>;
  kern<<<static_cast<unsigned>(r.T * parts), kCombineThreads, 0, s>>>(
      static_cast<const T *>(r.src), r.position, r.weights, static_cast<T *>(r.dst), r.T, r.topk, r.d, parts);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t grad_rows(const RouteRows &r, cudaStream_t s) {
  const int64_t zero = r.T * r.topk < kZeroBlocks ? r.T * r.topk : kZeroBlocks;
  route_combine_grad_kernel<T, VEC><<<static_cast<unsigned>(r.T + zero), kGradThreads, 0, s>>>(
      static_cast<const T *>(r.dout), static_cast<const T *>(r.src), r.position, r.weights, r.kept,
      static_cast<T *>(r.dst), r.dweights, r.T, r.topk, r.d);
  return cudaGetLastError();
}

// 16-byte words need rows of a multiple of 16 bytes from 16-byte aligned bases.
bool wide_rows(const RouteRows &r, int esize) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(r.src) | reinterpret_cast<uintptr_t>(r.dst) |
                      reinterpret_cast<uintptr_t>(r.dout);
  return p % 16 == 0 && (r.d * esize) % 16 == 0;
}

}  // namespace

// Up to kRouteOneChunk ids are one block's work, without counts in global memory;
// longer lists are cut into chunks of kRouteChunk.
int64_t route_chunks(int64_t n) { return n <= kRouteOneChunk ? 1 : (n + kRouteChunk - 1) / kRouteChunk; }

namespace {

template <int STEPS>
cudaError_t sort_ids(const int32_t *ids, int64_t n, int32_t n_experts, int64_t *offsets, int32_t *order, int32_t *position,
                     int32_t *counts, int64_t chunks, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_limit_once(route_place_kernel<STEPS>, (kSortWarps + 1) * kRouteMaxExperts * 4, smem_set);
  if (e != cudaSuccess) return e;
  if (chunks > 1) {
    route_count_kernel<STEPS><<<static_cast<unsigned>(chunks), kSortThreads, n_experts * 4, s>>>(ids, n, n_experts, counts);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = chunks > 1 ? 1 : 0;  // dependents of the kernel before
  if (chunks > kRouteScanChunks) {
    cfg.gridDim = dim3(static_cast<unsigned>((n_experts + 31) / 32));
    e = cudaLaunchKernelEx(&cfg, route_scan_kernel, counts, static_cast<int32_t>(chunks), n_experts);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(chunks));
  cfg.dynamicSmemBytes = static_cast<size_t>(kSortWarps + 1) * n_experts * 4;
  return cudaLaunchKernelEx(&cfg, route_place_kernel<STEPS>, ids, n, n_experts, static_cast<int32_t>(chunks),
                            static_cast<const int32_t *>(counts), offsets, order, position);
}

}  // namespace

cudaError_t launch_route_sort(const int32_t *ids, int64_t n, int32_t n_experts, int64_t *offsets, int32_t *order,
                              int32_t *position, int32_t *counts, cudaStream_t s) {
  const int64_t chunks = route_chunks(n);
  static_assert(kRouteChunk == 4 * kSortThreads && kRouteOneChunk == 16 * kSortThreads, "steps");
  if (chunks > 1 || (n > kSortThreads && n <= kRouteChunk))
    return sort_ids<4>(ids, n, n_experts, offsets, order, position, counts, chunks, s);
  if (n <= kSortThreads) return sort_ids<1>(ids, n, n_experts, offsets, order, position, counts, 1, s);
  return sort_ids<16>(ids, n, n_experts, offsets, order, position, counts, 1, s);
}

#define SPMM_ROUTE_ROWS(name)                                                                            \
  cudaError_t launch_route_##name(const RouteRows &r, int dtype, cudaStream_t s) {                      \
    if (r.T == 0) return cudaSuccess;                                                                   \
    if (dtype == 2) return wide_rows(r, 4) ? name##_rows<float, 4>(r, s) : name##_rows<float, 1>(r, s); \
    if (dtype == 1)                                                                                     \
      return wide_rows(r, 2) ? name##_rows<__nv_bfloat16, 8>(r, s) : name##_rows<__nv_bfloat16, 1>(r, s); \
    return wide_rows(r, 2) ? name##_rows<__half, 8>(r, s) : name##_rows<__half, 1>(r, s);               \
  }
SPMM_ROUTE_ROWS(gather)
SPMM_ROUTE_ROWS(combine)
SPMM_ROUTE_ROWS(grad)
#undef SPMM_ROUTE_ROWS

}  // namespace spmm
