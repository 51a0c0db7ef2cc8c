// adapter_wgrad_kernel.cu -- gradients of the adapters' weights
// (spmm_adapters_grad):
//   d_up_a[f][i]   = sum over rows n of adapter a of dY[n][f] * H[n][i]
//   d_down_a[i][f] = sum over rows n of adapter a of  X[n][f] * dH[n][i]
// Both are V^T S with V an N x F matrix of activations and S N x rank, so one
// kernel does both: the rows are the MMA's K, 128 features of V the M operand
// and the ranks the N operand, both MN-major as they lie in memory.
//
// CTA = (128 features, adapter, share of the adapter's rows).  A stage is 64 rows
// of one segment (a TMA box may start at any row), so K never runs across a
// segment; the rows after a segment's end that the last box brings are zeroed in
// shared memory in both operands before the MMA, as neither operand may hold
// another request's infinities.  Every element of dY and X is read once, so HBM
// bounds the kernel; S is read again by every feature tile, from L2.  The
// stages of an adapter are dealt in turn to a cluster of up to 8 CTAs where the
// features alone give too few, and the cluster adds its fp32 sums in CTA order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kFeat = 128;            // features per CTA
constexpr int kK = 64;                // rows per stage
constexpr int kBox = kK * 128;        // one box: 64 rows x 64 columns
constexpr int kVBytes = kFeat / 64 * kBox;
constexpr int kMaxQ = 4;
constexpr int kThreads = 192;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kEpiWarp0 = 2;
constexpr int kMiscBytes = 1024;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM

__host__ __device__ constexpr int rank16(int rank) { return (rank + 15) / 16 * 16; }
__host__ __device__ constexpr int rank_boxes(int rank) { return (rank + 63) / 64; }
__host__ __device__ constexpr int part_pitch(int rank) { return rank16(rank) + 4; }

struct Misc {
  uint64_t full[kMaxQ], empty[kMaxQ], acc_full;
  int32_t rows[kMaxQ];  // rows of the stage, 0: no more stages
  uint32_t tmem;
  int32_t any;          // the CTA had a stage
  volatile int32_t abort_flag;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float v) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) adapter_wgrad_kernel(const __grid_constant__ AdapterWgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int boxes = rank_boxes(p.rank);
  const int stage_bytes = kVBytes + boxes * kBox;
  Misc *mi = reinterpret_cast<Misc *>(smem + p.q * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t part = blockIdx.x % p.split;
  const int32_t tile = blockIdx.x / p.split;
  const bool up = tile < p.up_tiles;
  const int32_t f0 = (up ? tile : tile - p.up_tiles) * kFeat;
  const int32_t F = up ? p.M : p.K;
  const int32_t a = blockIdx.y;
  const int n16 = rank16(p.rank);
  uint32_t tmem_cols = 32;
  while (static_cast<int>(tmem_cols) < n16) tmem_cols <<= 1;

  if (threadIdx.x == 0) {
    for (int q = 0; q < p.q; ++q) {
      mbar_init(smem_addr(&mi->full[q]), 1);
      mbar_init(smem_addr(&mi->empty[q]), 1);
    }
    mbar_init(smem_addr(&mi->acc_full), 2);
    mi->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&mi->tmem), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = mi->tmem;

  if (warp == kTmaWarp) {
    const CUtensorMap *tmV = up ? &p.tm_dy : &p.tm_x;
    const CUtensorMap *tmS = up ? &p.tm_h : &p.tm_dh;
    uint32_t stage = 0, phase = 0;
    int64_t seq = 0;
    int32_t turn = 0;  // whose turn the next stage of the adapter is
    bool ok = true;
    auto claim = [&]() -> bool {
      const bool r = mbar_wait_warp(smem_addr(&mi->empty[stage]), phase ^ 1u, p.wait_limit_ns);
      return __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
    };
    auto advance = [&]() {
      ++seq;
      if (++stage == static_cast<uint32_t>(p.q)) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // the adapter's segments among 32, one a lane
    auto walk = [&](int64_t begin, int64_t end, int32_t adapter) {
      begin = max(begin, int64_t{0});
      end = min(end, static_cast<int64_t>(p.N));
      uint32_t todo = __ballot_sync(0xffffffffu, begin < end && adapter == a);
      while (todo && ok) {
        const int i = __ffs(todo) - 1;
        todo &= todo - 1;
        const int32_t sb = __shfl_sync(0xffffffffu, static_cast<int32_t>(begin), i);
        const int32_t se = __shfl_sync(0xffffffffu, static_cast<int32_t>(end), i);
        for (int32_t n = sb; n < se; n = se - n > kK ? n + kK : se) {
          const bool take = turn == part;
          if (++turn == p.split) turn = 0;
          if (!take) continue;
          ok = claim();
          if (!ok) break;
          if (lane == 0) {
            mi->rows[stage] = min(se - n, kK);
            const uint32_t fb = smem_addr(&mi->full[stage]);
            const uint32_t st = smem_addr(smem + stage * stage_bytes);
            mbar_arrive_expect_tx(fb, stage_bytes);
            tma_load_2d(st, tmV, fb, f0, n);
            tma_load_2d(st + kBox, tmV, fb, f0 + 64, n);
            for (int c = 0; c < boxes; ++c) tma_load_2d(st + kVBytes + c * kBox, tmS, fb, c * 64, n);
          }
          __syncwarp();
          advance();
        }
      }
    };
    if (p.n_seg <= kFewSegments) {
      const FewSegments few(p.seg_ptr, p.seg_adapter, p.n_seg);
#pragma unroll
      for (int g = 0; g < kFewGroups; ++g) walk(few.begin[g], few.end[g], few.adapter[g]);
    } else {
      for (int32_t base = 0; base < p.n_seg && ok; base += 32) {
        const int32_t s = base + lane;
        const bool in = s < p.n_seg;
        walk(in ? p.seg_ptr[s] : 0, in ? p.seg_ptr[s + 1] : 0, in ? p.seg_adapter[s] : -1);
      }
    }
    if (ok) {
      ok = claim();
      if (ok && lane == 0) {
        mi->rows[stage] = 0;
        mbar_arrive(smem_addr(&mi->full[stage]));
      }
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
      // let the copies in flight land before the block ends
      for (int64_t i = seq > p.q ? seq - p.q : 0; i < seq; ++i)
        mbar_wait(smem_addr(&mi->full[i % p.q]), static_cast<uint32_t>((i / p.q) & 1), 1000000ull);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = idesc_f16(BF16, /*a_mn_major=*/true, /*b_mn_major=*/true, kFeat, static_cast<uint32_t>(n16));
    uint32_t stage = 0, phase = 0;
    bool any = false, ok = true;
    while (true) {
      const bool r = mbar_wait_warp(smem_addr(&mi->full[stage]), phase, p.wait_limit_ns);
      ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
      if (!ok) break;
      const int32_t rows = mi->rows[stage];
      if (rows == 0) break;
      const int steps = (rows + 15) / 16;
      if (rows % 16 != 0) {
        // rows [rows, 16 * steps) belong to another segment: a swizzled row is
        // 128 contiguous bytes of its box, so whole rows can be cleared
        const int n = (16 * steps - rows) * 8;
        uint8_t *st = smem + stage * stage_bytes + rows * 128;
        for (int box = 0; box < kFeat / 64 + boxes; ++box)
          for (int u = lane; u < n; u += 32) *reinterpret_cast<uint4 *>(st + box * kBox + u * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        tc_fence_after_sync();
        const uint32_t st = smem_addr(smem + stage * stage_bytes);
        const uint64_t v = smem_desc_sw128(st, kBox, 1024);
        const uint64_t s = smem_desc_sw128(st + kVBytes, kBox, 1024);
        for (int kk = 0; kk < steps; ++kk)
          umma_f16(tmem, smem_desc_add(v, kk * 2048), smem_desc_add(s, kk * 2048), idesc, (any || kk > 0) ? 1u : 0u);
        umma_commit(smem_addr(&mi->empty[stage]));
      }
      any = true;
      __syncwarp();
      if (++stage == static_cast<uint32_t>(p.q)) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0) {
      if (!ok) {
        atomicOr(p.status, kDevTimeout);
        mi->abort_flag = 1;
      }
      mi->any = any;
      mbar_arrive(smem_addr(&mi->acc_full));
      umma_commit(smem_addr(&mi->acc_full));
    }
  } else {
    const int sp = warp & 3;
    const int r = sp * 32 + lane;  // feature f0 + r
    const bool ok = mbar_wait_warp(smem_addr(&mi->acc_full), 0, p.wait_limit_ns);
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
    }
    tc_fence_after_sync();
    const bool any = ok && mi->any;
    float *sums = reinterpret_cast<float *>(smem);  // the stages are done with
    for (int c0 = 0; c0 < n16 && ok; c0 += 16) {
      uint32_t v[16];
      if (any) {
        tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(sp * 32) << 16) + c0, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0u;
      }
      float4 *dst = reinterpret_cast<float4 *>(sums + r * part_pitch(p.rank) + c0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                             __uint_as_float(v[4 * i + 3]));
    }
    tc_fence_before_sync();
  }
  if (p.split > 1)
    cluster_sync();  // every CTA of the cluster comes here, whatever happened before
  else
    __syncthreads();
  {
    const int feats = kFeat / p.split, r0 = part * feats;
    const uint32_t base = smem_addr(smem);
    const int units = p.rank / 8;
    for (int u = threadIdx.x; u < feats * units; u += kThreads) {
      // d_up: a feature's ranks are contiguous; d_down: a rank's features are
      const int r = r0 + (up ? u / units : u % feats), j = (up ? u % units : u / feats) * 8;
      if (f0 + r >= F) continue;
      float o[8];
      cluster_sum8(base + (r * part_pitch(p.rank) + j) * 4, p.split, o);
      if (up) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = round16<BF16>(o[2 * i]) | static_cast<uint32_t>(round16<BF16>(o[2 * i + 1])) << 16;
        *reinterpret_cast<uint4 *>(p.d_up + (static_cast<int64_t>(a) * F + f0 + r) * p.rank + j) =
            make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          p.d_down[(static_cast<int64_t>(a) * p.rank + j + i) * F + f0 + r] = round16<BF16>(o[i]);
      }
    }
  }
  if (p.split > 1) cluster_sync();  // the others may still read this CTA's sums
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace

cudaError_t launch_adapter_wgrad(AdapterWgradParams p, int num_sms, bool bf16, cudaStream_t s) {
  p.up_tiles = (p.M + kFeat - 1) / kFeat;
  const int64_t tiles = p.up_tiles + (p.K + kFeat - 1) / kFeat;
  // adapters that can have rows, and CTAs per tile (a cluster) that keep about
  // two CTAs per SM busy with at least four stages each
  const int64_t active = p.n_seg < p.n_adapters ? (p.n_seg > 0 ? p.n_seg : 1) : p.n_adapters;
  p.split = 1;
  while (p.split < 8 && tiles * active * p.split < 2ll * num_sms && p.N >= 8ll * kK * active * p.split) p.split *= 2;
  const int stage = kVBytes + rank_boxes(p.rank) * kBox;
  p.q = (kSmemLimit - kMiscBytes - 1024) / stage;
  if (p.q > kMaxQ) p.q = kMaxQ;
  const int smem = p.q * stage + kMiscBytes + 1024;
  auto kern = bf16 ? adapter_wgrad_kernel<true> : adapter_wgrad_kernel<false>;
  static std::atomic<uint64_t> smem_set[2];
  cudaError_t e = set_smem_limit_once(kern, kSmemLimit, smem_set[bf16 ? 1 : 0]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split), static_cast<unsigned>(p.n_adapters));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(p.split);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace spmm
