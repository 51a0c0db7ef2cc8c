// adapter_decode_kernel.cu -- the projection with adapters for batches of few
// rows per adapter (decoding: one row a request), spmm_run_linear_adapters.
//
// CTA = one block row (64 output features) x a tile of 16, 32 or 64 rows of X.
// The shared product is y^T[64 x rows] = sum over stored blocks of blk * X^T:
// the block is the M = 64 operand and the rows of X the N operand of
// tcgen05.mma, both K-major as they lie, so a small batch costs small MMAs and
// 2-8 KB of X per block instead of a 256-row tile.  The adapters follow on the
// CUDA cores in fp32, since every row has its own U_a and an MMA would run for one
// row: the 64 rows of U_a that the block row needs are contiguous (64 * rank
// values), come by one bulk copy each through a ring of their own and are
// multiplied with h, kept in fp32, as they arrive.  A warp (two or four above 32
// ranks) takes a piece of up to 8 rows of one segment with a copy of U of its own, so 64 requests and one
// request of 64 rows keep all summing warps busy alike.  A row meets its own
// adapter alone.
//
// HBM bounds it: the blocks once (2 nnz bytes), each adapter's U once.  The ring
// of U starts filling, and the shared product runs, before the down projection's
// kernel has ended (a programmatic dependent launch); only h is waited for.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kBlk = 64;
constexpr int kBlkBytes = kBlk * kBlk * 2;
constexpr int kMaxQ = 8, kMaxQU = 32;
constexpr int kPiece = 8;               // rows of a segment that one warp takes
constexpr int kTmaWarp = 0, kMmaWarp = 1, kUpWarp = 2, kSumWarp0 = 4, kSumWarps = 8;
constexpr int kThreads = (kSumWarp0 + kSumWarps) * 32;
constexpr int kPitch = kBlk + 4;        // floats per row of y in shared memory
constexpr int kMiscBytes = 3072;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM
constexpr int kUpRing = 32 * 1024;

struct Misc {
  uint64_t full[kMaxQ], empty[kMaxQ], up_full[kMaxQU], up_empty[kMaxQU], acc_full, listed;
  TileSegment segs[kAdapterDecodeRows], pieces[kAdapterDecodeRows];
  int32_t n_pieces;
  uint32_t tmem;
  volatile int32_t abort_flag;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v;
    if constexpr (BF16)
      v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[i]));
    else
      v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ void sum_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory"); }

// y[row][feature] += U_a[feature] . h[row] for one piece, by one warp.  SPAN
// adjacent lanes share a feature, each with 8 of its ranks (SPAN is rank / 8
// rounded up to a power of two), so the warp reads U as contiguous 16-byte
// words and passes 2 * SPAN times over 32 / SPAN features; where several warps
// share a piece each takes passes [pass0, pass1).
template <bool BF16, int SPAN>
__device__ __forceinline__ void add_piece(const TileSegment s, const uint4 *__restrict__ U, const float *__restrict__ h,
                                          float *__restrict__ y, int rank, int sub, int subs) {
  const int pass0 = 2 * SPAN * sub / subs, pass1 = 2 * SPAN * (sub + 1) / subs;
  const int lane = threadIdx.x & 31, c = lane % SPAN, f0 = lane / SPAN;
  const int chunks = rank / 8;
  const bool on = c < chunks;
  auto load_h = [&](int n, float (&v)[8]) {
    const float4 *src = reinterpret_cast<const float4 *>(h + n * rank) + c * 2;
    const float4 a = on ? src[0] : make_float4(0, 0, 0, 0), b = on ? src[1] : make_float4(0, 0, 0, 0);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  };
  auto load_u = [&](int pass, float (&u)[8]) {
    const int f = pass * (32 / SPAN) + f0;
    unpack8<BF16>(on ? U[f * chunks + c] : make_uint4(0, 0, 0, 0), u);
  };
  auto add = [&](int n, int pass, const float (&u)[8], const float (&v)[8]) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) dot = fmaf(u[i], v[i], dot);
#pragma unroll
    for (int o = SPAN / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (c == 0) y[n * kPitch + pass * (32 / SPAN) + f0] += dot;
  };
  if (s.end - s.begin == 1) {
    float v[8];
    load_h(s.begin, v);
#pragma unroll 4
    for (int pass = pass0; pass < pass1; ++pass) {
      float u[8];
      load_u(pass, u);
      add(s.begin, pass, u, v);
    }
  } else {
    for (int pass = pass0; pass < pass1; ++pass) {
      float u[8];
      load_u(pass, u);
#pragma unroll 4
      for (int n = s.begin; n < s.end; ++n) {
        float v[8];
        load_h(n, v);
        add(n, pass, u, v);
      }
    }
  }
}

template <bool BF16, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads, 2)
    adapter_decode_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmX,
                          const AdapterDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kBlkBytes + p.tile * 128;
  const int slot_bytes = kBlk * p.rank * 2;
  uint8_t *ring = smem + p.q * stage_bytes;                                    // U
  float *h = reinterpret_cast<float *>(ring + p.qu * slot_bytes);              // [tile][rank]
  Misc *mi = reinterpret_cast<Misc *>(h + p.tile * p.rank);
  float *y = reinterpret_cast<float *>(smem);                                  // [tile][kPitch], once the stages are done with
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t br = blockIdx.x;
  const int32_t row0 = blockIdx.y * p.tile;
  const int32_t rows = min(p.N - row0, p.tile);
  const int32_t feats = min(p.M - br * kBlk, kBlk);
  const uint32_t tmem_cols = p.tile < 32 ? 32 : p.tile;
  // Every slot of U's ring belongs to the same summing warps each time round (a
  // warp that skipped uses of a slot could mistake an older phase of its
  // barrier for the one it waits for): as many groups as slots, or one warp each.
  const int groups = min(p.qu, kSumWarps), subs = kSumWarps / groups;
  const int64_t jb = p.block_row_ptr[br], je = p.block_row_ptr[br + 1];

  if (threadIdx.x == 0) {
    for (int q = 0; q < p.q; ++q) {
      mbar_init(smem_addr(&mi->full[q]), 1);
      mbar_init(smem_addr(&mi->empty[q]), 1);
    }
    for (int q = 0; q < p.qu; ++q) {
      mbar_init(smem_addr(&mi->up_full[q]), 1);
      mbar_init(smem_addr(&mi->up_empty[q]), subs);
    }
    mbar_init(smem_addr(&mi->acc_full), 1);
    mbar_init(smem_addr(&mi->listed), 1);
    mi->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmX);
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
    uint32_t stage = 0, phase = 0;
    int64_t seq = 0;
    bool ok = true;
    for (int64_t jbase = jb; jbase < je && ok; jbase += 32) {
      const int32_t my_col = jbase + lane < je ? p.block_col_idx[jbase + lane] : 0;
      const int cnt = static_cast<int>(min(je - jbase, int64_t{32}));
      for (int i = 0; i < cnt; ++i) {
        const int32_t bcol = __shfl_sync(0xffffffffu, my_col, i);
        const bool r = mbar_wait_warp(smem_addr(&mi->empty[stage]), phase ^ 1u, p.wait_limit_ns);
        ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = smem_addr(&mi->full[stage]);
          const uint32_t st = smem_addr(smem + stage * stage_bytes);
          mbar_arrive_expect_tx(fb, stage_bytes);
          tma_load_2d(st, &tmA, fb, 0, static_cast<int32_t>((jbase + i) * kBlk));
          tma_load_2d(st + kBlkBytes, &tmX, fb, bcol * kBlk, row0);
        }
        __syncwarp();
        ++seq;
        if (++stage == static_cast<uint32_t>(p.q)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
      for (int64_t i = seq > p.q ? seq - p.q : 0; i < seq; ++i)  // copies in flight land before the block ends
        mbar_wait(smem_addr(&mi->full[i % p.q]), static_cast<uint32_t>((i / p.q) & 1), 1000000ull);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = idesc_f16(BF16, false, false, kBlk, static_cast<uint32_t>(p.tile));
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int64_t j = jb; j < je; ++j) {
      const bool r = mbar_wait_warp(smem_addr(&mi->full[stage]), phase, p.wait_limit_ns);
      ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
      if (!ok) break;
      if (lane == 0) {
        tc_fence_after_sync();
        const uint32_t st = smem_addr(smem + stage * stage_bytes);
        const uint64_t a = smem_desc_sw128(st, 16, 1024), b = smem_desc_sw128(st + kBlkBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(tmem, smem_desc_add(a, kk * 32), smem_desc_add(b, kk * 32), idesc, (j > jb || kk > 0) ? 1u : 0u);
        umma_commit(smem_addr(&mi->empty[stage]));
      }
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
      umma_commit(smem_addr(&mi->acc_full));
    }
  } else if (warp == kUpWarp) {
    const int32_t n_segs = list_segments(p.seg_ptr, p.seg_adapter, p.n_seg, p.n_adapters, row0, row0 + rows, mi->segs,
                                         kAdapterDecodeRows, p.status);
    __syncwarp();
    int32_t n_pieces = 0;
    for (int32_t base = 0; base < n_segs; base += 32) {
      TileSegment s{-1, 0, 0, 0};
      if (base + lane < n_segs) s = mi->segs[base + lane];
      const int32_t count = (s.end - s.begin + kPiece - 1) / kPiece;
      int32_t incl = count;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      for (int32_t i = 0; i < count; ++i) {
        const int32_t at = n_pieces + incl - count + i;  // at most one per row
        if (at < kAdapterDecodeRows)
          mi->pieces[at] = TileSegment{s.adapter, s.begin + i * kPiece, min(s.begin + (i + 1) * kPiece, s.end), 0};
      }
      n_pieces += __shfl_sync(0xffffffffu, incl, 31);
    }
    n_pieces = min(n_pieces, kAdapterDecodeRows);
    if (lane == 0) mi->n_pieces = n_pieces;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&mi->listed));
    const uint32_t bytes = feats * p.rank * 2;
    bool ok = true;
    int32_t i = 0;
    for (; i < n_pieces; ++i) {
      const int slot = i % p.qu;
      const bool r = mbar_wait_warp(smem_addr(&mi->up_empty[slot]), (static_cast<uint32_t>(i / p.qu) & 1u) ^ 1u,
                                    p.wait_limit_ns);
      ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = smem_addr(&mi->up_full[slot]);
        mbar_arrive_expect_tx(fb, bytes);
        tma_bulk_load(smem_addr(ring + slot * slot_bytes),
                      static_cast<const uint16_t *>(p.up) +
                          (static_cast<int64_t>(mi->pieces[i].adapter) * p.M + br * kBlk) * p.rank,
                      bytes, fb);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
      for (int32_t j = i > p.qu ? i - p.qu : 0; j < i; ++j)
        mbar_wait(smem_addr(&mi->up_full[j % p.qu]), static_cast<uint32_t>(j / p.qu) & 1u, 1000000ull);
    }
  } else if (warp >= kSumWarp0) {
    const int tid = threadIdx.x - kSumWarp0 * 32;
    bool ok = true;
    if (warp < kSumWarp0 + 4) {
      // rows 16 s .. 16 s + 15 of the accumulator lie in lanes 32 s .. 32 s + 15
      const int sp = warp & 3;
      if (je > jb) {
        ok = mbar_wait_warp(smem_addr(&mi->acc_full), 0, p.wait_limit_ns);
        if (!ok && lane == 0) {
          atomicOr(p.status, kDevTimeout);
          mi->abort_flag = 1;
        }
        tc_fence_after_sync();
        for (int c0 = 0; c0 < p.tile && ok; c0 += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(sp * 32) << 16) + c0, v);
          tmem_ld_wait();
          if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) y[(c0 + i) * kPitch + sp * 16 + lane] = __uint_as_float(v[i]);
        }
        tc_fence_before_sync();
      } else {
        for (int i = tid; i < p.tile * kPitch; i += 128) y[i] = 0.0f;
      }
    } else {
      grid_dependency_wait();  // h; every block waits, so this kernel never ends before that one
      const float4 *src = reinterpret_cast<const float4 *>(p.H + static_cast<int64_t>(row0) * p.rank);
      for (int i = tid - 128; i < rows * p.rank / 4; i += 128) reinterpret_cast<float4 *>(h)[i] = src[i];
    }
    sum_warps_sync();
    ok = ok && mbar_wait_warp(smem_addr(&mi->listed), 0, p.wait_limit_ns);
    const int32_t n_pieces = ok ? mi->n_pieces : 0;
    const int sub = (warp - kSumWarp0) % subs;
    for (int32_t i = (warp - kSumWarp0) / subs; i < n_pieces; i += groups) {
      const int slot = i % p.qu;
      const bool r = mbar_wait_warp(smem_addr(&mi->up_full[slot]), static_cast<uint32_t>(i / p.qu) & 1u, p.wait_limit_ns);
      ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
      if (!ok) break;
      const TileSegment s = mi->pieces[i];
      const uint4 *U = reinterpret_cast<const uint4 *>(ring + slot * slot_bytes);
      if (p.rank == 8)
        add_piece<BF16, 1>(s, U, h, y, p.rank, sub, subs);
      else if (p.rank == 16)
        add_piece<BF16, 2>(s, U, h, y, p.rank, sub, subs);
      else if (p.rank <= 32)
        add_piece<BF16, 4>(s, U, h, y, p.rank, sub, subs);
      else if (p.rank <= 64)
        add_piece<BF16, 8>(s, U, h, y, p.rank, sub, subs);
      else
        add_piece<BF16, 16>(s, U, h, y, p.rank, sub, subs);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&mi->up_empty[slot]));
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
    }
    sum_warps_sync();
    for (int i = tid; i < rows * (kBlk / 8); i += kSumWarps * 32) {
      const int r = i / (kBlk / 8), f = i % (kBlk / 8) * 8;
      if (f >= feats) continue;  // M is a multiple of 8
      const float4 a = *reinterpret_cast<const float4 *>(y + r * kPitch + f);
      const float4 b = *reinterpret_cast<const float4 *>(y + r * kPitch + f + 4);
      const int64_t at = static_cast<int64_t>(row0 + r) * p.M + br * kBlk + f;
      if constexpr (OUT_BF16) {
        const __nv_bfloat162 v[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                                     __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.Y) + at) = *reinterpret_cast<const uint4 *>(v);
      } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.Y) + at) = a;
        *reinterpret_cast<float4 *>(static_cast<float *>(p.Y) + at + 4) = b;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace

cudaError_t launch_adapter_decode(const CUtensorMap &tmA, const CUtensorMap &tmX, AdapterDecodeParams p, bool bf16,
                                  bool out_bf16, cudaStream_t s) {
  // the stages get what U's ring and h leave of half an SM; y takes their place at the end
  const int slot = kBlk * p.rank * 2, stage = kBlkBytes + p.tile * 128;
  p.qu = kMaxQU;  // a power of two
  while (p.qu * slot > kUpRing) p.qu /= 2;
  const int fixed = p.qu * slot + p.tile * p.rank * 4 + kMiscBytes + 1024;
  p.q = (kSmemLimit - fixed) / stage;
  if (p.q < 2) p.q = 2;
  static_assert(2 * (kBlkBytes + 16 * 128) >= 16 * kPitch * 4 && 2 * (kBlkBytes + 64 * 128) >= 64 * kPitch * 4,
                "y fits in two stages");
  if (p.q > kMaxQ) p.q = kMaxQ;
  const int smem = fixed + p.q * stage;
  auto kern = bf16 ? (out_bf16 ? adapter_decode_kernel<true, true> : adapter_decode_kernel<true, false>)
                   : (out_bf16 ? adapter_decode_kernel<false, true> : adapter_decode_kernel<false, false>);
  static std::atomic<uint64_t> smem_set[4];
  cudaError_t e = set_smem_limit_once(kern, 160 * 1024, smem_set[(bf16 ? 2 : 0) + (out_bf16 ? 1 : 0)]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.M + kBlk - 1) / kBlk), static_cast<unsigned>((p.N + p.tile - 1) / p.tile));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tmA, tmX, p);
}

}  // namespace spmm
