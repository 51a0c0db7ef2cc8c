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
// values); every lane of the summing warps copies its own 16-byte words of them to
// shared memory (cp.async, two units of 2 KB in flight per warp), so nothing but
// the lane waits for them, and multiplies them with h, kept in fp32.  64
// single-row requests with 64 adapters through 18944 features take 16.5 us at rank
// 16 (46 MB of U), 37 at rank 64 (30 at the HBM rate).  In its place, a ring of
// bulk copies took 26 us at rank 16 whatever the bytes (an SM's copy engine starts
// one copy per ~110 cycles), loads into two sets of registers 19 and 46 us (they
// spill, and a spilled load is waited for), three units per warp 18 us (a stage of
// blocks less).  A row meets its own adapter alone.
//
// HBM bounds large batches of adapters (the blocks once, 2 nnz bytes, and each
// adapter's U once), the chain of dependent loads the small ones: block row
// pointer -> block and its column -> rows of X -> MMA -> sums -> store.  So
// everything that does not hang on something else starts at once: blocks are
// fetched before their columns are known, the first of U as soon as the segments
// are, and all of it before the down projection's kernel has ended (a
// programmatic dependent launch); only h is waited for, and the adapters' sums
// and the shared product run side by side and meet in the store.  A layer with few block rows is
// split over a cluster of up to 8 CTAs, each with a share of the blocks and of
// the adapters, whose fp32 sums are added through distributed shared memory in
// CTA order.
//
// The tensor cores cut what their fp32 sums shift out instead of rounding it, ~1e-9
// of the result for every term of a chain.  So blocks go to 8 accumulators in turn (4
// with 64 rows), which are added with rounding; one alone is no faster.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kBlk = 64;
constexpr int kBlkBytes = kBlk * kBlk * 2;
constexpr int kMaxQ = 8;
constexpr int kPiece = 8;               // rows of a segment that one warp takes
constexpr int kTmaWarp = 0, kMmaWarp = 1, kSumWarp0 = 2, kSumWarps = 8;
constexpr int kThreads = (kSumWarp0 + kSumWarps) * 32;
constexpr int kUnitDepth = 2;           // units of U (2 KB) in flight per summing warp
constexpr int kPitch = kBlk + 4;        // floats per row of y in shared memory
constexpr int kAccCols = 256;           // TMEM columns of the accumulators, half an SM's
constexpr int kMiscBytes = 2560;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM

struct Misc {
  uint64_t full[kMaxQ], empty[kMaxQ], acc_full, listed;
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

// The adapters' share of y: y[row][feature] += U_a[feature] . h[row].  SPAN
// adjacent lanes share a feature, each with 8 of its ranks (SPAN is rank / 8
// rounded up to a power of two), so a warp reads U as contiguous 16-byte words,
// 32 / SPAN features a pass.  A unit is up to four passes of one piece (up to
// kPiece rows of one segment); the warps take units in turn.  Pieces share no
// row and units of a piece no feature, so no two warps add to the same sum.
template <bool BF16, int SPAN>
struct Adders {
  static constexpr int kPasses = SPAN == 1 ? 2 : 4;              // per unit
  static constexpr int kUnits = kBlk * SPAN / 32 / kPasses;      // per piece
  static constexpr int kFeats = 32 / SPAN;                       // per pass
  const AdapterDecodeParams &p;
  const Misc *mi;
  uint32_t ring;  // the lane's words: kDepth units of kPasses words, 512 bytes apart
  int32_t br, feats, part, n_units;
  int c, f0, chunks;

  __device__ __forceinline__ Adders(const AdapterDecodeParams &p_, const Misc *mi_, int32_t br_, int32_t feats_, int32_t part_,
                                  uint32_t ring_)
      : p(p_), mi(mi_), br(br_), feats(feats_), part(part_) {
    const int lane = threadIdx.x & 31;
    ring = ring_ + ((threadIdx.x >> 5) - kSumWarp0) * (kUnitDepth * 2048) + lane * 16;
    c = lane % SPAN;
    f0 = lane / SPAN;
    chunks = p.rank / 8;
    const int32_t mine = mi->n_pieces > part ? (mi->n_pieces - part + p.split - 1) / p.split : 0;
    n_units = mine * kUnits;
  }
  __device__ __forceinline__ TileSegment piece(int32_t v) const { return mi->pieces[part + v / kUnits * p.split]; }
  __device__ __forceinline__ int feature(int32_t v, int pass) const { return (v % kUnits * kPasses + pass) * kFeats + f0; }
  __device__ __forceinline__ void load(int32_t v, int slot) const {
    if (v < n_units) {
      const uint4 *U = static_cast<const uint4 *>(p.up) +
                       (static_cast<int64_t>(piece(v).adapter) * p.M + br * kBlk) * chunks;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int f = feature(v, i);
        cp_async_16(ring + slot * 2048 + i * 512, U + f * chunks + c, c < chunks && f < feats ? 16 : 0);
      }
    }
    cp_async_commit();
  }
  // ROWS rows of the piece from row n on: U is unpacked once for them.
  template <int ROWS>
  __device__ __forceinline__ void add_rows(int32_t v, int slot, const float *__restrict__ h, float *__restrict__ y,
                                           int n) const {
    float hv[ROWS][8] = {}, d[ROWS][kPasses];
    if (c < chunks) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const float4 *src = reinterpret_cast<const float4 *>(h + (n + r) * p.rank) + c * 2;
        const float4 a = src[0], b = src[1];
        hv[r][0] = a.x, hv[r][1] = a.y, hv[r][2] = a.z, hv[r][3] = a.w;
        hv[r][4] = b.x, hv[r][5] = b.y, hv[r][6] = b.z, hv[r][7] = b.w;
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      float uf[8];
      unpack8<BF16>(ld_shared_16(ring + slot * 2048 + i * 512), uf);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        d[r][i] = uf[0] * hv[r][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) d[r][i] = fmaf(uf[e], hv[r][e], d[r][i]);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float *row = y + (n + r) * kPitch;
      if constexpr (SPAN == 1) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) row[feature(v, i)] += d[r][i];
      } else {
        // the lanes of a feature add up and share the passes out between them
        const bool up = (c & (SPAN / 2)) != 0;
        const float e0 = (up ? d[r][2] : d[r][0]) + __shfl_xor_sync(0xffffffffu, up ? d[r][0] : d[r][2], SPAN / 2);
        const float e1 = (up ? d[r][3] : d[r][1]) + __shfl_xor_sync(0xffffffffu, up ? d[r][1] : d[r][3], SPAN / 2);
        if constexpr (SPAN == 2) {
          row[feature(v, up ? 2 : 0)] += e0;
          row[feature(v, up ? 3 : 1)] += e1;
        } else {
          const bool odd = (c & (SPAN / 4)) != 0;
          float e = (odd ? e1 : e0) + __shfl_xor_sync(0xffffffffu, odd ? e0 : e1, SPAN / 4);
#pragma unroll
          for (int o = SPAN / 8; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
          if (c % (SPAN / 4) == 0) row[feature(v, c / (SPAN / 4))] += e;
        }
      }
    }
  }
  __device__ __forceinline__ void add(int32_t v, int slot, const float *__restrict__ h, float *__restrict__ y) const {
    const TileSegment s = piece(v);
    int n = s.begin;
    for (; n + 1 < s.end; n += 2) add_rows<2>(v, slot, h, y, n);
    if (n < s.end) add_rows<1>(v, slot, h, y, n);
  }
};

// The summing warps' part, from the list of pieces to y complete in shared memory.
// ready() returns once y is cleared and h is there.
template <bool BF16, int SPAN, class Ready>
__device__ __forceinline__ void sum_adapters(const AdapterDecodeParams &p, const Misc *mi, int32_t br, int32_t feats,
                                             int32_t part, uint32_t ring, const float *h, float *y, Ready &&ready) {
  const Adders<BF16, SPAN> a(p, mi, br, feats, part, ring);
  int32_t v = (threadIdx.x >> 5) - kSumWarp0;
  for (int i = 0; i < kUnitDepth; ++i) a.load(v + i * kSumWarps, i);
  ready();
  for (int slot = 0; v < a.n_units; v += kSumWarps) {
    cp_async_wait_group<kUnitDepth - 1>();
    a.add(v, slot, h, y);
    a.load(v + kUnitDepth * kSumWarps, slot);
    if (++slot == kUnitDepth) slot = 0;
  }
  cp_async_wait_group<0>();
}

template <bool BF16, bool OUT_BF16>
__global__ void __launch_bounds__(kThreads, 2)
    adapter_decode_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmX,
                          const AdapterDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kBlkBytes + p.tile * 128;
  uint8_t *ring = smem + p.q * stage_bytes;                        // U
  float *h = reinterpret_cast<float *>(ring + kSumWarps * kUnitDepth * 2048);  // [tile][rank]
  float *y = h + p.tile * p.rank;                                  // [tile][kPitch]
  Misc *mi = reinterpret_cast<Misc *>(y + p.tile * kPitch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t br = blockIdx.x / p.split, part = blockIdx.x % p.split;  // part = rank in the cluster
  const int32_t row0 = blockIdx.y * p.tile;
  const int32_t rows = min(p.N - row0, p.tile);
  const int32_t feats = min(p.M - br * kBlk, kBlk);
  const uint32_t acc_cols = p.tile < 32 ? 32 : p.tile;
  const uint32_t n_acc = kAccCols / acc_cols;
  const int64_t row_begin = p.block_row_ptr[br];
  const int64_t blocks = p.block_row_ptr[br + 1] - row_begin;

  if (warp == kMmaWarp) {
    if (lane < p.q) {
      mbar_init(smem_addr(&mi->full[lane]), 1);
      mbar_init(smem_addr(&mi->empty[lane]), 1);
    }
    if (lane == 0) {
      mbar_init(smem_addr(&mi->acc_full), 1);
      mbar_init(smem_addr(&mi->listed), 1);
      mi->abort_flag = 0;
    }
    fence_barrier_init();
    __syncwarp();
    tmem_alloc(smem_addr(&mi->tmem), kAccCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = mi->tmem;
  const int64_t jb = row_begin + blocks * part / p.split;  // the block row's bounds are waited for only here
  const int64_t je = row_begin + blocks * (part + 1) / p.split;

  if (warp == kTmaWarp) {
    // The first stages, a lane each: their blocks at once, their rows of X as soon
    // as their columns are known.
    const int32_t ahead = static_cast<int32_t>(min(je - jb, static_cast<int64_t>(p.q)));
    if (lane < ahead) {
      const int32_t first_col = p.block_col_idx[jb + lane];
      const uint32_t fb = smem_addr(&mi->full[lane]), st = smem_addr(smem + lane * stage_bytes);
      mbar_arrive_expect_tx(fb, stage_bytes);
      tma_load_2d(st, &tmA, fb, 0, static_cast<int32_t>((jb + lane) * kBlk));
      tma_load_2d(st + kBlkBytes, &tmX, fb, first_col * kBlk, row0);
    }
    __syncwarp();
    uint32_t stage = 0, phase = 1;
    int64_t seq = ahead;
    bool ok = true;
    for (int64_t jbase = jb + ahead; jbase < je && ok; jbase += 32) {
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
    // first the list of pieces, while the first stage is on its way
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

    const uint32_t idesc = idesc_f16(BF16, false, false, kBlk, static_cast<uint32_t>(p.tile));
    uint32_t stage = 0, phase = 0, acc = 0, accumulate = 0;
    bool ok = true;
    for (int64_t j = jb; j < je;) {
      // how many stages in a row are there, a lane each; one wait for all of them
      const int32_t left = static_cast<int32_t>(min(je - j, static_cast<int64_t>(p.q)));
      const bool wrap = stage + lane >= static_cast<uint32_t>(p.q);
      const bool there = lane < left && mbar_test_wait(smem_addr(&mi->full[stage + lane - (wrap ? p.q : 0)]),
                                                       phase ^ (wrap ? 1u : 0u));
      int32_t ready = __ffs(~__ballot_sync(0xffffffffu, there)) - 1;
      if (ready == 0) {
        const bool r = mbar_wait_warp(smem_addr(&mi->full[stage]), phase, p.wait_limit_ns);
        ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
        if (!ok) break;
        ready = 1;
      }
      tc_fence_after_sync();
      for (; ready > 0; --ready, ++j) {
        const uint32_t st = smem_addr(smem + stage * stage_bytes);
        const uint64_t a = smem_desc_sw128(st, 16, 1024), b = smem_desc_sw128(st + kBlkBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_elect(tmem + acc * acc_cols, smem_desc_add(a, kk * 32), smem_desc_add(b, kk * 32), idesc,
                         kk > 0 ? 1u : accumulate);
        if (++acc == n_acc) {
          acc = 0;
          accumulate = 1;
        }
        if (j + p.q < je) umma_commit_elect(smem_addr(&mi->empty[stage]));  // the stage is filled once more
        if (++stage == static_cast<uint32_t>(p.q)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
    }
    __syncwarp();
    umma_commit_elect(smem_addr(&mi->acc_full));
  } else {
    const int tid = threadIdx.x - kSumWarp0 * 32;
    auto give_up = [&] {
      if (lane == 0) {
        atomicOr(p.status, kDevTimeout);
        mi->abort_flag = 1;
      }
    };
    auto ready = [&] {
      for (int i = tid; i < p.tile * kPitch / 4; i += kSumWarps * 32) reinterpret_cast<float4 *>(y)[i] = float4{};
      grid_dependency_wait();  // h; every block waits, so this kernel never ends before that one
      const float4 *src = reinterpret_cast<const float4 *>(p.H + static_cast<int64_t>(row0) * p.rank);
      for (int i = tid; i < rows * p.rank / 4; i += kSumWarps * 32) reinterpret_cast<float4 *>(h)[i] = src[i];
      sum_warps_sync();
    };
    if (!mbar_wait_warp(smem_addr(&mi->listed), 0, p.wait_limit_ns)) {
      give_up();
      ready();
    } else if (p.rank == 8) {
      sum_adapters<BF16, 1>(p, mi, br, feats, part, smem_addr(ring), h, y, ready);
    } else if (p.rank == 16) {
      sum_adapters<BF16, 2>(p, mi, br, feats, part, smem_addr(ring), h, y, ready);
    } else if (p.rank <= 32) {
      sum_adapters<BF16, 4>(p, mi, br, feats, part, smem_addr(ring), h, y, ready);
    } else if (p.rank <= 64) {
      sum_adapters<BF16, 8>(p, mi, br, feats, part, smem_addr(ring), h, y, ready);
    } else {
      sum_adapters<BF16, 16>(p, mi, br, feats, part, smem_addr(ring), h, y, ready);
    }
    sum_warps_sync();
    if (je > jb) {
      // Rows 16 s .. 16 s + 15 of the accumulator lie in lanes 32 s .. 32 s + 15.
      // Two warps share them, each every other 16 columns (rows of X).
      const int sp = warp & 3;
      const bool ok = mbar_wait_warp(smem_addr(&mi->acc_full), 0, p.wait_limit_ns);
      if (!ok) give_up();
      tc_fence_after_sync();
      const uint32_t used = static_cast<uint32_t>(min(je - jb, static_cast<int64_t>(n_acc)));
      for (int c0 = (warp - kSumWarp0) / 4 * 16; c0 < p.tile && ok; c0 += 32) {
        float sum[16] = {};
        for (uint32_t i = 0; i < used; ++i) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(sp * 32) << 16) + i * acc_cols + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[e] += __uint_as_float(v[e]);
        }
        if (lane < 16)
#pragma unroll
          for (int e = 0; e < 16; ++e) y[(c0 + e) * kPitch + sp * 16 + lane] += sum[e];
      }
    }
  }
  tc_fence_before_sync();
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  {
    const int32_t r0 = rows * part / p.split, r1 = rows * (part + 1) / p.split;
    for (int i = threadIdx.x; i < (r1 - r0) * (kBlk / 8); i += kThreads) {
      const int r = r0 + i / (kBlk / 8), f = i % (kBlk / 8) * 8;
      if (f >= feats) continue;  // M is a multiple of 8
      float4 a, b;
      if (p.split > 1) {
        float o[8];
        cluster_sum8(smem_addr(y + r * kPitch + f), p.split, o);
        a = make_float4(o[0], o[1], o[2], o[3]);
        b = make_float4(o[4], o[5], o[6], o[7]);
      } else {
        a = *reinterpret_cast<const float4 *>(y + r * kPitch + f);
        b = *reinterpret_cast<const float4 *>(y + r * kPitch + f + 4);
      }
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
  if (p.split > 1) cluster_sync();  // the others may still read this CTA's sums
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kAccCols);
  }
}

}  // namespace

cudaError_t launch_adapter_decode(const CUtensorMap &tmA, const CUtensorMap &tmX, AdapterDecodeParams p, int num_sms,
                                  bool bf16, bool out_bf16, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(p.M) + kBlk - 1) / kBlk * ((p.N + p.tile - 1) / p.tile);
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= 2ll * num_sms) p.split *= 2;
  // the stages get what h and y leave of half an SM
  const int stage = kBlkBytes + p.tile * 128;
  const int fixed = kSumWarps * kUnitDepth * 2048 + p.tile * (p.rank + kPitch) * 4 + kMiscBytes + 1024;
  p.q = (kSmemLimit - fixed) / stage;
  if (p.q > kMaxQ) p.q = kMaxQ;
  static_assert((kSmemLimit - kSumWarps * kUnitDepth * 2048 - 64 * (64 + kPitch) * 4 - kMiscBytes - 1024) / (kBlkBytes + 64 * 128) >= 2 &&
                    (kSmemLimit - kSumWarps * kUnitDepth * 2048 - 32 * (kMaxRank + kPitch) * 4 - kMiscBytes - 1024) / (kBlkBytes + 32 * 128) >= 2,
                "at least two stages: 64 rows up to rank 64, 32 above");
  const int smem = fixed + p.q * stage;
  auto kern = bf16 ? (out_bf16 ? adapter_decode_kernel<true, true> : adapter_decode_kernel<true, false>)
                   : (out_bf16 ? adapter_decode_kernel<false, true> : adapter_decode_kernel<false, false>);
  static std::atomic<uint64_t> smem_set[4];
  cudaError_t e = set_smem_limit_once(kern, kSmemLimit, smem_set[(bf16 ? 2 : 0) + (out_bf16 ? 1 : 0)]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.M + kBlk - 1) / kBlk * p.split), static_cast<unsigned>((p.N + p.tile - 1) / p.tile));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tmA, tmX, p);
}

}  // namespace spmm
