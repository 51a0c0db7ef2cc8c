// adapter_wgrad_kernel.cu -- gradients of the adapters' weights
// (spmm_adapters_grad):
//   d_up_a[f][i]   = sum over rows n of adapter a of dY[n][f] * H[n][i]
//   d_down_a[i][f] = sum over rows n of adapter a of  X[n][f] * dH[n][i]
// Both are V^T S with V an N x F matrix of activations and S N x rank, so one
// kernel does both: the rows are the MMA's K, 128 features of V the M operand
// and the ranks the N operand, both MN-major as they lie in memory.
//
// Work item = (128 features, adapter).  A stage is 64, 48 or 32 rows of one segment (a TMA
// box may start at any row), so K never runs across a segment; the rows after a
// segment's end that the last box brings are zeroed in shared memory in both
// operands before the MMA, as neither operand may hold another request's
// infinities.  With fp16 a stage does not run either from one power of two that S is
// divided by to another (see kHParts), and the sums are taken out and multiplied where the
// power changes (every piece by itself: 402 us for 301 with 16384 rows of 4 adapters of rank
// 64, 18944 x 3584, the down projections among them; bf16 279).  Every element of dY and X is read once, so HBM bounds the kernel;
// S is read again by every feature tile, from L2.  16384 rows of 4 adapters of rank
// 64, 18944 + 3584 features: 152 us, 4.9 TB/s of activations.
//
// S comes in kHParts 16-bit parts, 24 bits of bf16 together, whose sums are added at
// the end: with h and dh rounded to two, sums that cancel kept 16 bits of theirs.
// One MMA takes as many parts as N = 256 holds, side by side (three up to rank 80, two
// above), so that the features' operand passes shared memory less often: its bandwidth is
// the bound at the larger ranks (the gradient of 16384 rows, 4 adapters of rank 64,
// 18944 x 3584: 621 us, with an MMA for each part 729).
//
// The tensor cores cut what their fp32 sums shift out instead of rounding it: sums of
// 131072 positive rows came out 7.8e-4 low, more than rounding to fp16 does.  So the sums
// leave them every kTurnRows rows and are added in registers (16384 rows, rank 64: 278 us
// with the down projections; every 512 rows 283, every 2048 275, never 272).
//
// With items enough for every SM, CTAs (two per SM) are persistent and take items
// in turn, two TMEM accumulators alternating (one above 42 ranks, whose three parts fill an
// SM's half), so one item's sums are stored while
// the next one's rows arrive.  A CTA per item instead, each with a start and an end
// of its own, with one part of S: 37 us for 24 with 100 segments of 20 rows (20 adapters of
// rank 32, 4096 + 4096 features), 52 for 39 with 4096 rows of 4 adapters of rank 64
// (18944 + 3584 features), 109 for 75 with 500 segments of 16 rows.  With fewer
// items a cluster of up to 8 CTAs shares one: an adapter's stages are dealt to it
// in turn and it adds its fp32 sums through distributed shared memory in CTA order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kFeat = 128;            // features per CTA
constexpr int kMaxQ = 6;
constexpr int kThreads = 192;
constexpr int kTmaWarp = 0, kMmaWarp = 1;
constexpr int kMiscBytes = 1024;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM

// Parts of S that the first MMA takes; a second one takes the rest, if there is one.
__host__ __device__ constexpr int joint_parts(int rank) { return kHParts * rank16(rank) <= 256 ? kHParts : kHParts - 1; }
static_assert((kHParts - 1) * kMaxRank <= 256, "two MMAs at most");
__host__ __device__ constexpr int col_boxes(int cols) { return (cols + 63) / 64; }
// Boxes of S in a stage, the second MMA's after the first one's.
__host__ __device__ constexpr int joint_boxes(int rank) { return col_boxes(joint_parts(rank) * rank16(rank)); }
__host__ __device__ constexpr int s_boxes(int rank) {
  return joint_boxes(rank) + (joint_parts(rank) < kHParts ? col_boxes(rank16(rank)) : 0);
}
// Rows of a stage: as many as leave three stages or more in half an SM's shared memory.
__host__ __device__ constexpr int stage_rows(int rank) { return s_boxes(rank) <= 2 ? 64 : s_boxes(rank) <= 4 ? 48 : 32; }
__host__ __device__ constexpr int part_pitch(int rank) { return rank16(rank) + 4; }

constexpr int kNbuf = 2;              // accumulators, where two CTAs have the columns for that

constexpr int kTurnRows = 1024;       // rows between two drains of an accumulator
constexpr int32_t kTurnSums = 1, kTurnLast = 2;  // it has sums; it is the item's last

struct Misc {
  uint64_t full[kMaxQ], empty[kMaxQ], acc_full[kNbuf], acc_empty[kNbuf], drained;
  int32_t rows[kMaxQ];  // rows of the stage, 0: the item has no more stages
  float by[kMaxQ], turn_by[kNbuf];  // fp16: what the rows of S in a stage, and in an accumulator, were divided by
  uint32_t tmem;
  int32_t turn[kNbuf];  // what the accumulator holds: kTurnSums | kTurnLast
  volatile int32_t abort_flag;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float v) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// Item i: features of d_up's tiles, then of d_down's, for one adapter after another.
struct Item {
  bool up;
  int32_t a, f0, F;
  __device__ __forceinline__ Item(const AdapterWgradParams &p, int64_t i) {
    a = static_cast<int32_t>(i / p.tiles);
    const int32_t tile = static_cast<int32_t>(i - static_cast<int64_t>(a) * p.tiles);
    up = tile < p.up_tiles;
    f0 = (up ? tile : tile - p.up_tiles) * kFeat;
    F = up ? p.M : p.K;
  }
};

// Eight ranks j.. of feature f0 + r of the item's gradient.
template <bool BF16>
__device__ __forceinline__ void store_grad(const AdapterWgradParams &p, const Item &item, int r, int j, const float (&o)[8]) {
  if (item.up) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = round16<BF16>(o[2 * i]) | static_cast<uint32_t>(round16<BF16>(o[2 * i + 1])) << 16;
    *reinterpret_cast<uint4 *>(p.d_up + (static_cast<int64_t>(item.a) * item.F + item.f0 + r) * p.rank + j) =
        make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p.d_down[(static_cast<int64_t>(item.a) * p.rank + j + i) * item.F + item.f0 + r] = round16<BF16>(o[i]);
  }
}

// SPLIT: a cluster of p.split CTAs per item; else persistent CTAs.  Ranks up to RANKS.
template <bool BF16, bool SPLIT, int RANKS>
__global__ void __launch_bounds__(kThreads, 2) adapter_wgrad_kernel(const __grid_constant__ AdapterWgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int joint = joint_parts(p.rank), jb = joint_boxes(p.rank), boxes = s_boxes(p.rank);
  const int stage_k = stage_rows(p.rank);
  const int box_bytes = stage_k * 128, v_bytes = kFeat / 64 * box_bytes;  // a box: a stage's rows x 64 columns
  const int stage_bytes = v_bytes + boxes * box_bytes;
  Misc *mi = reinterpret_cast<Misc *>(smem + p.q * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t part = SPLIT ? blockIdx.x % p.split : 0, split = SPLIT ? p.split : 1;
  const int64_t first = blockIdx.x / split, step = gridDim.x / split;  // this CTA's items
  const int64_t items = SPLIT ? first + 1 : static_cast<int64_t>(p.tiles) * p.n_adapters;
  const int n16 = rank16(p.rank);                  // ranks of an accumulator
  const int mma_n = joint * n16;
  uint32_t acc_cols = 32;
  while (static_cast<int>(acc_cols) < mma_n) acc_cols <<= 1;
  const uint32_t nbuf = acc_cols > 128 ? 1 : kNbuf;

  if (threadIdx.x == 0) {
    for (int q = 0; q < p.q; ++q) {
      mbar_init(smem_addr(&mi->full[q]), 1);
      mbar_init(smem_addr(&mi->empty[q]), 1);
    }
    for (int b = 0; b < kNbuf; ++b) {
      mbar_init(smem_addr(&mi->acc_full[b]), 2);
      mbar_init(smem_addr(&mi->acc_empty[b]), 4);
    }
    mbar_init(smem_addr(&mi->drained), 1);
    mi->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&mi->tmem), nbuf * acc_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = mi->tmem;
  auto wait_phase = [&](uint64_t &bar, uint32_t parity) -> bool {
    const bool r = mbar_wait_warp(smem_addr(&bar), parity, p.wait_limit_ns);
    return __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
  };
  auto give_up = [&] {
    if (lane == 0) {
      atomicOr(p.status, kDevTimeout);
      mi->abort_flag = 1;
    }
    __syncwarp();
  };

  if (warp == kTmaWarp) {
    uint32_t stage = 0, phase = 0;
    int64_t seq = 0;
    bool ok = true;
    auto claim = [&]() -> bool { return wait_phase(mi->empty[stage], phase ^ 1u); };
    auto advance = [&]() {
      ++seq;
      if (++stage == static_cast<uint32_t>(p.q)) {
        stage = 0;
        phase ^= 1u;
      }
    };
    const FewSegments few(p.seg_ptr, p.seg_adapter, p.n_seg);  // all of them, in short batches
    for (int64_t it = first; it < items && ok; it += step) {
      const Item item(p, it);
      const CUtensorMap *tmV = item.up ? &p.tm_dy : &p.tm_x;
      const CUtensorMap *tmS = item.up ? &p.tm_h : &p.tm_dh;
      int32_t turn = 0;  // whose turn the next stage of the adapter is
      // the adapter's segments among 32, one a lane
      auto walk = [&](int64_t begin, int64_t end, int32_t adapter) {
        begin = max(begin, int64_t{0});
        end = min(end, static_cast<int64_t>(p.N));
        const bool mine = begin < end && adapter == item.a;
        uint32_t todo = __ballot_sync(0xffffffffu, mine);
        // fp16: the power of two of the piece that a row lies in
        const float *powers = item.up ? p.h_scale : p.dh_scale;
        const float first_power = !BF16 && mine ? powers[begin] : 1.0f;
        while (todo && ok) {
          const int i = __ffs(todo) - 1;
          todo &= todo - 1;
          const int32_t sb = __shfl_sync(0xffffffffu, static_cast<int32_t>(begin), i);
          const int32_t se = __shfl_sync(0xffffffffu, static_cast<int32_t>(end), i);
          // where the piece of row n ends, and the next one's power, read ahead
          int32_t piece_end = (sb / kPieceRows + 1) * kPieceRows, next = sb;
          float power = __shfl_sync(0xffffffffu, first_power, i), next_power = !BF16 && piece_end < se ? powers[piece_end] : 1.0f;
          for (int32_t n = sb; n < se; n = next) {
            next = se - n > stage_k ? n + stage_k : se;
            const float by = power;
            if (!BF16 && next >= piece_end) {
              if (next_power != power) next = piece_end;
              power = next_power;
              piece_end += kPieceRows;
              if (piece_end < se) next_power = powers[piece_end];
            }
            const bool take = turn == part;
            if (++turn == split) turn = 0;
            if (!take) continue;
            ok = claim();
            if (!ok) break;
            if (lane == 0) {
              mi->rows[stage] = next - n;
              if (!BF16) mi->by[stage] = by;
              const uint32_t fb = smem_addr(&mi->full[stage]);
              const uint32_t st = smem_addr(smem + stage * stage_bytes);
              mbar_arrive_expect_tx(fb, stage_bytes);
              tma_load_2d(st, tmV, fb, item.f0, n);
              tma_load_2d(st + box_bytes, tmV, fb, item.f0 + 64, n);
              for (int c = 0; c < boxes; ++c) {
                const int32_t col = c < jb ? c * 64 : joint * n16 + (c - jb) * 64;
                tma_load_2d(st + v_bytes + c * box_bytes, tmS, fb, col, n);
              }
            }
            __syncwarp();
            advance();
          }
        }
      };
#pragma unroll
      for (int g = 0; g < kFewGroups; ++g) walk(few.begin[g], few.end[g], few.adapter[g]);
      for (int32_t base = kFewSegments; base < p.n_seg && ok; base += kFewSegments) {
        const FewSegments more(p.seg_ptr, p.seg_adapter, p.n_seg, base);
#pragma unroll
        for (int g = 0; g < kFewGroups; ++g) walk(more.begin[g], more.end[g], more.adapter[g]);
      }
      if (ok) ok = claim();
      if (ok) {
        if (lane == 0) {
          mi->rows[stage] = 0;
          mbar_arrive(smem_addr(&mi->full[stage]));
        }
        __syncwarp();
        advance();
      }
    }
    if (!ok) {
      give_up();
      if (lane == 0)  // let the copies in flight land before the block ends
        for (int64_t i = seq > p.q ? seq - p.q : 0; i < seq; ++i)
          mbar_wait(smem_addr(&mi->full[i % p.q]), static_cast<uint32_t>((i / p.q) & 1), 1000000ull);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = idesc_f16(BF16, /*a_mn_major=*/true, /*b_mn_major=*/true, kFeat, static_cast<uint32_t>(mma_n));
    const uint32_t idesc_rest = idesc_f16(BF16, true, true, kFeat, static_cast<uint32_t>(n16));
    const int turn_stages = kTurnRows / stage_k;
    uint32_t stage = 0, phase = 0, count = 0;
    bool ok = true;
    for (int64_t it = first; it < items && ok; it += step) {
      for (bool last = false; !last && ok; ++count) {  // a turn
        const uint32_t buf = count % nbuf, acc = tmem + buf * acc_cols;
        ok = wait_phase(mi->acc_empty[buf], ((count / nbuf) & 1u) ^ 1u);
        if (!ok) break;
        tc_fence_after_sync();
        int stages = 0;
        float by = 1.0f;
        while (stages < turn_stages) {
          ok = wait_phase(mi->full[stage], phase);
          if (!ok) break;
          const int32_t rows = mi->rows[stage];
          last = rows == 0;
          if (!BF16 && !last) {  // one power of two a turn
            const float next_by = mi->by[stage];
            if (stages > 0 && next_by != by) break;
            by = next_by;
          }
          if (!last) {
            const int steps = (rows + 15) / 16;
            if (rows % 16 != 0) {
              // rows [rows, 16 * steps) belong to another segment: a swizzled row is
              // 128 contiguous bytes of its box, so whole rows can be cleared
              const int n = (16 * steps - rows) * 8;
              uint8_t *st = smem + stage * stage_bytes + rows * 128;
              for (int box = 0; box < kFeat / 64 + boxes; ++box)
                for (int u = lane; u < n; u += 32) *reinterpret_cast<uint4 *>(st + box * box_bytes + u * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc_fence_after_sync();
            const uint32_t st = smem_addr(smem + stage * stage_bytes);
            const uint64_t v = smem_desc_sw128(st, box_bytes, 1024);
            const uint64_t s = smem_desc_sw128(st + v_bytes, box_bytes, 1024);
            for (int kk = 0; kk < steps; ++kk) {
              umma_f16_elect(acc, smem_desc_add(v, kk * 2048), smem_desc_add(s, kk * 2048), idesc, (stages > 0 || kk > 0) ? 1u : 0u);
              if (joint < kHParts)
                umma_f16_elect(acc, smem_desc_add(v, kk * 2048), smem_desc_add(s, jb * box_bytes + kk * 2048), idesc_rest, 1u);
            }
            ++stages;
          }
          umma_commit_elect(smem_addr(&mi->empty[stage]));
          if (++stage == static_cast<uint32_t>(p.q)) {
            stage = 0;
            phase ^= 1u;
          }
          if (last) break;
        }
        if (!ok) break;
        if (lane == 0) {
          if (!BF16) mi->turn_by[buf] = by;
          mi->turn[buf] = (stages > 0 ? kTurnSums : 0) | (last ? kTurnLast : 0);
          mbar_arrive(smem_addr(&mi->acc_full[buf]));
        }
        __syncwarp();
        umma_commit_elect(smem_addr(&mi->acc_full[buf]));
      }
    }
    if (!ok) {
      give_up();
      // wait for what was issued: nothing may be in flight when the block ends
      umma_commit_elect(smem_addr(&mi->drained));
      mbar_wait_warp(smem_addr(&mi->drained), 0, 1000000ull);
    }
  } else {
    const int sp = warp & 3;
    const int r = sp * 32 + lane;  // feature f0 + r
    uint32_t count = 0;
    bool ok = true;
    for (int64_t it = first; it < items && ok; it += step) {
      const Item item(p, it);
      float sum[RANKS] = {};
      for (int32_t turn = 0; (turn & kTurnLast) == 0; ++count) {
        const uint32_t buf = count % nbuf;
        ok = wait_phase(mi->acc_full[buf], (count / nbuf) & 1u);
        if (!ok) {
          give_up();
          break;
        }
        tc_fence_after_sync();
        turn = mi->turn[buf];
        if (turn & kTurnSums) {
          const uint32_t at = tmem + buf * acc_cols + (static_cast<uint32_t>(sp * 32) << 16);
          const float by = BF16 ? 1.0f : mi->turn_by[buf];
#pragma unroll
          for (int c0 = 0; c0 < RANKS; c0 += 16) {
            if (c0 >= n16) break;
            constexpr int kAtOnce = RANKS > 64 ? 1 : kHParts;  // what the registers hold beside the sums
            uint32_t v[kAtOnce][16];
#pragma unroll
            for (int q = kHParts - 1; q >= 0; --q) {  // the smallest first
              if (q >= joint) continue;
              if (kAtOnce == 1 || q == joint - 1) {
#pragma unroll
                for (int o = 0; o < kAtOnce; ++o)
                  if (o < joint) tmem_ld_32x32b_x16(at + (kAtOnce == 1 ? q : o) * n16 + c0, v[o]);
                tmem_ld_wait();
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float s = __uint_as_float(v[kAtOnce == 1 ? 0 : q][i]);
                sum[c0 + i] = BF16 ? sum[c0 + i] + s : fmaf(by, s, sum[c0 + i]);
              }
            }
          }
          tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&mi->acc_empty[buf]));
      }
      if (!ok) break;
#pragma unroll
      for (int c0 = 0; c0 < RANKS; c0 += 8) {
        if (c0 >= p.rank) break;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = sum[c0 + i];
        if constexpr (SPLIT) {
          float4 *dst = reinterpret_cast<float4 *>(reinterpret_cast<float *>(smem) + r * part_pitch(p.rank) + c0);  // the stages are done with
          dst[0] = make_float4(o[0], o[1], o[2], o[3]);
          dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else if (item.f0 + r < item.F) {
          store_grad<BF16>(p, item, r, c0, o);
        }
      }
    }
  }
  if constexpr (SPLIT) {
    cluster_sync();  // every CTA of the cluster comes here, whatever happened before
    const Item item(p, first);
    const int feats = kFeat / split, r0 = part * feats, units = p.rank / 8;
    const uint32_t base = smem_addr(smem);
    for (int u = threadIdx.x; u < feats * units; u += kThreads) {
      // d_up: a feature's ranks are contiguous; d_down: a rank's features are
      const int r = r0 + (item.up ? u / units : u % feats), j = (item.up ? u % units : u / feats) * 8;
      if (item.f0 + r >= item.F) continue;
      float o[8];
      cluster_sum8(base + (r * part_pitch(p.rank) + j) * 4, split, o);
      store_grad<BF16>(p, item, r, j, o);
    }
    cluster_sync();  // the others may still read this CTA's sums
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, nbuf * acc_cols);
  }
}

}  // namespace

int wgrad_stage_rows(int rank) { return stage_rows(rank); }

cudaError_t launch_adapter_wgrad(AdapterWgradParams p, int num_sms, bool bf16, cudaStream_t s) {
  p.up_tiles = (p.M + kFeat - 1) / kFeat;
  p.tiles = p.up_tiles + (p.K + kFeat - 1) / kFeat;
  // Items of adapters that can have rows.  While clusters of twice the size still fit
  // beside each other and leave each CTA at least four stages, they are the faster
  // (us with 1 / 2 / 4 / 8 CTAs an item, 16384 rows, the down projections among them; 16
  // items, rank 64: 182 / 112 / 77 / 63; 64 items, rank 16: 179 / 117 / 90 / 110; 128 items, rank
  // 64: 271 / 201 / 222 / 281); with more items they only wait for one another (176: 316 /
  // 331 / 315 / 356; 256: 200 / 212 / 244 / 324, and 67 / 78 / 103 / 158 for 4096 rows).  Clusters
  // are not persistent, so the items of adapters without rows limit them too (one adapter
  // of 28 with 740 rows, 176 tiles: 42 / 153).
  const int64_t active = p.n_seg < p.n_adapters ? (p.n_seg > 0 ? p.n_seg : 1) : p.n_adapters;
  p.split = 1;
  while (p.split < 8 && p.tiles * active * p.split * 2 <= 2ll * num_sms && p.N >= 512ll * active * p.split &&
         p.tiles * static_cast<int64_t>(p.n_adapters) * p.split * 2 <= 8ll * num_sms)
    p.split *= 2;
  const bool split = p.split > 1;
  const int stage = (kFeat / 64 + s_boxes(p.rank)) * stage_rows(p.rank) * 128;
  p.q = (kSmemLimit - kMiscBytes - 1024) / stage;
  if (p.q > kMaxQ) p.q = kMaxQ;
  const int smem = p.q * stage + kMiscBytes + 1024;
  const bool wide = p.rank > 64;
  auto kern = wide ? (bf16 ? (split ? adapter_wgrad_kernel<true, true, 128> : adapter_wgrad_kernel<true, false, 128>)
                           : (split ? adapter_wgrad_kernel<false, true, 128> : adapter_wgrad_kernel<false, false, 128>))
                   : (bf16 ? (split ? adapter_wgrad_kernel<true, true, 64> : adapter_wgrad_kernel<true, false, 64>)
                           : (split ? adapter_wgrad_kernel<false, true, 64> : adapter_wgrad_kernel<false, false, 64>));
  static std::atomic<uint64_t> smem_set[8];
  cudaError_t e = set_smem_limit_once(kern, kSmemLimit, smem_set[(wide ? 4 : 0) + (bf16 ? 2 : 0) + (split ? 1 : 0)]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t items = static_cast<int64_t>(p.tiles) * p.n_adapters;
  cfg.gridDim = dim3(static_cast<unsigned>(split ? items * p.split : items < 2 * num_sms ? items : 2 * num_sms));
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
