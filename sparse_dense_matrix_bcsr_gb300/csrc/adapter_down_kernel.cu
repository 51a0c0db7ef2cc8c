// adapter_down_kernel.cu -- the adapters' down projection for long batches,
//   H[n] = scale[a] * D_a X[n]    (spmm_run_linear_adapters, spmm_adapters_grad)
// on the tensor cores, with H in the 16-bit type that the projection's MMAs
// take it in.
//
// Work unit = the part of a 128-row tile that lies in one segment: the tile's
// rows of X are the M operand and the adapter's ranks the N operand (D_a's rows),
// both K-major as they lie in memory (the gradient's dY U_a takes U_a as it lies
// too, MN-major); one stage is 64 columns of both.  Rows of the tile outside the
// segment run along and are not stored, so every row meets its own adapter alone; a
// tile that several segments share is read once per segment, from L2.  (Loading a
// segment's rows alone, in boxes of 32, 16 or 8 rows, is slower: 22, 28 and 35 us for
// 20 with 777 rows in 40 segments, 61, 72 and 89 for 46 with 8192 rows in 500 segments
// of 4096 columns.)  2 N r k FLOP against 2 N k bytes are far below the tensor
// rate, so HBM bounds it for prompts.  Few units leave SMs idle: a cluster of up to
// 16 CTAs then splits a unit's columns and adds the fp32 sums through distributed
// shared memory in CTA order (no atomics, no second launch).
// One CTA per tile that walked the tile's segments one after another took 56
// against 20 us for 777 rows in 40 segments (8192 columns, rank 64).
//
// The gradient wants two such products of a batch, of X and of dY: one launch
// runs both, so that short batches fill the GPU with their sum.
//
// H is kept in 16-bit parts (the value in 16 bits, the rest in 16 bits, ...), kHParts of
// them, all 24 bits of a float (two of bf16, 16 bits, left 1.2e-6 of an fp32 Y off where
// the adapters are most of it, three 0.6e-6).  The sums leave the tensor cores, which cut
// what an fp32 sum shifts out instead of rounding it (~1e-9 of the sum for every term),
// every kTurn stages and are added in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.cuh"

namespace spmm {
namespace {

constexpr int kRows = kPieceRows;
static_assert(kRows == 128, "the MMA's M");
constexpr int kXBytes = kRows * 128;  // 128 rows x 64 columns
constexpr int kMaxQ = 8;
constexpr int kMaxSplit = 16;           // CTAs of a cluster (above 8 a kernel has to ask for it)
constexpr int kThreads = 192;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kEpiWarp0 = 2;
constexpr int kNbuf = 2;                // accumulators
constexpr int kTurn = 8;                // stages between two drains of the accumulator
constexpr int kMiscBytes = 1024;
constexpr int kSmemLimit = 112 * 1024;  // two CTAs per SM

// D's part of a stage: rank rows of 64 columns, or (transposed, never less) 64
// rows of 64 ranks per box.
__host__ __device__ constexpr int d_boxes(int rank) { return (rank + 63) / 64; }
__host__ __device__ constexpr int d_bytes(int rank, bool transposed) {
  return transposed ? d_boxes(rank) * 8192 : (rank16(rank) * 128 + 1023) / 1024 * 1024;
}
__host__ __device__ constexpr int part_pitch(int rank) { return rank16(rank) + 4; }  // floats per row of the CTA's sums

struct Misc {
  uint64_t full[kMaxQ], empty[kMaxQ], acc_full[kNbuf], acc_empty[kNbuf], drained;
  RowPiece piece;
  uint32_t row_max[kRows], piece_max;  // bits of the largest finite |h| of each row, of the CTA's rows
  uint32_t tmem;
  volatile int32_t abort_flag;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc area");

// Two values as 16-bit parts.  bf16: cut, not rounded: three times 8 bits are a float's 24, and
// no finite value becomes infinite.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// Powers of two that the fp16 values of a group are multiplied and divided by, from the
// bits of its largest finite |h|: a value of 2^e .. 2^(e + 1) comes to 2^14 .. 2^15, a
// piece's, whose e is rounded up to 2, 6, 10, ..., to 2^11 .. 2^15 (so that pieces whose
// largest values lie about 4, those of h's scale, share a power).
struct Power {
  float down, up;
  __device__ __forceinline__ explicit Power(uint32_t max_bits, bool piece = false) {
    uint32_t e = max(max_bits >> 23, 40u);  // zeros and values below 2^-87: as 2^-87
    if (piece) e = (e + 2) / 4 * 4 + 1;  // biased by 127
    down = __uint_as_float((268u - e) << 23);
    up = __uint_as_float((e - 14u) << 23);
  }
};
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Eight ranks of one row of H in parts; a further part holds what the ones
// before it left (nothing of what is infinite).  Ranks past the last are zeros.
template <bool BF16>
__device__ __forceinline__ void store_h(uint16_t *H, int64_t row, int32_t rank, int32_t j, const float (&h)[8], float by) {
  const int pitch = rank16(rank);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = j >= rank ? 0.0f : h[i] * by;
#pragma unroll
  for (int q = 0; q < kHParts; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack2<BF16>(v[2 * i], v[2 * i + 1]);
      const float2 f = unpack2<BF16>(w[i]);
      v[2 * i] = isinf(f.x) ? 0.0f : v[2 * i] - f.x;
      v[2 * i + 1] = isinf(f.y) ? 0.0f : v[2 * i + 1] - f.y;
    }
    *reinterpret_cast<uint4 *>(H + (row * kHParts + q) * pitch + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) adapter_down_kernel(const __grid_constant__ AdapterDownParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int32_t part = blockIdx.x % p.split;  // rank in the cluster
  const bool second = static_cast<int32_t>(blockIdx.x / p.split) >= p.units;
  const int32_t unit = blockIdx.x / p.split - (second ? p.units : 0);
  const AdapterDownJob &job = p.job[second ? 1 : 0];
  const bool transposed = job.transposed != 0;
  grid_launch_dependents();  // the projection may set up and start on its blocks beside this
  const int stage_bytes = p.stage_bytes;
  Misc *mi = reinterpret_cast<Misc *>(smem + p.q * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n16 = rank16(p.rank);
  uint32_t acc_cols = 32;
  while (static_cast<int>(acc_cols) < n16) acc_cols <<= 1;
  const uint32_t tmem_cols = kNbuf * acc_cols;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      for (int q = 0; q < p.q; ++q) {
        mbar_init(smem_addr(&mi->full[q]), 1);
        mbar_init(smem_addr(&mi->empty[q]), 1);
      }
      for (int b = 0; b < kNbuf; ++b) {
        mbar_init(smem_addr(&mi->acc_full[b]), 1);
        mbar_init(smem_addr(&mi->acc_empty[b]), 4);
      }
      mbar_init(smem_addr(&mi->drained), 1);
      mi->abort_flag = 0;
      fence_barrier_init();
      tma_prefetch_desc(&job.tmX);
      tma_prefetch_desc(&job.tmD);
    }
    __syncwarp();
    const RowPiece r = find_piece(p.seg_ptr, p.seg_adapter, p.n_seg, p.n_adapters, kRows, p.N, unit, p.status);
    if (lane == 0) mi->piece = r;
  } else if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&mi->tmem), tmem_cols);
    tmem_relinquish();
  } else if (warp == kEpiWarp0 && part == 0 && !second && static_cast<int64_t>(unit) * p.tile_rows < p.N) {
    // the projection's own tiles: their segments, for its producers
    const int64_t tile0 = static_cast<int64_t>(unit) * p.tile_rows;
    const int32_t c = list_segments(p.seg_ptr, p.seg_adapter, p.n_seg, p.n_adapters, tile0,
                                    min(tile0 + p.tile_rows, static_cast<int64_t>(p.N)), p.tile_segs + tile0,
                                    p.tile_rows, p.status);
    if (lane == 0) p.tile_count[unit] = c;
    if (p.row_scale) {  // rows outside every segment
      const int64_t b = p.n_seg > 0 ? p.seg_ptr[0] : p.N, e = p.n_seg > 0 ? p.seg_ptr[p.n_seg] : 0;
      for (int64_t n = tile0 + lane; n < min(tile0 + p.tile_rows, static_cast<int64_t>(p.N)); n += 32)
        if (n < b || n >= e) p.row_scale[n] = 0.0f;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = mi->tmem;
  const RowPiece piece = mi->piece;
  const int64_t row0 = static_cast<int64_t>(piece.tile) * kRows;
  const int32_t nk = (job.K + 63) / 64;
  const int32_t k_begin = static_cast<int32_t>(static_cast<int64_t>(nk) * part / p.split);
  const int32_t k_end = static_cast<int32_t>(static_cast<int64_t>(nk) * (part + 1) / p.split);

  if (!BF16 && piece.adapter < 0 && part == 0 && job.rows)
    for (int64_t n = piece.begin + threadIdx.x; n < piece.end; n += kThreads) p.row_scale[n] = 0.0f;
  if (piece.adapter >= 0) {
    if (warp == kTmaWarp) {
      uint32_t stage = 0, phase = 0;
      int64_t seq = 0;
      bool ok = true;
      for (int32_t c = k_begin; c < k_end; ++c) {
        const bool r = mbar_wait_warp(smem_addr(&mi->empty[stage]), phase ^ 1u, p.wait_limit_ns);
        ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = smem_addr(&mi->full[stage]);
          const uint32_t st = smem_addr(smem + stage * stage_bytes);
          mbar_arrive_expect_tx(fb, kXBytes + (transposed ? d_boxes(p.rank) * 8192 : p.rank * 128));
          tma_load_2d(st, &job.tmX, fb, c * 64, static_cast<int32_t>(row0));
          if (transposed)
            for (int b = 0; b < d_boxes(p.rank); ++b)
              tma_load_3d(st + kXBytes + b * 8192, &job.tmD, fb, b * 64, c * 64, piece.adapter);
          else
            tma_load_2d(st + kXBytes, &job.tmD, fb, c * 64, piece.adapter * p.rank);
        }
        __syncwarp();
        ++seq;
        if (++stage == static_cast<uint32_t>(p.q)) {
          stage = 0;
          phase ^= 1u;
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
      const uint32_t idesc = idesc_f16(BF16, false, transposed, kRows, static_cast<uint32_t>(n16));
      const uint32_t lbo = transposed ? 8192 : 16, step = transposed ? 2048 : 32;  // D: groups of 64 ranks, 16 columns
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int32_t c = k_begin; c < k_end; ++c) {
        const int32_t i = c - k_begin;
        const uint32_t turn = i / kTurn, buf = turn % kNbuf, acc = tmem + buf * acc_cols;
        const bool first = i % kTurn == 0;
        if (first) {
          const bool r = mbar_wait_warp(smem_addr(&mi->acc_empty[buf]), ((turn / kNbuf) & 1u) ^ 1u, p.wait_limit_ns);
          ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
          if (!ok) break;
        }
        const bool r = mbar_wait_warp(smem_addr(&mi->full[stage]), phase, p.wait_limit_ns);
        ok = __shfl_sync(0xffffffffu, r && !mi->abort_flag, 0);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t st = smem_addr(smem + stage * stage_bytes);
        const uint64_t x = smem_desc_sw128(st, 16, 1024);
        const uint64_t d = smem_desc_sw128(st + kXBytes, lbo, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_elect(acc, smem_desc_add(x, kk * 32), smem_desc_add(d, kk * step), idesc, (first && kk == 0) ? 0u : 1u);
        umma_commit_elect(smem_addr(&mi->empty[stage]));
        if (c == k_end - 1 || i % kTurn == kTurn - 1) umma_commit_elect(smem_addr(&mi->acc_full[buf]));
        if (++stage == static_cast<uint32_t>(p.q)) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        if (lane == 0) {
          atomicOr(p.status, kDevTimeout);
          mi->abort_flag = 1;
        }
        __syncwarp();
        // nothing may be in flight when the block ends
        umma_commit_elect(smem_addr(&mi->drained));
        mbar_wait_warp(smem_addr(&mi->drained), 0, 1000000ull);
        if (lane == 0)
          for (int b = 0; b < kNbuf; ++b) mbar_arrive(smem_addr(&mi->acc_full[b]));
      }
    }
    if (warp >= kEpiWarp0) {
      const int sp = warp & 3;
      const int r = sp * 32 + lane;
      float *sums = reinterpret_cast<float *>(smem);  // the stages are done with by then
      const float f = p.scale[piece.adapter];
      const bool mine = row0 + r >= piece.begin && row0 + r < piece.end;
      bool ok = true;
      auto wait_acc = [&](uint32_t turn) {
        const bool there = mbar_wait_warp(smem_addr(&mi->acc_full[turn % kNbuf]), (turn / kNbuf) & 1u, p.wait_limit_ns);
        ok = __shfl_sync(0xffffffffu, there && !mi->abort_flag, 0);
        if (!ok && lane == 0) {
          atomicOr(p.status, kDevTimeout);
          mi->abort_flag = 1;
        }
        tc_fence_after_sync();
      };
      auto load16 = [&](uint32_t buf, int c0, uint32_t (&v)[16]) {
        tmem_ld_32x32b_x16(tmem + buf * acc_cols + (static_cast<uint32_t>(sp * 32) << 16) + c0, v);
        tmem_ld_wait();
      };
      float sum[kMaxRank] = {};
      const int32_t turns = (k_end - k_begin + kTurn - 1) / kTurn;
      for (int32_t t = 0; t < turns && ok; ++t) {
        wait_acc(t);
        if (!ok) break;
#pragma unroll
        for (int c0 = 0; c0 < kMaxRank; c0 += 16) {
          if (c0 >= n16) break;
          uint32_t v[16];
          load16(t % kNbuf, c0, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c0 + i] += __uint_as_float(v[i]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&mi->acc_empty[t % kNbuf]));
      }
      if (p.split > 1) {
        if (ok)
#pragma unroll
          for (int c0 = 0; c0 < kMaxRank; c0 += 4) {
            if (c0 >= n16) break;
            *reinterpret_cast<float4 *>(sums + r * part_pitch(p.rank) + c0) =
                make_float4(sum[c0], sum[c0 + 1], sum[c0 + 2], sum[c0 + 3]);
          }
      } else {
        uint32_t top = 0, piece_top = 0;
        if constexpr (!BF16) {
#pragma unroll
          for (int c = 0; c < kMaxRank; c += 8) {
            if (c >= p.rank || !mine) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, finite_bits(f * sum[c + i]));
          }
          if (job.sums) {  // one power of two for the piece
            const uint32_t warp_top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) mi->row_max[sp] = warp_top;
            epilogue_sync();
#pragma unroll
            for (int w = 0; w < 4; ++w) piece_top = max(piece_top, mi->row_max[w]);
          }
        }
        const Power row(top), all(piece_top, true);
        if (mine && ok) {
          if (!BF16 && job.rows) p.row_scale[row0 + r] = row.up;
          if (!BF16 && job.sums) job.sum_scale[row0 + r] = all.up;
#pragma unroll
          for (int c = 0; c < kMaxRank; c += 8) {
            if (c >= n16) break;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = f * sum[c + i];
            if (BF16 || job.rows) store_h<BF16>(job.rows, row0 + r, p.rank, c, o, BF16 ? 1.0f : row.down);
            if (!BF16 && job.sums) store_h<BF16>(job.sums, row0 + r, p.rank, c, o, all.down);
          }
        }
      }
    }
  }
  if (p.split > 1) {
    if (!BF16 && threadIdx.x < kRows) mi->row_max[threadIdx.x] = 0;
    // every CTA of the cluster comes here, whatever happened before
    cluster_sync();
    if (piece.adapter >= 0) {
      // the segment's rows in equal shares
      const int32_t begin = static_cast<int32_t>(piece.begin - row0), n = static_cast<int32_t>(piece.end - piece.begin);
      const int32_t r0 = begin + n * part / p.split, r1 = begin + n * (part + 1) / p.split, units = n16 / 8;
      const uint32_t base = smem_addr(smem);
      const float f = p.scale[piece.adapter];
      float o[8];
      auto each = [&](auto &&eight) {  // eight(row, its first rank, where the eight sums lie)
        for (int u = threadIdx.x; u < (r1 - r0) * units; u += kThreads) {
          const int r = r0 + u / units, j = (u % units) * 8;
          eight(r, j, (r * part_pitch(p.rank) + j) * 4);
        }
      };
      if constexpr (BF16) {
        each([&](int r, int j, int at) {
          cluster_sum8(base + at, p.split, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] *= f;
          store_h<BF16>(job.rows, row0 + r, p.rank, j, o, 1.0f);
        });
      } else {
        // the share's sums in the place of this CTA's own, which no other CTA reads
        each([&](int r, int j, int at) {
          cluster_sum8(base + at, p.split, o);
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] *= f;
            if (j < p.rank) top = max(top, finite_bits(o[i]));
          }
          float4 *own = reinterpret_cast<float4 *>(smem + at);
          own[0] = make_float4(o[0], o[1], o[2], o[3]);
          own[1] = make_float4(o[4], o[5], o[6], o[7]);
          atomicMax(&mi->row_max[r], top);
        });
        __syncthreads();
        uint32_t piece_top = 0;
        if (job.sums) {
          if (warp == 0) {
            uint32_t top = 0;
            for (int r = lane; r < kRows; r += 32) top = max(top, mi->row_max[r]);
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) mi->piece_max = top;
          }
          cluster_sync();
          for (int c = 0; c < p.split; ++c) piece_top = max(piece_top, cluster_load_u32(cluster_map(smem_addr(&mi->piece_max), c)));
        }
        const Power all(piece_top, true);
        each([&](int r, int j, int at) {
          const Power row(mi->row_max[r]);
          const float4 *own = reinterpret_cast<const float4 *>(smem + at);
          const float4 a = own[0], b = own[1];
          o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
          o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
          if (job.rows) {
            if (j == 0) p.row_scale[row0 + r] = row.up;
            store_h<BF16>(job.rows, row0 + r, p.rank, j, o, row.down);
          }
          if (job.sums) {
            if (j == 0) job.sum_scale[row0 + r] = all.up;
            store_h<BF16>(job.sums, row0 + r, p.rank, j, o, all.down);
          }
        });
      }
    }
    cluster_sync();  // the others may still read this CTA's sums
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, tmem_cols);
  }
}

}  // namespace

cudaError_t launch_adapter_down(AdapterDownParams p, int num_sms, bool bf16, cudaStream_t s) {
  // units: see find_piece; about as many have rows
  const int64_t units = (static_cast<int64_t>(p.N) + kRows - 1) / kRows + p.n_seg;
  int32_t k = p.job[0].K, longest = k;
  bool transposed = p.job[0].transposed != 0;
  if (p.jobs > 1) {
    k = k < p.job[1].K ? k : p.job[1].K;
    longest = longest > p.job[1].K ? longest : p.job[1].K;
    transposed = transposed || p.job[1].transposed != 0;
  }
  const int nk = (k + 63) / 64;
  // As many CTAs per unit (a cluster) as keep the grid within two per SM, what an
  // SM holds, with at least four stages each; within four where one product's
  // CTAs are far longer than the other's and would run on alone (gradient of 4096
  // rows through 18944 x 3584: 200 -> 187 us; with four throughout, 1000 rows
  // through 8192 x 8192 take 60 in place of 52 us).
  const int64_t most = (longest >= 2 * k ? 4ll : 2ll) * num_sms;
  p.units = static_cast<int32_t>(units);
  p.split = 1;
  while (p.split < kMaxSplit && p.jobs * units * p.split * 2 <= most && nk >= 8 * p.split) p.split *= 2;
  p.stage_bytes = kXBytes + d_bytes(p.rank, transposed);
  p.q = (kSmemLimit - kMiscBytes - 1024) / p.stage_bytes;
  if (p.q > kMaxQ) p.q = kMaxQ;
  const int smem = p.q * p.stage_bytes + kMiscBytes + 1024;
  auto kern = bf16 ? adapter_down_kernel<true> : adapter_down_kernel<false>;
  const int variant = bf16 ? 1 : 0;
  static std::atomic<uint64_t> smem_set[2];
  cudaError_t e = set_smem_limit_once(kern, kSmemLimit, smem_set[variant]);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> cluster_set[2];
  e = allow_large_clusters_once(kern, cluster_set[variant]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.jobs * units * p.split));
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
